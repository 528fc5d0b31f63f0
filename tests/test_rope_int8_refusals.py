"""rope_table, norm_rope and the 8-bit integer calls refuse on the host, before any launch, what they
do not take: in the C ABI (no GPU needed) and in the binding's checks of tensors."""
import ctypes

import pytest
import torch

import precision_quantized_attention_b200 as qa
from precision_quantized_attention_b200 import _lib

FAKE = ctypes.c_void_p(0x10000)       # aligned, never dereferenced: checks come first
ODD = ctypes.c_void_p(0x10001)
S0 = ctypes.c_void_p(0)
INVALID, UNSUPPORTED = _lib.ERR_INVALID_ARG, _lib.ERR_UNSUPPORTED


def _with(names, ok, kw):
    return [kw.get(n, v) for n, v in zip(names, ok)]


@pytest.mark.parametrize("kw,status", [
    ({"pos": None}, INVALID), ({"table": None}, INVALID), ({"table": ctypes.c_void_p(0x10008)}, INVALID),
    ({"pos": ctypes.c_void_p(0x10002)}, INVALID), ({"type": 2}, INVALID), ({"stride": 2}, INVALID),
    ({"tokens": 0}, INVALID), ({"n": 0}, INVALID), ({"n": 9}, INVALID), ({"dims": (16, 55, 56)}, INVALID),
    ({"dims": (16, 0, 56)}, INVALID), ({"dims": (128, 128, 2)}, UNSUPPORTED), ({"dims": (258, 2, 2)}, INVALID),
    ({"theta": (1e4, 0.0, 1e4)}, INVALID), ({"theta": (1e4, float("nan"), 1e4)}, INVALID),
    ({"tokens": (1 << 30) + 1}, UNSUPPORTED), ({"theta": (float("inf"),) * 3}, INVALID), ({"theta": (1e4, 0.5, 1e4)}, INVALID)])
def test_rope_table_abi(kw, status):
    names = ("pos", "type", "stride", "tokens", "n", "dims", "theta", "table")
    a = _with(names, (FAKE, 0, 3, 16, 3, (16, 56, 56), (1e4,) * 3, FAKE), kw)
    a[5] = (ctypes.c_int * 9)(*a[5])
    a[6] = (ctypes.c_double * 9)(*a[6])
    assert _lib.load().qattn_rope_table(*a, S0) == status


def _io(**kw):
    d = dict(x=0x10000, out=0x10000, weight=0x10000, table=0x10000, x_stride_b=0, x_stride_t=256, x_stride_h=128,
             out_stride_b=0, out_stride_h=2048, out_stride_t=128, H=2, L=16)
    d.update(kw)
    io = _lib.NormRopeIO()
    for k, v in d.items():
        setattr(io, k, v)
    return io


@pytest.mark.parametrize("io,kw,status", [
    ({"x": None}, {}, INVALID), ({"out": None}, {}, INVALID), ({"x": 0x10008}, {}, INVALID),
    ({"out": 0x10008}, {}, INVALID), ({"weight": 0x10004}, {}, INVALID), ({"table": 0x10008}, {}, INVALID),
    ({"H": 0}, {}, INVALID), ({"L": 0}, {}, INVALID), ({"L": 2 ** 31 - 1}, {}, UNSUPPORTED),
    ({"H": 2 ** 31 - 1}, {}, UNSUPPORTED), ({"x_stride_t": 260}, {}, INVALID),
    ({"out_stride_h": 2044}, {}, INVALID), ({"out_stride_h": 0}, {}, INVALID), ({"out_stride_t": 0}, {}, INVALID),
    ({}, {"B": 2}, INVALID),                             # batch rows of the output share elements
    ({"table_stride_b": 2}, {}, INVALID), ({}, {"R": 0}, INVALID), ({}, {"R": 24}, INVALID),
    ({}, {"R": 144}, INVALID), ({}, {"D": 100}, INVALID), ({}, {"D": 0}, INVALID), ({}, {"D": 264}, UNSUPPORTED),
    ({}, {"dtype": 2}, INVALID), ({}, {"eps": -1.0}, INVALID), ({}, {"eps": float("nan")}, INVALID),
    ({}, {"n": 0}, INVALID), ({}, {"n": 13}, UNSUPPORTED), ({}, {"B": 0}, INVALID),
    ({"out_e4m3": 1}, {}, INVALID),                      # codes without amax and scale
    ({"out_e4m3": 1, "amax": 0x10000}, {}, INVALID),
    ({"out_e4m3": 1, "amax": 0x10000, "scale_out": 0x10000, "out": 0x10004}, {}, INVALID),
    ({"amax": 0x10002}, {}, INVALID)])
def test_norm_rope_abi(io, kw, status):
    a = _with(("n", "B", "D", "R", "inter", "eps", "dtype"), (1, 1, 128, 128, 1, 1e-6, 0), kw)
    ios = (_lib.NormRopeIO * 13)(*[_io(**io) for _ in range(13)])
    assert _lib.load().qattn_norm_rope(ios, *a, S0) == status
    assert _lib.load().qattn_norm_rope(None, *a, S0) == INVALID


QUANT = ("x", "ldx", "dtype", "M", "K", "out", "ldo", "scale")
GEMM = ("a8", "lda", "b8", "ldb", "y", "ldy", "dtype", "M", "N", "K", "s_a", "s_b", "bias")


@pytest.mark.parametrize("kw,status", [
    ({"x": None}, INVALID), ({"out": None}, INVALID), ({"scale": None}, INVALID), ({"x": ODD}, INVALID),
    ({"out": ctypes.c_void_p(0x10008)}, INVALID), ({"scale": ctypes.c_void_p(0x10002)}, INVALID), ({"M": 0}, INVALID),
    ({"K": 0}, INVALID), ({"ldx": 99}, INVALID), ({"ldo": 96}, INVALID), ({"ldo": 120}, INVALID),
    ({"dtype": 3}, INVALID), ({"ldo": 1 << 41}, UNSUPPORTED), ({"M": 2 ** 31 - 1}, UNSUPPORTED),
    ({"K": 2 ** 31 - 1, "ldx": 1 << 31, "ldo": 1 << 31}, UNSUPPORTED)])
def test_quantize_int8_rows_abi(kw, status):
    a = _with(QUANT, (FAKE, 100, 0, 4, 100, FAKE, 112, FAKE), kw)
    assert _lib.load().qattn_quantize_int8_rows(*a, S0) == status


@pytest.mark.parametrize("kw,status", [
    ({"a8": None}, INVALID), ({"b8": None}, INVALID), ({"y": None}, INVALID), ({"s_a": None}, INVALID),
    ({"s_b": None}, INVALID), ({"a8": ODD}, INVALID), ({"b8": ctypes.c_void_p(0x10008)}, INVALID), ({"y": ODD}, INVALID),
    ({"bias": ctypes.c_void_p(0x10002)}, INVALID), ({"M": 0}, INVALID), ({"N": 0}, INVALID), ({"K": 0}, INVALID),
    ({"lda": 100}, INVALID), ({"lda": 96}, INVALID), ({"ldb": 104}, INVALID), ({"ldy": 6}, INVALID),
    ({"dtype": -1}, INVALID), ({"K": 131072, "lda": 131072, "ldb": 131072}, UNSUPPORTED),
    ({"lda": 1 << 41}, UNSUPPORTED), ({"M": 1 << 30, "N": 1 << 20, "ldy": 1 << 20}, UNSUPPORTED),
    ({"N": (1 << 30) + 1, "ldy": 1 << 31}, UNSUPPORTED)])
def test_gemm_int8_abi(kw, status):
    ok = (FAKE, 112, FAKE, 112, FAKE, 7, 0, 4, 7, 100, FAKE, FAKE, None)
    a = _with(GEMM, ok, kw)
    assert _lib.load().qattn_gemm_int8(*a, S0) == status
    d = dict(zip(GEMM, a))
    # the same through the linear layer (x valid): x8 and s_x are the GEMM's a8 and s_a
    st = _lib.load().qattn_linear_int8(FAKE, max(d["K"], 1), d["dtype"], d["M"], d["N"], d["K"], d["a8"], d["lda"], d["s_a"],
                                       d["b8"], d["ldb"], d["s_b"], d["bias"], d["y"], d["ldy"], S0)
    assert st == status


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def _refused(match, f, *a, **kw):
    with pytest.raises(ValueError, match=match):
        f(*a, **kw)


def test_binding_refuses_tensors_that_do_not_fit():
    i8, f32 = torch.int8, torch.float32
    _refused("CUDA", qa.quantize_int8_rows, _t(4, 100), _t(4, 112, dtype=i8)[:, :100], _t(4, dtype=f32))
    _refused("2-D", qa.quantize_int8_rows, _t(4, 100, dtype=f32), _t(4, 112, dtype=i8)[:, :100], _t(4, dtype=f32))
    _refused("multiple of 16", qa.quantize_int8_rows, _t(4, 100), _t(4, 100, dtype=i8), _t(4, dtype=f32))
    _refused("contiguous", qa.quantize_int8_rows, _t(100, 4).T, _t(4, 112, dtype=i8)[:, :100], _t(4, dtype=f32))
    _refused("overlap", qa.quantize_int8_rows, _t(100).expand(4, 100), _t(4, 112, dtype=i8)[:, :100], _t(4, dtype=f32))
    gemm = lambda a=_t(4, 112, dtype=i8), b=_t(7, 112, dtype=i8), y=_t(4, 7), sa=_t(4, dtype=f32), sb=_t(7, dtype=f32), bias=None: \
        qa.gemm_int8(a, b, y, sa, sb, bias)
    _refused("CUDA", gemm)
    _refused("b8 must be", gemm, b=_t(7, 96, dtype=i8))
    _refused("a8 must be", gemm, a=_t(3, 112, dtype=i8))
    _refused("2-D", gemm, y=_t(4, 7, dtype=f32))
    _refused("type", qa.linear_int8, _t(4, 112), _t(4, 112, dtype=i8), _t(4, dtype=f32), _t(7, 112, dtype=i8),
             _t(7, dtype=f32), _t(4, 7, dtype=torch.float16))
    pos = _t(5, 3, dtype=torch.int32)
    _refused("CUDA", qa.rope_table, pos, (16, 56, 56), _t(5, 64, 2, dtype=f32))
    _refused("positions", qa.rope_table, pos.long(), (16, 56, 56), _t(5, 64, 2, dtype=f32))
    _refused("table must be", qa.rope_table, pos, (16, 56, 56), _t(5, 32, 2, dtype=f32))
    _refused("theta", qa.rope_table, pos, (16, 56, 56), _t(5, 64, 2, dtype=f32), theta=(1.0, 2.0))
    seg = lambda x=_t(1, 5, 2, 64), out=_t(1, 2, 5, 64), **kw: qa.norm_rope([qa.NormRopeSegment(x, out, **kw)])
    _refused("CUDA", seg)
    _refused("1 to 12", qa.norm_rope, [])
    _refused("bfloat16", seg, x=_t(1, 5, 2, 64, dtype=f32))


@pytest.mark.gpu
def test_binding_refuses_device_tensors_that_do_not_fit():
    f32, u8 = torch.float32, torch.uint8
    c = lambda *s, dtype=torch.bfloat16: _t(*s, dtype=dtype).cuda()
    seg = lambda x=c(1, 5, 2, 64), out=c(1, 2, 5, 64), **kw: qa.norm_rope([qa.NormRopeSegment(x, out, **kw)])
    _refused("out must be", seg, out=c(1, 5, 2, 64))
    _refused("x's type", seg, out=c(1, 2, 5, 64, dtype=torch.float16))
    _refused("amax and scale", seg, out=c(1, 2, 5, 64, dtype=u8))
    _refused("weight", seg, weight=c(32, dtype=f32))
    _refused("weight", seg, weight=c(64))
    _refused("table must be", seg, table=c(4, 32, 2, dtype=f32))
    _refused("table must be", seg, table=c(5, 32, 2))
    _refused("rows of a table", seg, table=c(5, 64, 2, dtype=f32)[:, ::2])
    _refused("channels", seg, x=c(1, 5, 2, 128)[..., ::2])
    _refused("same number of pairs", qa.norm_rope,
             [qa.NormRopeSegment(c(1, 5, 2, 64), c(1, 2, 5, 64), table=c(5, r, 2, dtype=f32)) for r in (32, 16)])
    _refused("same type", qa.norm_rope,
             [qa.NormRopeSegment(c(1, 5, 2, d), c(1, 2, 5, d)) for d in (64, 128)])
    _refused("is on cpu", seg, weight=_t(64, dtype=f32))
    with pytest.raises(qa.QattnError):               # rows 8 bytes off
        seg(x=c(1, 5, 2, 72)[..., 4:68])
    _refused("contiguous float32", qa.gemm_int8, c(4, 112, dtype=torch.int8), c(8, 112, dtype=torch.int8), c(4, 8),
             c(3, dtype=f32), c(8, dtype=f32))
    _refused("int8", qa.gemm_int8, c(4, 112, dtype=u8), c(8, 112, dtype=torch.int8), c(4, 8), c(4, dtype=f32), c(8, dtype=f32))
    with pytest.raises(qa.QattnError):               # no tokens
        qa.linear_int8(c(0, 112), c(0, 112, dtype=torch.int8), c(0, dtype=f32), c(8, 112, dtype=torch.int8),
                       c(8, dtype=f32), c(0, 8))
    assert qa.get_error() == 0
