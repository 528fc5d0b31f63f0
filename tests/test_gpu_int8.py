"""quantize_int8_rows, gemm_int8, linear_int8 and Int8Linear against their definitions: codes and scales
bit for bit; products from exact integer sums, so that the bar is half a step of the 16-bit output plus the
FP32 roundings behind the sum (its conversion, two scales and the bias: 4 of 2^-24 of the terms)."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle
import precision_quantized_attention_b200 as qa
from precision_quantized_attention_b200 import _lib

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U = 2.0 ** -24


def _padded(rows, cols, extra=0, fill=0x33):
    """int8 [rows, cols] on a row stride that is a multiple of 16, within a larger buffer."""
    ld = -(-cols // 16) * 16 + extra
    whole = torch.full((rows + 2, ld), fill, dtype=torch.int8, device="cuda")
    return whole, whole[1:rows + 1, :cols]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,K", [(1, 1), (3, 7), (5, 8), (9, 100), (2, 1024), (7, 1025), (3, 4096), (4, 4097),
                                 (2, 8192), (3, 8200), (2, 12288), (3, 12300), (2, 16384), (2, 16385), (3, 40000), (300, 64),
                                 (513, 1100)])
def test_quantize_rows(M, K, dtype):
    g = torch.Generator().manual_seed(M * K)
    x = torch.randn(M, K, generator=g) * torch.exp(4 * torch.randn(M, 1, generator=g))
    if K >= 7:
        x[0] = torch.arange(K) % 7 * 0.5             # ties: 127 * 0.5 / 3 is none, 127 * 1.5 / 3 = 63.5
        x[-1] *= 0.0 if M > 2 else 1.0
    x = x.to(dtype)
    finite = x.isfinite().all(1)                     # FP16 overflows in some rows: scale NaN, codes 0
    want, scale = oracle.quantize_int8_rows(torch.where(finite[:, None], x, 0).double().numpy())
    scale[~finite.numpy()] = np.nan
    status = 0 if finite.all() else _lib.ERR_NONFINITE
    for pad in (0, 3, 8):                            # contiguous, odd and 16-byte row strides
        xd = torch.zeros(M, K + pad, dtype=dtype, device="cuda")[:, :K]
        xd.copy_(x)
        whole, out = _padded(M, K, extra=16)
        s = torch.zeros(M, device="cuda")
        qa.quantize_int8_rows(xd, out, s)
        assert qa.get_error() == status
        assert np.array_equal(s.cpu().numpy(), scale, equal_nan=True)
        assert np.array_equal(out.cpu().numpy(), want)
        rest = whole.clone()
        rest[1:M + 1, :K] = 0x33
        assert bool((rest == 0x33).all())            # nothing else was written


def test_every_bf16_pair_of_element_and_maximum_rounds_right():
    """All mantissas of the element against all mantissas of the maximum, in exponents from the type's
    smallest to its largest: no quotient is rounded to the wrong side, ties go to even."""
    man = np.arange(128)
    for e in (0, 1, 60, 127, 200, 246, 254):         # exponent field of the maximum
        for de in (0, 1, 3, 6, 8):
            if e < de:
                continue
            bits = np.empty((128, 130), dtype=np.uint16)
            bits[:, 0] = (e << 7) | man              # the row's maximum (its largest exponent)
            bits[:, 1:129] = np.where(((e - de) << 7 | man) <= ((e << 7) | man)[:, None], ((e - de) << 7) | man, 0)
            bits[:, 129] = bits[:, 0] | 0x8000
            x = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16)
            want, scale = oracle.quantize_int8_rows(x.double().numpy())
            _, out = _padded(128, 130)
            s = torch.zeros(128, device="cuda")
            qa.quantize_int8_rows(x.cuda(), out, s)
            assert qa.get_error() == 0
            assert np.array_equal(out.cpu().numpy(), want), (e, de)
            assert np.array_equal(s.cpu().numpy(), scale), (e, de)


def test_nonfinite_row_is_reported_and_alone():
    x = torch.randn(5, 72, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    want, scale = oracle.quantize_int8_rows(x.double().numpy())
    for bad in (float("nan"), float("inf"), float("-inf")):
        y = x.clone()
        y[3, 71] = bad
        _, out = _padded(5, 72)
        s = torch.zeros(5, device="cuda")
        qa.quantize_int8_rows(y.cuda(), out, s)
        assert qa.get_error() == _lib.ERR_NONFINITE
        assert s[3].isnan().item() and not out[3].any().item()
        keep = [0, 1, 2, 4]
        assert np.array_equal(out.cpu().numpy()[keep], want[keep]) and np.array_equal(s.cpu().numpy()[keep], scale[keep])


def _operands(M, N, K, seed, bias=True):
    rng = np.random.default_rng(seed)
    a, b = (rng.integers(-128, 128, size=(r, K), dtype=np.int8) for r in (M, N))
    sa = np.exp(rng.normal(size=M)).astype(np.float32) * np.float32(1e-3)
    sb = np.exp(rng.normal(size=N)).astype(np.float32) * np.float32(1e-3)
    return a, b, sa, sb, rng.normal(size=N).astype(np.float32) if bias else None


def _gemm(a, b, sa, sb, bias, dtype=torch.bfloat16, ldy_extra=0):
    (M, K), N = a.shape, b.shape[0]
    dev = []
    for t in (a, b):
        _, d = _padded(t.shape[0], K, extra=16)
        d.copy_(torch.from_numpy(t))
        dev.append(d)
    whole = torch.full((M + 2, N + ldy_extra), 9.0, dtype=dtype, device="cuda")
    y = whole[1:M + 1, :N]
    v = lambda t: None if t is None else torch.from_numpy(t).cuda()
    qa.gemm_int8(dev[0], dev[1], y, v(sa), v(sb), v(bias))
    assert qa.get_error() == 0
    rest = whole.clone()
    rest[1:M + 1, :N] = 9.0
    assert bool((rest == 9.0).all())                 # rows and columns around the output are as they were
    return y


def _check(y, a, b, sa, sb, bias):
    want, size = oracle.gemm_int8(a, b, sa, sb, bias)
    got = y.double().cpu().numpy()
    if y.dtype == torch.float16:
        big = np.abs(want) >= 65504.0
        assert not big.any()
    tol = 4 * U * size + torch.finfo(y.dtype).eps / 2 * (np.abs(want) + 4 * U * size) + (2.0 ** -25 if y.dtype == torch.float16 else 0)
    off = np.abs(got - want)
    assert (off <= tol).all(), f"worst {np.max(off / tol):.3f} of the bar"


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 31, 33, 64, 65, 127, 128, 129, 200, 256, 257, 385, 513])
@pytest.mark.parametrize("N,K", [(1, 1), (7, 15), (33, 128), (127, 129), (128, 640), (257, 1000), (1000, 2064)])
def test_gemm_shapes(M, N, K):
    """Every token-tile size, ragged row, column and K tiles, clusters of several sizes (few weight rows
    with a long K) and pairs of SMs."""
    ops = _operands(M, N, K, seed=M + N + K, bias=(M + N) % 2 == 0)
    dtype = torch.float16 if (M + K) % 3 == 0 else torch.bfloat16
    _check(_gemm(*ops, dtype=dtype, ldy_extra=(M % 3) * 4), *ops)


@pytest.mark.parametrize("M,N,K", [(4, 128, 16384), (100, 384, 8192), (24, 4096, 1920), (1, 20000, 512),
                                   (1200, 2100, 700), (640, 5000, 320), (1000, 4090, 4100), (260, 5301, 1030),
                                   (300, 6904, 1100), (520, 4700, 1200)])
def test_gemm_larger(M, N, K):
    """Long sums over clusters, and shapes that take tiles of 160, 128, 256, 160, 192 and 224 columns on 74 pairs."""
    ops = _operands(M, N, K, seed=K)
    _check(_gemm(*ops), *ops)


@pytest.mark.parametrize("M", [2, 130])
def test_longest_sums_stay_exact(M):
    """K at its limit with every product at its largest: the int32 sums reach 2^31 - 2^14; outputs equal the
    rounded definition."""
    K, N = 131071, 5
    a, b = np.full((M, K), -128, np.int8), np.full((N, K), -128, np.int8)
    b[1], b[2, 0], b[3] = 127, 127, 0
    ops = (a, b, np.full(M, 1e-4, np.float32), np.full(N, 1e-4, np.float32), None)
    _check(_gemm(*ops), *ops)


def test_result_does_not_depend_on_the_path():
    """The first rows of a product are the same bits whether few tokens or many are in the call."""
    a, b, sa, sb, bias = _operands(700, 515, 1100, seed=8)
    y = _gemm(a, b, sa, sb, bias)
    for M in (1, 16, 30, 64, 128, 129, 256, 512):
        assert torch.equal(_gemm(a[:M], b, sa[:M], sb, bias), y[:M])


def test_offsets_past_32_bits():
    """Rows of the output and of the codes more than 2^31 elements apart."""
    M, N, K = 3, 40, 48
    a, b, sa, sb, _ = _operands(M, N, K, seed=4)
    far = 2 ** 30 + 16
    y = torch.empty(2 * far + N, dtype=torch.bfloat16, device="cuda").as_strided((M, N), (far, 1))
    w8 = torch.empty(2 * (2 ** 31) + K, dtype=torch.int8, device="cuda").as_strided((3, K), (2 ** 31, 1))
    w8.copy_(torch.from_numpy(a))
    v = lambda t: torch.from_numpy(t).cuda()
    qa.gemm_int8(w8, v(b), y, v(sa), v(sb))
    assert qa.get_error() == 0
    _check(y, a, b, sa, sb, None)
    x = torch.empty(2 * far + K, dtype=torch.bfloat16, device="cuda").as_strided((M, K), (far, 1))
    x.copy_(torch.from_numpy(a).to(torch.bfloat16))
    s = torch.zeros(M, device="cuda")
    qa.quantize_int8_rows(x, w8, s)
    want, scale = oracle.quantize_int8_rows(x.double().cpu().numpy())
    assert np.array_equal(w8.cpu().numpy(), want) and np.array_equal(s.cpu().numpy(), scale)


@pytest.mark.parametrize("M,N,K,dtype", [(1, 96, 200, torch.bfloat16), (2, 5001, 1003, torch.float16), (1, 40, 100000, torch.bfloat16),
                                         (2, 300, 4096, torch.bfloat16), (20, 515, 1003, torch.float16), (300, 260, 512, torch.bfloat16)])
def test_linear_is_its_two_calls(M, N, K, dtype):
    g = torch.Generator().manual_seed(M)
    x = torch.randn(M, K, generator=g).to(dtype).cuda()
    w = (torch.randn(N, K, generator=g) * K ** -0.5).to(dtype).cuda()
    bias = torch.randn(N, generator=g).cuda()
    layer = qa.Int8Linear(w, bias, max_tokens=512)
    x8, s = _padded(M, K)[1], torch.zeros(M, device="cuda")
    y = torch.empty(M, N, dtype=dtype, device="cuda")
    qa.quantize_int8_rows(x, x8, s)
    qa.gemm_int8(x8, layer.w8, y, s, layer.s_w, bias)
    got = layer(x)
    assert qa.get_error() == 0
    assert torch.equal(got, y)
    assert torch.equal(layer._x8[:M], x8) and torch.equal(layer._s_x[:M], s)
    assert layer(x[:0]).shape == (0, N)
    xc, xs = oracle.quantize_int8_rows(x.double().cpu().numpy())
    wc, ws = oracle.quantize_int8_rows(w.double().cpu().numpy())
    assert np.array_equal(x8.cpu().numpy(), xc) and np.array_equal(layer.w8.cpu().numpy(), wc)
    _check(got, xc, wc, xs, ws, bias.cpu().numpy())
    assert torch.equal(layer(x.view(1, M, K)), y.view(1, M, N))
    with pytest.raises(ValueError):
        layer(torch.zeros(513, K, dtype=dtype, device="cuda"))


@pytest.mark.parametrize("M", [1, 2, 40, 200])
def test_linear_in_the_place_of_its_input_and_with_its_own_codes(M):
    """y = x, and the product of the tokens' codes with themselves."""
    K = 768
    g = torch.Generator().manual_seed(M)
    x = torch.randn(M, K, generator=g).to(torch.bfloat16).cuda()
    layer = qa.Int8Linear((torch.randn(K, K, generator=g) * K ** -0.5).to(torch.bfloat16).cuda())
    want = layer(x)
    for _ in range(20):
        y = x.clone()
        assert layer(y, out=y).data_ptr() == y.data_ptr()
        assert torch.equal(y, want)
    x8, s = _padded(M, K)[1], torch.zeros(M, device="cuda")
    gram = torch.empty(M, M, dtype=torch.bfloat16, device="cuda")
    for i in range(5):
        qa.linear_int8(x * (i + 1), x8, s, x8, s, gram)
        codes, scale = oracle.quantize_int8_rows((x * (i + 1)).double().cpu().numpy())
        _check(gram, codes, codes, scale, scale, None)
    assert qa.get_error() == 0


def test_first_calls_of_a_process_inside_a_capture():
    """Nothing of the set-up needs a call outside the capture (buffers and codes exist)."""
    code = ("import torch, precision_quantized_attention_b200 as qa\n"
            "x = torch.randn(1, 5, 2, 64, device='cuda').to(torch.bfloat16); w = torch.ones(64, device='cuda')\n"
            "o = torch.zeros(1, 2, 5, 64, dtype=torch.bfloat16, device='cuda'); t = torch.zeros(5, 32, 2, device='cuda')\n"
            "p = torch.arange(5, dtype=torch.int32, device='cuda')[:, None]\n"
            "rows = [torch.randn(m, 1024, device='cuda').to(torch.bfloat16) for m in (1, 20, 200)]\n"
            "w8 = torch.ones(256, 1024, dtype=torch.int8, device='cuda'); sw = torch.ones(256, device='cuda')\n"
            "x8 = [torch.zeros(r.shape[0], 1024, dtype=torch.int8, device='cuda') for r in rows]\n"
            "sx = [torch.zeros(r.shape[0], device='cuda') for r in rows]\n"
            "y = [torch.zeros(r.shape[0], 256, dtype=torch.bfloat16, device='cuda') for r in rows]\n"
            "torch.cuda.synchronize()\n"
            "def step():\n"
            "    qa.rope_table(p, (64,), t); qa.norm_rope([qa.NormRopeSegment(x, o, weight=w, table=t)])\n"
            "    for r, a, s, b in zip(rows, x8, sx, y): qa.linear_int8(r, a, s, w8, sw, b)\n"
            "g = torch.cuda.CUDAGraph()\n"
            "with torch.cuda.graph(g): step()\n"
            "g.replay(); torch.cuda.synchronize()\n"
            "got = [o.clone()] + [b.clone() for b in y]\n"
            "step(); assert qa.get_error() == 0\n"
            "assert all(torch.equal(a, b) for a, b in zip(got, [o] + y)) and o.abs().sum() > 0 and y[2].abs().sum() > 0\n"
            "print('captured')\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, (r.stdout + r.stderr)[-3000:]


def test_linear_nonfinite_token_gives_nan_in_its_row_only():
    g = torch.Generator().manual_seed(7)
    x = torch.randn(40, 128, generator=g).to(torch.bfloat16).cuda()
    layer = qa.Int8Linear(torch.randn(64, 128, generator=g).to(torch.bfloat16).cuda(), torch.ones(64).cuda())
    want = layer(x)
    x[11, 5] = float("inf")
    y = layer(x)
    assert qa.get_error() == _lib.ERR_NONFINITE
    assert bool(y[11].isnan().all())
    keep = torch.arange(40, device="cuda") != 11
    assert torch.equal(y[keep], want[keep])


def test_linear_back_to_back_on_two_streams_and_in_graphs():
    """Calls in a row reuse their buffers of codes while the next one's quantize starts; two layers on
    two streams; a captured call replayed with new inputs between eager ones."""
    g = torch.Generator().manual_seed(9)
    K, N = 2048, 1536
    layers = [qa.Int8Linear((torch.randn(N, K, generator=g) * K ** -0.5).to(torch.bfloat16).cuda()) for _ in range(2)]
    xs = [torch.randn(m, K, generator=g).to(torch.bfloat16).cuda() for m in (3, 40, 300, 1, 128, 700)]

    def slow(layer, x):
        x8, s = _padded(x.shape[0], K)[1], torch.zeros(x.shape[0], device="cuda")
        y = torch.empty(x.shape[0], N, dtype=torch.bfloat16, device="cuda")
        qa.quantize_int8_rows(x, x8, s)
        torch.cuda.synchronize()
        qa.gemm_int8(x8, layer.w8, y, s, layer.s_w)
        torch.cuda.synchronize()
        return y

    want = [[slow(layer, x) for x in xs] for layer in layers]
    for _ in range(3):
        got = [layers[0](x) for x in xs]
        assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    streams = [torch.cuda.Stream() for _ in layers]
    outs = [[torch.empty_like(w) for w in ws] for ws in want]
    torch.cuda.synchronize()
    for _ in range(4):
        for i, layer in enumerate(layers):
            with torch.cuda.stream(streams[i]):
                for x, o in zip(xs, outs[i]):
                    layer(x, out=o)
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(outs[i], want[i]))
    x, o = xs[1].clone(), torch.empty_like(want[0][1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layers[0](x, out=o)
        o2 = layers[1](x)
    graph.replay()
    eager = layers[0](xs[2])
    assert torch.equal(o, want[0][1]) and torch.equal(o2, want[1][1]) and torch.equal(eager, want[0][2])
    x.copy_(xs[5][:40])
    graph.replay()
    assert torch.equal(o, slow(layers[0], xs[5][:40]))
    assert qa.get_error() == 0


@pytest.mark.skipif(_lib.CHECKED, reason="starts the checked-build run")
def test_rope_and_int8_suites_pass_in_the_checked_build():
    from precision_quantized_attention_b200 import build
    build.build(checked=True)
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", "tests/test_gpu_rope.py",
           "tests/test_gpu_int8.py", "tests/test_gpu_block.py", "-k", "not past_32_bits and not every_bf16"]
    r = subprocess.run(cmd, cwd=ROOT, env=dict(os.environ, QATTN_DEBUG="1"), capture_output=True, text=True, timeout=1500)
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
