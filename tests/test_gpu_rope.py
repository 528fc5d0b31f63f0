"""rope_table and norm_rope against their FP64 definitions.

Bars (u = 2^-24): a table entry is off by the rest's rounding (2^-28 turns, 2^-25 in angle), one ulp of
the 32-bit sine or cosine (2^-23), and the 64-bit product (2^-50 of the angle, the oracle's own
rounding included).  A normed and rotated value: the sum of D squares (a lane's 8, then at most 5 shuffles)
halves to 7 u, mean and eps u, rsqrt 2 ulp = 4 u, coefficient, its product with r, the product and the sum
4 u, and the FP32 weight and table are inputs: 16 u, 24 allowed, of the magnitudes of its terms; then half a
step of the 16-bit type.  An E4M3 code lies between the codes of the ends of the FP32 value's bar (28 u: two
roundings of 1 / scale and one of the product more); a copied tensor's codes are exact."""
import numpy as np
import pytest
import torch

import oracle
import precision_quantized_attention_b200 as qa
from precision_quantized_attention_b200 import _lib

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _table(pos, dims, theta):
    table = torch.full((pos.shape[0], sum(dims) // 2, 2), 7.0, device="cuda")
    qa.rope_table(pos, dims, table, theta=theta)
    assert qa.get_error() == 0
    return table


@pytest.mark.parametrize("dims,theta,tokens", [((16, 56, 56), 10000.0, 1), ((16, 56, 56), 10000.0, 333),
                                               ((44, 42, 42), (1e4, 3e4, 5e5), 70001), ((128,), 500000.0, 9),
                                               ((2,), 10.0, 5), ((64, 64, 64, 64), 1e4, 77),
                                               ((2,) * 8, 1e4, 1000)])
@pytest.mark.parametrize("kind", ["int", "far", "float"])
def test_rope_table(dims, theta, tokens, kind):
    g = torch.Generator().manual_seed(len(dims) * tokens)
    n = len(dims)
    if kind == "int":
        pos = torch.randint(0, 5000, (tokens, n), generator=g, dtype=torch.int32)
    elif kind == "far":
        pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (tokens, n), generator=g, dtype=torch.int64).to(torch.int32)
        pos[0] = -2 ** 31
        pos[-1] = 2 ** 31 - 1
    else:
        pos = torch.randn(tokens, n, generator=g) * 100.0
    got = _table(pos.cuda(), dims, theta).double().cpu().numpy()
    bases = theta if isinstance(theta, tuple) else (theta,) * n
    a = oracle.rope_angles(pos.numpy(), dims, bases)
    tol = 2.0 ** -25 + 2.0 ** -23 + np.abs(a) * 2.0 ** -50
    assert (np.abs(got[..., 0] - np.cos(a)) <= tol).all()
    assert (np.abs(got[..., 1] - np.sin(a)) <= tol).all()


def test_rope_table_strided_positions_and_nothing_behind():
    pos = torch.arange(60, dtype=torch.int32, device="cuda").view(12, 5)
    whole = torch.full((20, 32, 2), -3.0, device="cuda")
    qa.rope_table(pos[:, 1:4], (16, 24, 24), whole[4:16])
    want = _table(pos[:, 1:4].contiguous(), (16, 24, 24), 10000.0)
    assert torch.equal(whole[4:16], want)
    assert bool((whole[:4] == -3.0).all()) and bool((whole[16:] == -3.0).all())


def test_rope_table_nonfinite_position_stays_in_its_axis():
    pos = torch.tensor([[1.0, 2.0], [float("nan"), 3.0], [float("inf"), 4.0]], device="cuda")
    t = _table(pos, (4, 4), 100.0)
    assert bool(t[1:, :2].isnan().all()) and bool(t[:, 2:].isfinite().all()) and bool(t[0].isfinite().all())


def _check(got, x, weight, table, eps, inter, dtype):
    """got [B, H, L, D] of dtype against the definition, on the CPU."""
    want, size = oracle.norm_rope(x.double().cpu().numpy(), None if weight is None else weight.double().cpu().numpy(),
                                  None if table is None else table.double().cpu().numpy(), eps, inter)
    half = torch.finfo(dtype).eps / 2
    tol = 24 * U * size + half * (np.abs(want) + 24 * U * size)
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25                       # half a step of its subnormals
    off = np.abs(got.double().cpu().numpy() - want)
    assert (off <= tol).all(), f"worst {np.max(off / tol):.3f} of the bar"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("inter", [True, False])
@pytest.mark.parametrize("B,L,H,Hkv,D,R", [(1, 1, 1, 1, 8, 0), (1, 1, 32, 8, 128, 128), (2, 5, 3, 1, 16, 16),
                                           (1, 37, 5, 5, 32, 16), (3, 9, 7, 2, 64, 32), (1, 130, 24, 24, 128, 128),
                                           (2, 33, 6, 3, 96, 96), (2, 11, 3, 3, 96, 64), (1, 17, 4, 2, 256, 256),
                                           (1, 3, 9, 4, 184, 48), (1, 700, 2, 2, 64, 64)])
def test_norm_rope_from_a_projection(B, L, H, Hkv, D, R, inter, dtype):
    """Q, K, V slices of one projection's output, small and odd lengths, grouped heads, head sizes that
    do not fill the lanes, partial rotation; V is copied bit for bit; nothing else is written."""
    g = torch.Generator().manual_seed(B * 1000 + L + H + D + R)
    qkv = (torch.randn(B, L, (H + 2 * Hkv) * D, generator=g) * torch.exp(torch.randn(B, L, 1, generator=g))).to(dtype).cuda()
    q, k, v = qkv.view(B, L, H + 2 * Hkv, D).split([H, Hkv, Hkv], 2)
    w = (1.0 + 0.2 * torch.randn(2, D, generator=g)).cuda()
    table = None
    if R:
        a = torch.rand(L, R // 2, generator=g, dtype=torch.float64) * 100
        table = torch.stack([a.cos(), a.sin()], -1).float().cuda()
    outs = [torch.full((B, h, L + 2, D), 5.0, dtype=dtype, device="cuda") for h in (H, Hkv, Hkv)]
    seg = qa.NormRopeSegment
    qa.norm_rope([seg(q, outs[0][:, :, 1:L + 1], weight=w[0], table=table),
                  seg(k, outs[1][:, :, 1:L + 1], weight=w[1], table=table),
                  seg(v, outs[2][:, :, 1:L + 1])], eps=1e-5, interleaved=inter)
    assert qa.get_error() == 0
    _check(outs[0][:, :, 1:L + 1], q, w[0], table, 1e-5, inter, dtype)
    _check(outs[1][:, :, 1:L + 1], k, w[1], table, 1e-5, inter, dtype)
    assert torch.equal(outs[2][:, :, 1:L + 1].view(torch.int16), v.transpose(1, 2).contiguous().view(torch.int16))
    for o in outs:
        assert bool((o[:, :, 0] == 5.0).all()) and bool((o[:, :, L + 1] == 5.0).all())


@pytest.mark.parametrize("inter", [True, False])
def test_parts_of_it_alone_and_tables_of_batch_rows(inter):
    """The rotation without the norm, the norm without the rotation, a table for each batch row."""
    B, L, H, D, R = 3, 21, 4, 64, 48
    g = torch.Generator().manual_seed(3)
    x = torch.randn(B, L, H, D, generator=g).to(torch.bfloat16).cuda()
    a = torch.rand(B, L, R // 2, generator=g, dtype=torch.float64) * 50
    table = torch.stack([a.cos(), a.sin()], -1).float().cuda()
    w = torch.randn(D, generator=g).cuda()
    outs = [torch.empty(B, H, L, D, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    qa.norm_rope([qa.NormRopeSegment(x, outs[0], table=table), qa.NormRopeSegment(x, outs[1], weight=w),
                  qa.NormRopeSegment(x, outs[2], weight=w, table=table)], interleaved=inter)
    assert qa.get_error() == 0
    _check(outs[0], x, None, table, 1e-6, inter, torch.bfloat16)
    _check(outs[1], x, w, None, 1e-6, inter, torch.bfloat16)
    _check(outs[2], x, w, table, 1e-6, inter, torch.bfloat16)


def test_zero_rows_need_eps_only():
    x = torch.zeros(1, 3, 2, 64, dtype=torch.bfloat16, device="cuda")
    x[0, 1] = 1e-20
    out = torch.empty(1, 2, 3, 64, dtype=torch.bfloat16, device="cuda")
    qa.norm_rope([qa.NormRopeSegment(x, out, weight=torch.ones(64, device="cuda"))], eps=1e-6)
    assert qa.get_error() == 0
    _check(out, x, torch.ones(64), None, 1e-6, True, torch.bfloat16)


def _e4m3(y, amax):
    """Codes of the framework's per-tensor FP8 quantize of a 16-bit tensor, on the CPU."""
    s = np.float32(1.0) if amax == 0 else np.float32(amax) / np.float32(448.0)
    with np.errstate(over="ignore"):
        q = y.float().cpu().numpy() / s
    return torch.from_numpy(q).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), s


def check_codes(codes, scale, x, weight, table, eps, inter):
    """Codes [B, H, L, D] of a normed and rotated tensor: between those of the ends of the value's bar."""
    host = lambda t: None if t is None else t.double().cpu().numpy()
    want, size = oracle.norm_rope(host(x), host(weight), host(table), eps, inter)
    value = lambda v: torch.from_numpy(np.clip(v / scale, -448.0, 448.0)).float().to(torch.float8_e4m3fn).float().numpy()
    got = codes.cpu().view(torch.float8_e4m3fn).float().numpy()
    assert (value(want - 28 * U * size) <= got).all() and (got <= value(want + 28 * U * size)).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D,R,inter", [(128, 128, True), (64, 64, False), (96, 32, False), (256, 256, False)])
@pytest.mark.parametrize("amax", [3.0, 0.0, 1e-38, 2e-2, 3e38])
def test_codes(D, R, inter, dtype, amax):
    """Also with an amax below the largest value (saturation), of zero, and so small or large that the
    scale leaves the range of the fast path.  The copied tensor's are the framework's own quantize."""
    B, L, H = 2, 45, 6
    g = torch.Generator().manual_seed(D)
    x = torch.randn(B, L, H, D, generator=g).to(dtype).cuda()
    w = (1 + 0.1 * torch.randn(D, generator=g)).cuda()
    a = torch.rand(L, R // 2, generator=g) * 9
    table = torch.stack([a.cos(), a.sin()], -1).cuda()
    c = [torch.full((B, H, L + 1, D), 0x55, dtype=torch.uint8, device="cuda") for _ in range(3)]
    am, sc = torch.full((3,), amax, device="cuda"), torch.zeros(3, device="cuda")
    qa.norm_rope([qa.NormRopeSegment(x, c[0][:, :, :L], weight=w, table=table, amax=am[:1], scale=sc[:1]),
                  qa.NormRopeSegment(x, c[1][:, :, :L], amax=am[1:2], scale=sc[1:2]),
                  qa.NormRopeSegment(x, c[2][:, :, :L], table=table, amax=am[2:], scale=sc[2:])], interleaved=inter)
    assert qa.get_error() == 0
    want, s = _e4m3(x.transpose(1, 2).contiguous(), np.float32(amax))
    for i in range(3):
        assert np.float32(sc[i].item()) == s
        assert bool((c[i][:, :, L] == 0x55).all())
    assert torch.equal(c[1][:, :, :L].cpu(), want)
    check_codes(c[0][:, :, :L], float(s), x, w, table, 1e-6, inter)
    check_codes(c[2][:, :, :L], float(s), x, None, table, 1e-6, inter)
    if dtype == torch.bfloat16:
        code, scale = torch.empty_like(want, device="cuda"), torch.zeros(1, device="cuda")
        qa.quantize_fp8(x.transpose(1, 2).contiguous(), am[:1], code, scale)
        assert torch.equal(code.cpu(), want)


def test_running_amax_joins_streams_and_calls():
    D, H = 64, 3
    g = torch.Generator().manual_seed(11)
    amax = torch.zeros(1, device="cuda")
    most = 0.0
    for L in (4, 301):
        x = [(torch.randn(1, n, H, D, generator=g) * 3).to(torch.bfloat16).cuda() for n in (L, 7)]
        out = torch.empty(1, H, L + 7, D, dtype=torch.bfloat16, device="cuda")
        qa.norm_rope([qa.NormRopeSegment(x[0], out[:, :, :L], amax=amax), qa.NormRopeSegment(x[1], out[:, :, L:], amax=amax)])
        most = max(most, out.abs().max().item())
        assert amax.item() == most
    assert qa.get_error() == 0


def test_nonfinite_elements_are_reported_and_stay_in_their_rows():
    D, H, L = 128, 2, 6
    x = torch.randn(1, L, H, D, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).cuda()
    w = torch.ones(D, device="cuda")
    clean = torch.empty(1, H, L, D, dtype=torch.bfloat16, device="cuda")
    out, v, codes = torch.empty_like(clean), torch.empty_like(clean), torch.empty_like(clean, dtype=torch.uint8)
    qa.norm_rope([qa.NormRopeSegment(x, clean, weight=w)])
    assert qa.get_error() == 0
    for bad in (float("nan"), float("inf"), 3e38):       # the last: finite, its square is not
        y = x.clone()
        y[0, 2, 1, 9] = bad
        qa.norm_rope([qa.NormRopeSegment(y, out, weight=w)])
        assert qa.get_error() == _lib.ERR_NONFINITE
        ok = torch.ones(1, H, L, 1, dtype=torch.bool, device="cuda")
        ok[0, 1, 2] = False
        assert torch.equal(torch.where(ok, out, 0), torch.where(ok, clean, 0))
    y[0, 2, 1, 9], y[0, 2, 1, 10] = float("nan"), float("-inf")
    am, sc = torch.ones(1, device="cuda"), torch.zeros(1, device="cuda")
    qa.norm_rope([qa.NormRopeSegment(y, v)])
    assert qa.get_error() == _lib.ERR_NONFINITE
    assert torch.equal(v.view(torch.int16), y.transpose(1, 2).contiguous().view(torch.int16))
    qa.norm_rope([qa.NormRopeSegment(y, codes, amax=am, scale=sc)])
    assert qa.get_error() == _lib.ERR_NONFINITE
    assert codes[0, 1, 2, 9].item() & 0x7F == 0x7F and codes[0, 1, 2, 10].item() == 0xFE
    codes.fill_(0x55)
    qa.norm_rope([qa.NormRopeSegment(x, codes, amax=torch.full((1,), float("inf"), device="cuda"), scale=sc)])
    assert qa.get_error() == _lib.ERR_NONFINITE
    assert bool((codes == 0x55).all()) and sc.item() == np.float32(1) / np.float32(448)   # of the call before
    run = torch.zeros(1, device="cuda")
    qa.norm_rope([qa.NormRopeSegment(y, v, amax=run)])
    assert qa.get_error() == _lib.ERR_NONFINITE and run.isnan().item()


def test_offsets_past_32_bits():
    """Heads of the input and rows of the output more than 2^31 elements apart."""
    far, D = 2 ** 31 + 64, 64
    big = torch.empty(far + 2 * D, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((1, 2, 2, D), (0, D, far - D, 1))          # [1, L, H, D]
    x.copy_(torch.randn(1, 2, 2, D, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16))
    dst = torch.empty(far + 2 * D, dtype=torch.bfloat16, device="cuda")
    out = dst.as_strided((1, 2, 2, D), (0, D, far - D, 1))        # [1, H, L, D]
    w = torch.ones(D, device="cuda")
    qa.norm_rope([qa.NormRopeSegment(x, out, weight=w)])
    assert qa.get_error() == 0
    _check(out, x.contiguous(), w, None, 1e-6, True, torch.bfloat16)


def test_twelve_tensors_another_stream_and_a_replayed_graph():
    D = 128
    g = torch.Generator().manual_seed(5)
    xs = [torch.randn(1, 3 + 11 * i, 1 + i % 3, D, generator=g).to(torch.bfloat16).cuda() for i in range(12)]
    w = torch.ones(D, device="cuda")
    new = lambda: [torch.zeros(1, x.shape[2], x.shape[1], D, dtype=torch.bfloat16, device="cuda") for x in xs]
    call = lambda outs: qa.norm_rope([qa.NormRopeSegment(x, o, weight=w if i % 2 else None) for i, (x, o) in enumerate(zip(xs, outs))])
    want, side_out, graph_out = new(), new(), new()
    call(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(side_out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(graph_out)
    for o in graph_out:
        o.zero_()
    graph.replay()
    assert qa.get_error() == 0
    for a, b, c in zip(want, side_out, graph_out):
        assert torch.equal(a, b) and torch.equal(a, c)
    for x in xs:
        x.mul_(-2.0)
    graph.replay()
    call(want)
    assert all(torch.equal(a, c) for a, c in zip(want, graph_out))
    assert qa.get_error() == 0
