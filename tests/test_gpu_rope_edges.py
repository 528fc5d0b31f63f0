"""Edges of rope_table and norm_rope: small sines, rows and groups without data, infinities next to
channels that are not rotated, values near the type's largest, amax values that are no maximum.

Bars (u = 2^-24).  A sine or cosine: the rest of the angle after whole quarter turns is rounded twice (2 u of
itself) and resolved to 2^-53 quarter turns; its square, the sum's last steps, the first coefficient and the
product add less than 4 u: 6 u of the value.  The angle: the frequency is held to 2^-65 turns and, as a power
formed by up to 128 products in 64 bits, to 2^-56 of itself, the oracle's FP64 angle to 2^-51: together less than
|a| 2^-50 + (|pos| + 6) 2^-62.  norm_rope: the bars of test_gpu_rope."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle
import precision_quantized_attention_b200 as qa
from precision_quantized_attention_b200 import _lib
from test_gpu_rope import _check as check_norm_rope, check_codes

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U = 2.0 ** -24
# whole numbers near multiples of pi: sines down to 1e-7
NEAR_PI = [3, 22, 333, 355, 710, 103993, 104348, 208341, 312689, 833719, 1146408]


@pytest.mark.parametrize("kind", ["int", "whole", "fraction", "small"])
@pytest.mark.parametrize("dims,theta", [((128,), 1e4), ((128,), 1e6), ((16, 56, 56), 1e4), ((2,), 10.0), ((256,), 1e10)])
def test_small_sines_keep_their_relative_accuracy(dims, theta, kind):
    n = len(dims)
    if kind in ("int", "whole"):
        p = np.array([s * v for v in list(range(100)) + NEAR_PI for s in (1, -1)], dtype=np.int64)
        pos = torch.from_numpy(p).to(torch.int32 if kind == "int" else torch.float32)
    elif kind == "fraction":                         # close to quarter turns, and anywhere
        p = [s * k * math.pi / 2 for k in range(1, 200) for s in (1, -1)]
        pos = torch.cat([torch.tensor(p), torch.randn(500, generator=torch.Generator().manual_seed(1)) * 30])
    else:
        pos = torch.randn(500, generator=torch.Generator().manual_seed(2)) * torch.logspace(-9, 0, 500)
    pos = pos[:, None].expand(-1, n).contiguous()
    table = torch.full((pos.shape[0], sum(dims) // 2, 2), 7.0, device="cuda")
    qa.rope_table(pos.cuda(), dims, table, theta=theta)
    assert qa.get_error() == 0
    got = table.double().cpu().numpy()
    a = oracle.rope_angles(pos.numpy(), dims, (theta,) * n)
    size = np.abs(pos.double().numpy())[:, :1]
    for i, want in ((0, np.cos(a)), (1, np.sin(a))):
        tol = 6 * U * np.abs(want) + 2.0 ** -52 + np.abs(a) * 2.0 ** -50 + (size + 6) * 2.0 ** -62
        off = np.abs(got[..., i] - want)
        assert (off <= tol).all(), f"worst {np.max(off / tol):.2f} of the bar"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("inter", [True, False])
@pytest.mark.parametrize("B,L,H,D,R", [(1, 5, 3, 128, 128), (1, 1, 1, 64, 0), (2, 3, 5, 8, 0), (1, 7, 9, 24, 16),
                                       (1, 2, 33, 256, 128), (1, 301, 2, 64, 64)])
def test_running_amax_behind_a_norm_without_eps(B, L, H, D, R, inter, dtype):
    """Lanes of a warp that hold no token, head or channel add nothing to the maximum, with eps = 0 too."""
    g = torch.Generator().manual_seed(L * H + D)
    x = (1 + torch.randn(B, L, H, D, generator=g).abs()).to(dtype).cuda()
    w = (1 + 0.2 * torch.randn(D, generator=g)).cuda()
    table = None
    if R:
        a = torch.rand(L, R // 2, generator=g) * 9
        table = torch.stack([a.cos(), a.sin()], -1).cuda()
    for eps in (0.0, 1e-6):
        amax = torch.zeros(1, device="cuda")
        out = torch.empty(B, H, L, D, dtype=dtype, device="cuda")
        qa.norm_rope([qa.NormRopeSegment(x, out, weight=w, table=table, amax=amax)], eps=eps, interleaved=inter)
        assert qa.get_error() == 0
        assert amax.item() == out.abs().max().item()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("D,R,inter", [(64, 32, True), (64, 32, False), (64, 48, False), (96, 64, True), (128, 0, True),
                                       (128, 0, False), (184, 48, False), (256, 240, False)])
def test_an_infinity_in_a_channel_that_is_not_rotated_stays_there(D, R, inter, weighted, dtype):
    L, H = 6, 3
    g = torch.Generator().manual_seed(D + R)
    x = torch.randn(1, L, H, D, generator=g).to(dtype)
    x[0, 1, 0, R + 2] = float("inf")
    x[0, 2, 1, D - 1] = float("-inf")
    x[0, 4, 2, R] = float("inf")
    x[0, 4, 2, R + 1] = float("-inf")
    if R:
        x[0, 5, 0, 3] = float("inf")                 # a rotated one: its pair, and no other channel
    w = (1 + 0.1 * torch.randn(D, generator=g)).cuda() if weighted else None
    table = None
    if R:
        a = 0.3 + torch.rand(L, R // 2, generator=g)
        table = torch.stack([a.cos(), a.sin()], -1).cuda()
    elif not weighted:
        return                                       # a copy
    out = torch.empty(1, H, L, D, dtype=dtype, device="cuda")
    codes = torch.empty(1, H, L, D, dtype=torch.uint8, device="cuda")
    amax, scale = torch.full((1,), 3.0, device="cuda"), torch.zeros(1, device="cuda")
    qa.norm_rope([qa.NormRopeSegment(x.cuda(), out, weight=w, table=table)], eps=1e-6, interleaved=inter)
    assert qa.get_error() == _lib.ERR_NONFINITE
    qa.norm_rope([qa.NormRopeSegment(x.cuda(), codes, weight=w, table=table, amax=amax, scale=scale)], eps=1e-6,
                 interleaved=inter)
    assert qa.get_error() == _lib.ERR_NONFINITE
    host = lambda t: None if t is None else t.double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        want, size = oracle.norm_rope(host(x), host(w), host(table), 1e-6, inter)
    got, got8 = host(out), codes.cpu().view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isnan(got8), np.isnan(want))
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]) and np.array_equal(got8[inf], np.sign(want[inf]) * 448)
    ok = np.isfinite(want)
    half = torch.finfo(dtype).eps / 2
    tol = 24 * U * size[ok] + half * (np.abs(want[ok]) + 24 * U * size[ok]) + 2.0 ** -25
    assert (np.abs(got[ok] - want[ok]) <= tol).all()
    s = float(scale.item())
    value = lambda v: torch.from_numpy(np.clip(v / s, -448.0, 448.0)).float().to(torch.float8_e4m3fn).float().numpy()
    assert (value(want[ok] - 28 * U * size[ok]) <= got8[ok]).all() and (got8[ok] <= value(want[ok] + 28 * U * size[ok])).all()


@pytest.mark.parametrize("inter", [True, False])
@pytest.mark.parametrize("amax", [1e-5, 3.0, 1e30])
def test_codes_of_a_rotation_of_values_near_the_largest(amax, inter):
    """Products with 1 / scale would pass FP32's range and cancel to NaN; the rotated values do not."""
    D, L, H = 64, 9, 2
    g = torch.Generator().manual_seed(1)
    x = (torch.rand(1, L, H, D, generator=g) * 1e38 + 2e38).to(torch.bfloat16).cuda()
    a = math.pi / 4 + 0.01 * torch.randn(L, D // 2, generator=g)
    table = torch.stack([a.cos(), a.sin()], -1).cuda()
    codes = torch.empty(1, H, L, D, dtype=torch.uint8, device="cuda")
    scale = torch.zeros(1, device="cuda")
    qa.norm_rope([qa.NormRopeSegment(x, codes, table=table, amax=torch.full((1,), amax, device="cuda"), scale=scale)],
                 interleaved=inter)
    assert qa.get_error() == 0
    check_codes(codes, float(scale.item()), x, None, table, 1e-6, inter)


def test_a_given_amax_of_minus_infinity_writes_no_code():
    x = torch.ones(1, 5, 2, 64, dtype=torch.bfloat16, device="cuda")
    for bad in (float("-inf"), float("inf"), float("nan")):
        for w in (None, torch.ones(64, device="cuda")):
            amax, scale = torch.full((1,), bad, device="cuda"), torch.full((1,), 5.0, device="cuda")
            codes = torch.full((1, 2, 5, 64), 0x55, dtype=torch.uint8, device="cuda")
            qa.norm_rope([qa.NormRopeSegment(x, codes, weight=w, amax=amax, scale=scale)])
            assert qa.get_error() == _lib.ERR_NONFINITE
            assert bool((codes == 0x55).all()) and scale.item() == 5.0
        new = lambda n, v=0x55: torch.full((n,), v, dtype=torch.uint8, device="cuda")
        codes, e2m1, block = new(640), new(320), new(40)
        scale, scales = torch.full((1,), 5.0, device="cuda"), torch.full((3,), 5.0, device="cuda")
        qa.quantize_fp8(x.view(-1), amax, codes, scale)
        assert qa.get_error() == _lib.ERR_NONFINITE
        qa.quantize_fp4_block(x.view(-1), amax, e2m1, block, scale)
        assert qa.get_error() == _lib.ERR_NONFINITE
        qa.quantize_qkv([x.view(-1)] * 3, amax.expand(3).contiguous(), [codes] * 3, scales)
        assert qa.get_error() == _lib.ERR_NONFINITE
        a8 = new(128 * 128, 0x30).view(128, 128)
        one, product = torch.ones(1, device="cuda"), new(128 * 32).view(128, 32)
        qa.gemm_fp8_e4m3(a8, a8[:32], product, one, one, amax, scale)
        assert qa.get_error() == _lib.ERR_NONFINITE
        for t in (codes, e2m1, block, product):
            assert bool((t == 0x55).all())
        assert scale.item() == 5.0 and bool((scales == 5.0).all())


@pytest.mark.parametrize("start", [float("-inf"), -1.0, -0.0, 0.5, 1e30])
def test_running_amax_continues_from_any_number(start):
    x = torch.randn(1, 7, 3, 64, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).cuda()
    for w in (None, torch.ones(64, device="cuda")):
        out = torch.empty(1, 3, 7, 64, dtype=torch.bfloat16, device="cuda")
        amax = torch.full((1,), start, device="cuda")
        qa.norm_rope([qa.NormRopeSegment(x, out, weight=w, amax=amax)])
        assert qa.get_error() == 0
        assert amax.item() == max(np.float32(start), out.abs().max().item())


@pytest.mark.parametrize("inter", [True, False])
@pytest.mark.parametrize("D", [16, 64, 96, 128, 256])
def test_a_whole_rotation_next_to_a_norm_without_one(D, inter):
    """All channels of one tensor rotated, none of another, in one call; each as in a call of its own."""
    B, L, H = 2, 19, 5
    g = torch.Generator().manual_seed(D)
    x = torch.randn(B, L, H, D, generator=g).to(torch.bfloat16).cuda()
    w = (1 + 0.2 * torch.randn(D, generator=g)).cuda()
    a = torch.rand(L, D // 2, generator=g) * 9
    table = torch.stack([a.cos(), a.sin()], -1).cuda()
    forms = [dict(weight=w, table=table), dict(weight=w), dict(table=table), {}]
    new = lambda: torch.empty(B, H, L, D, dtype=torch.bfloat16, device="cuda")
    outs = [new() for _ in forms]
    qa.norm_rope([qa.NormRopeSegment(x, o, **f) for o, f in zip(outs, forms)], interleaved=inter)
    assert qa.get_error() == 0
    for o, f in zip(outs, forms):
        check_norm_rope(o, x, f.get("weight"), f.get("table"), 1e-6, inter, torch.bfloat16)
    whole = [new(), new()]
    qa.norm_rope([qa.NormRopeSegment(x, o, **f) for o, f in zip(whole, (forms[0], forms[2]))], interleaved=inter)
    assert torch.equal(whole[0], outs[0]) and torch.equal(whole[1], outs[2])
    x[1, 3, 2, D // 2] = float("inf")
    qa.norm_rope([qa.NormRopeSegment(x, o, **f) for o, f in zip(outs, forms)], interleaved=inter)
    assert qa.get_error() == _lib.ERR_NONFINITE
    row = outs[1][1, 2, 3]
    assert row[D // 2].isnan().item() and int(row.count_nonzero()) == 1      # the others times 1 / infinity


@pytest.mark.skipif(_lib.CHECKED, reason="starts the checked-build run")
def test_edges_pass_in_the_checked_build():
    from precision_quantized_attention_b200 import build
    build.build(checked=True)
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", "tests/test_gpu_rope_edges.py",
           "tests/test_int8_linear_streams.py", "tests/test_int8_linear_buffers.py"]
    r = subprocess.run(cmd, cwd=ROOT, env=dict(os.environ, QATTN_DEBUG="1"), capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
