"""The attention half of a transformer block in one run: token positions to a rotary table, the QKV
projections of the text and image streams in 8-bit integers, per-head norm + rotation + FP8 quantize into the
joint sequence, quantized attention, output projection.  Every stage is held to its definition on what the
stage before it gave, and the run captured into a graph gives the same bits."""
import numpy as np
import pytest
import torch

import oracle
import precision_quantized_attention_b200 as qa
from parity import assert_close
from test_gpu_rope import check_codes

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,axes,inter", [(128, (16, 56, 56), True), (64, (32, 16, 16), False)])
def test_block_attention_half(D, axes, inter):
    H, Lt, side = 3, 37, 15
    L, C = Lt + side * side, H * D
    g = torch.Generator().manual_seed(D)
    rnd = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()
    x = {"text": rnd(Lt, C), "image": rnd(side * side, C)}
    qkv = {s: qa.Int8Linear(rnd(3 * C, C) * C ** -0.5, torch.zeros(3 * C).cuda(), max_tokens=256) for s in x}
    proj = qa.Int8Linear(rnd(C, C) * C ** -0.5, max_tokens=512)
    w = (1 + 0.1 * torch.randn(4, D, generator=g)).cuda()
    pos = torch.zeros(L, 3, dtype=torch.int32)
    pos[Lt:, 1] = torch.arange(side * side) // side
    pos[Lt:, 2] = torch.arange(side * side) % side
    table = torch.empty(L, D // 2, 2, device="cuda")
    qa.rope_table(pos.cuda(), axes, table)
    joint = lambda dt: [torch.empty(1, H, L, D, dtype=dt, device="cuda") for _ in range(3)]
    bf, codes, out = joint(torch.bfloat16), joint(torch.uint8), torch.empty(1, H, L, D, dtype=torch.bfloat16, device="cuda")
    running, scale = torch.zeros(3, device="cuda"), torch.zeros(3, device="cuda")
    amax, sc = running.split(1), scale.split(1)

    def segments(dst, proj_out, scales):
        segs = []
        for s, rows, i in (("text", slice(0, Lt), 0), ("image", slice(Lt, L), 2)):
            q, k, v = proj_out[s].view(1, -1, 3, H, D).unbind(2)
            for j, (t, weight) in enumerate(((q, w[i]), (k, w[i + 1]), (v, None))):
                segs.append(qa.NormRopeSegment(t, dst[j][:, :, rows], weight=weight, table=None if weight is None else table[rows],
                                               amax=amax[j], scale=sc[j] if scales else None))
        return segs

    def step():
        y = {s: qkv[s](x[s]) for s in x}
        qa.norm_rope(segments(codes, y, True), interleaved=inter)
        qa.forward(codes[0], codes[1], codes[2], out, *sc, D ** -0.5)
        return y, proj(out.transpose(1, 2).reshape(L, C))

    first = {s: qkv[s](x[s]) for s in x}
    qa.norm_rope(segments(bf, first, False), interleaved=inter)          # calibration: the running amax
    for j in range(3):
        assert running[j].item() == bf[j].abs().max().item()
    y, last = step()
    assert qa.get_error() == 0
    host = lambda t: t.double().cpu().numpy()
    for s in x:                                                          # projections
        xc, xs = oracle.quantize_int8_rows(host(x[s]))
        want, size = oracle.gemm_int8(xc, qkv[s].w8.cpu().numpy(), xs, host(qkv[s].s_w))
        assert (np.abs(host(y[s]) - want) <= 2.0 ** -8 * np.abs(want) + 5 * 2.0 ** -24 * size).all()
    for j in range(3):                                                   # the calibrated tensors and their codes
        want, s = oracle.quantize_fp8(bf[j].cpu(), float(running[j].item()))
        assert np.float32(scale[j].item()) == s
        assert j < 2 or np.array_equal(codes[j].cpu().numpy().reshape(-1), want)
        for i, rows in ((0, slice(0, Lt)), (2, slice(Lt, L))):
            src = y["text" if i == 0 else "image"].view(1, -1, 3, H, D)[:, :, j]
            val, size = oracle.norm_rope(host(src), None if j == 2 else host(w[i + j]), None if j == 2 else host(table[rows]), 1e-6, inter)
            assert (np.abs(host(bf[j][:, :, rows]) - val) <= 2.0 ** -8 * np.abs(val) + 25 * 2.0 ** -24 * size).all()
            if j < 2:
                check_codes(codes[j][:, :, rows], float(s), src, w[i + j], table[rows], 1e-6, inter)
    n = [c.cpu().numpy() for c in codes]
    want, amb = oracle.attention_e4m3(*n, (1, H, L, D), *[float(s.item()) for s in sc], with_ambiguity=True)
    assert_close(out.float().cpu().numpy(), want, "attention", amb)
    oc, os_ = oracle.quantize_int8_rows(host(out.transpose(1, 2).reshape(L, C)))
    want, size = oracle.gemm_int8(oc, proj.w8.cpu().numpy(), os_, host(proj.s_w))
    assert (np.abs(host(last) - want) <= 2.0 ** -8 * np.abs(want) + 5 * 2.0 ** -24 * size).all()

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, replayed = step()
    out.zero_()
    graph.replay()
    assert qa.get_error() == 0
    assert torch.equal(replayed, last)
