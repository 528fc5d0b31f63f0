"""Cases of the operators around the quantized attention, for measuring: the multi-axis rotary table
(``rope_table``), the per-head norm with the rotation and layout change (``norm_rope``) and the linear
layer in 8-bit integers with a scale for each token and output channel (``linear_int8``).

``run`` computes a case in plain torch operations, or, with ``own`` true, through the package's calls.
"""
from __future__ import annotations

import math

import torch

own = False

# FLUX-like split of a 128-wide head over (stream, height, width), and a video split
AXES = {"16,56,56": (16, 56, 56), "44,42,42": (44, 42, 42), "32,16,16": (32, 16, 16),
        "128": (128,), "32": (32,)}
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
THETA = 10000.0
EPS = 1e-6
# static amax of Q, K (unit rows after the norm, weights near 1) and V of an earlier calibration
AMAX = (7.5, 7.5, 6.5)


def listed():
    return [
        # positions of one image's joint sequence: 512 text tokens and a 64 x 64 patch grid
        {"name": "table_image_4608", "op": "table", "tokens": 4608, "axes": "16,56,56", "float": True},
        # positions of a video: frames x 60 x 60 patches
        {"name": "table_video_118800", "op": "table", "tokens": 118800, "axes": "44,42,42", "float": False},
        # one new token of a decoder with grouped heads, rotation of halves
        {"name": "rope_one_token", "op": "rope", "B": 1, "text": 0, "image": 1, "Hq": 32, "Hkv": 8,
         "D": 128, "axes": "128", "pairs": False, "dtype": "bf16", "e4m3": False},
        # text and image streams of an image generation step, bf16 for a calibrating attention
        {"name": "rope_gen_4608", "op": "rope", "B": 1, "text": 512, "image": 4096, "Hq": 24, "Hkv": 24,
         "D": 128, "axes": "16,56,56", "pairs": True, "dtype": "bf16", "e4m3": False},
        # an editing step (target and context image), straight to the attention's E4M3 codes
        {"name": "rope_edit_8704_e4m3", "op": "rope", "B": 1, "text": 512, "image": 8192, "Hq": 24,
         "Hkv": 24, "D": 128, "axes": "16,56,56", "pairs": True, "dtype": "bf16", "e4m3": True},
        # batch with odd lengths, narrow heads, half of the head rotated, fp16
        {"name": "rope_ragged_d64_fp16", "op": "rope", "B": 3, "text": 77, "image": 4131, "Hq": 16,
         "Hkv": 4, "D": 64, "axes": "32", "pairs": False, "dtype": "fp16", "e4m3": False},
        # linear layers: one token, a few tokens, ...
        {"name": "int8_1x6144x4096", "op": "linear", "M": 1, "N": 6144, "K": 4096, "dtype": "bf16", "bias": False},
        {"name": "int8_24x4096x11008", "op": "linear", "M": 24, "N": 4096, "K": 11008, "dtype": "fp16", "bias": True},
        # ... an odd prompt with ragged widths, ...
        {"name": "int8_333x5125x5003", "op": "linear", "M": 333, "N": 5125, "K": 5003, "dtype": "bf16", "bias": True},
        # ... a text stream, ...
        {"name": "int8_512x9216x4096", "op": "linear", "M": 512, "N": 9216, "K": 4096, "dtype": "bf16", "bias": True},
        # ... and the joint sequences of a generation and an editing step
        {"name": "int8_4608x4096x12288", "op": "linear", "M": 4608, "N": 4096, "K": 12288, "dtype": "bf16", "bias": True},
        {"name": "int8_8704x12288x4096", "op": "linear", "M": 8704, "N": 12288, "K": 4096, "dtype": "bf16", "bias": True},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["table", "rope", "rope", "linear", "linear", "linear"])
    if op == "table":
        return {"op": op, "tokens": _log(rng, 1, 118800), "axes": rng.choice(["16,56,56", "44,42,42", "32,16,16", "128"]),
                "float": rng.random() < 0.5}
    if op == "rope":
        D = rng.choice([64, 128])
        axes = rng.choice(["16,56,56", "44,42,42", "128", "32"] if D == 128 else ["32,16,16", "32"])
        Hkv = rng.choice([2, 4, 8, 24])
        B = rng.choice([1, 1, 2, 3])
        return {"op": op, "B": B, "text": rng.choice([0, 0, 77, 512, rng.randint(1, 600)]),
                "image": _log(rng, 1, 8192 // B), "Hq": 24 if Hkv == 24 else Hkv * rng.choice([1, 2, 3]), "Hkv": Hkv, "D": D,
                "axes": axes, "pairs": rng.random() < 0.5, "dtype": rng.choice(["bf16", "bf16", "fp16"]),
                "e4m3": rng.random() < 0.5}
    N, K = _log(rng, 64, 16384), _log(rng, 64, 16384)
    most = 8704 * 12288 * 4096 // (N * K)
    M = min(_log(rng, 1, 8704), max(1, most))
    if rng.random() < 0.6:                       # most layers have even widths
        N, K = max(64, N // 64 * 64), max(64, K // 64 * 64)
    return {"op": op, "M": M, "N": N, "K": K, "dtype": rng.choice(["bf16", "bf16", "fp16"]),
            "bias": rng.random() < 0.5}


def _positions(tokens, axes, g):
    """Token ids as image and video models give them: (frame, row, column) counted up from a start
    that the seed sets, for one axis the token's own number."""
    t = torch.arange(tokens, device="cuda")
    start = torch.randint(0, 4096, (1,), generator=g, device="cuda")
    if axes == 1:
        return (t + start)[:, None]
    side = 60
    return torch.stack([t // (side * side) + start, t // side % side, t % side], 1)


def _angles(pos, axes):
    """[tokens, sum(axes) / 2] angles in 64 bits: position of the pair's axis times its frequency."""
    which = torch.cat([torch.full((d // 2,), a) for a, d in enumerate(axes)]).to(pos.device)
    expo = torch.cat([torch.arange(0, d, 2, dtype=torch.float64) / d for d in axes]).to(pos.device)
    return pos.double()[:, which] * torch.pow(THETA, -expo)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")
    if case["op"] == "table":
        axes = AXES[case["axes"]]
        pos = _positions(case["tokens"], len(axes), g)
        pos = pos.float() if case["float"] else pos.int()
        table = torch.empty(case["tokens"], sum(axes) // 2, 2, device="cuda")
        return {"case": case, "pos": pos, "axes": axes, "table": table}
    dt = DTYPES[case["dtype"]]
    if case["op"] == "rope":
        B, Lt, Li, Hq, Hkv, D = (case[k] for k in ("B", "text", "image", "Hq", "Hkv", "D"))
        axes = AXES[case["axes"]]
        L, width = Lt + Li, (Hq + 2 * Hkv) * D
        scale = torch.exp(0.3 * normal(width))   # channels of a projection differ in size
        a = _angles(_positions(L, len(axes), g), axes)
        table = torch.stack([a.cos(), a.sin()], -1).float()
        out = lambda H: torch.empty(B, H, L, D, dtype=torch.uint8 if case["e4m3"] else dt, device="cuda")
        return {"case": case, "text": (normal(B, Lt, width) * scale).to(dt), "image": (normal(B, Li, width) * scale).to(dt),
                "weights": 1.0 + 0.1 * normal(4, D),       # text q, text k, image q, image k
                "table": table, "amax": torch.tensor(AMAX, device="cuda"), "scale": torch.zeros(3, device="cuda"),
                "q": out(Hq), "k": out(Hkv), "v": out(Hkv)}
    M, N, K = case["M"], case["N"], case["K"]
    x = normal(M, K)
    x[:, :: max(1, K // 7)] *= 8.0               # a few outlier channels, as activations have
    w = normal(N, K) * (K ** -0.5)
    s_w = w.abs().amax(1) / 127.0
    padded = -(-K // 16) * 16                    # rows of codes start on 16 bytes
    w8 = torch.zeros(N, padded, dtype=torch.int8, device="cuda")
    w8[:, :K] = torch.round(w / s_w[:, None]).clamp(-127, 127).to(torch.int8)
    return {"case": case, "x": x.to(dt), "w8": w8[:, :K], "s_w": s_w, "bias": normal(N) if case["bias"] else None,
            "x8": torch.empty(M, padded, dtype=torch.int8, device="cuda")[:, :K], "s_x": torch.empty(M, device="cuda"),
            "y": torch.empty(M, N, dtype=dt, device="cuda")}


def _split(s, qkv):
    """Query, key and value heads [B, tokens, H, D] of a projection's output, as views."""
    c = s["case"]
    B, tokens, _ = qkv.shape
    x = qkv.view(B, tokens, c["Hq"] + 2 * c["Hkv"], c["D"])
    return x.split([c["Hq"], c["Hkv"], c["Hkv"]], 2)


def _run_own(s):
    import precision_quantized_attention_b200 as qa
    c = s["case"]
    if c["op"] == "table":
        qa.rope_table(s["pos"], s["axes"], s["table"], theta=THETA)
        return {"table": s["table"]}
    if c["op"] == "linear":
        qa.linear_int8(s["x"], s["x8"], s["s_x"], s["w8"], s["s_w"], s["y"], bias=s["bias"])
        return {"y": s["y"], "s_x": s["s_x"]}
    Lt, w, codes = c["text"], s["weights"], c["e4m3"]
    amax = s["amax"].split(1) if codes else (None, None, None)
    scale = s["scale"].split(1) if codes else (None, None, None)
    segments = []
    for x, rows, wq, wk in ((s["text"], slice(0, Lt), w[0], w[1]), (s["image"], slice(Lt, None), w[2], w[3])):
        if x.shape[1] == 0:
            continue
        q, k, v = _split(s, x)
        table = s["table"][rows]
        segments.append(qa.NormRopeSegment(q, s["q"][:, :, rows], weight=wq, table=table, amax=amax[0], scale=scale[0]))
        segments.append(qa.NormRopeSegment(k, s["k"][:, :, rows], weight=wk, table=table, amax=amax[1], scale=scale[1]))
        segments.append(qa.NormRopeSegment(v, s["v"][:, :, rows], amax=amax[2], scale=scale[2]))
    qa.norm_rope(segments, eps=EPS, interleaved=c["pairs"])
    if codes:
        e = torch.float8_e4m3fn
        return {"q": s["q"].view(e), "k": s["k"].view(e), "v": s["v"].view(e), "scale": s["scale"]}
    return {"q": s["q"], "k": s["k"], "v": s["v"]}


def _norm(x, w):
    x = x.float()
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w


def _rotate(x, table, pairs):
    """x [B, tokens, H, D] fp32, its first 2 * table.shape[1] channels rotated."""
    R = 2 * table.shape[1]
    c, s = table[:, None, :, 0], table[:, None, :, 1]
    x0, x1 = (x[..., 0:R:2], x[..., 1:R:2]) if pairs else (x[..., : R // 2], x[..., R // 2: R])
    y0, y1 = x0 * c - x1 * s, x1 * c + x0 * s
    y = torch.stack([y0, y1], -1).flatten(-2) if pairs else torch.cat([y0, y1], -1)
    return torch.cat([y, x[..., R:]], -1)


def _e4m3(y, scale):
    return (y / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def run(state):
    s = state
    if own:
        return _run_own(s)
    c = s["case"]
    if c["op"] == "table":
        a = _angles(s["pos"], s["axes"])
        return {"table": torch.stack([a.cos(), a.sin()], -1).float()}
    if c["op"] == "linear":
        x = s["x"].float()
        amax = x.abs().amax(1)
        amax = torch.where(amax == 0, 127.0, amax)
        codes = torch.round((x * 127.0).double() / amax.double()[:, None]).float()   # 64 bits: next to a border
        s_x = amax / 127.0
        y = (codes @ s["w8"].float().T) * s_x[:, None] * s["s_w"]
        y = y if s["bias"] is None else y + s["bias"]
        return {"y": y.to(s["x"].dtype), "s_x": s_x}
    (tq, tk, tv), (iq, ik, iv) = _split(s, s["text"]), _split(s, s["image"])
    w = s["weights"]
    q = _rotate(torch.cat([_norm(tq, w[0]), _norm(iq, w[2])], 1), s["table"], c["pairs"])
    k = _rotate(torch.cat([_norm(tk, w[1]), _norm(ik, w[3])], 1), s["table"], c["pairs"])
    v = torch.cat([tv, iv], 1).float()
    q, k, v = (t.transpose(1, 2).contiguous() for t in (q, k, v))
    if c["e4m3"]:
        scale = s["amax"] / 448.0
        return {"q": _e4m3(q, scale[0]), "k": _e4m3(k, scale[1]), "v": _e4m3(v, scale[2]), "scale": scale}
    dt = DTYPES[c["dtype"]]
    return {"q": q.to(dt), "k": k.to(dt), "v": v.to(dt)}


def work(case):
    if case["op"] == "table":
        axes = AXES[case["axes"]]
        return {"bytes": case["tokens"] * 4 * (len(axes) + sum(axes)), "flops": case["tokens"] * sum(axes) // 2 * 40}
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": 2 * M * K + N * K + 2 * M * N + 4 * N * (2 if case["bias"] else 1) + 4 * M, "flops": 2 * M * N * K}
    L, R = case["text"] + case["image"], sum(AXES[case["axes"]])
    n = case["B"] * L * (case["Hq"] + 2 * case["Hkv"]) * case["D"]
    return {"bytes": n * (3 if case["e4m3"] else 4) + 4 * L * R + 16 * case["D"], "flops": 10 * n}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "table":
        pos, out = s["pos"].double(), []
        for a, d in enumerate(s["axes"]):
            freq = torch.exp(torch.arange(d // 2, device="cuda", dtype=torch.float64) * (-2.0 * math.log(THETA) / d))
            turn = torch.polar(torch.ones((), device="cuda", dtype=torch.float64), torch.outer(pos[:, a], freq))
            out.append(torch.view_as_real(turn))
        return {"table": torch.cat(out, 1)}
    if case["op"] == "linear":
        x = s["x"].double()
        top = x.abs().max(1, keepdim=True).values
        top[top == 0] = 127.0
        ints = torch.round(x * 127.0 / top)
        y = torch.einsum("mk,nk->mn", ints, s["w8"].double())
        y = y * (top / 127.0) * s["s_w"].double()[None]
        return {"y": y + s["bias"].double() if s["bias"] is not None else y, "s_x": (top / 127.0)[:, 0]}
    turn = torch.view_as_complex(s["table"].double())
    half = turn.shape[1]
    w = s["weights"].double()

    def one(stream, first, heads, weight):
        x = s[stream].double().unflatten(-1, (-1, case["D"]))[:, :, first:first + heads].movedim(2, 1)
        if weight is None:
            return x
        x = x / (x.pow(2).sum(-1, keepdim=True) / case["D"] + EPS).sqrt() * weight
        rows = turn[: case["text"]] if stream == "text" else turn[case["text"]:]
        if case["pairs"]:
            z = torch.view_as_complex(x[..., : 2 * half].reshape(*x.shape[:-1], half, 2)) * rows
            z = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(x[..., :half], x[..., half: 2 * half]) * rows
            z = torch.cat([z.real, z.imag], -1)
        return torch.cat([z, x[..., 2 * half:]], -1)

    Hq, Hkv = case["Hq"], case["Hkv"]
    out = {"q": torch.cat([one("text", 0, Hq, w[0]), one("image", 0, Hq, w[2])], 2),
           "k": torch.cat([one("text", Hq, Hkv, w[1]), one("image", Hq, Hkv, w[3])], 2),
           "v": torch.cat([one("text", Hq + Hkv, Hkv, None), one("image", Hq + Hkv, Hkv, None)], 2)}
    if case["e4m3"]:
        scale = s["amax"].double() / 448.0
        for i, t in enumerate("qkv"):
            out[t] = (out[t] / scale[i]).clamp(-448.0, 448.0)
        out["scale"] = scale
    return out
