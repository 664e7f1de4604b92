"""Workloads of the attention operators beside the chunk's own self-attention: cross attention to
an encoder's states (forward and backward) and the latent ring held in 4 bits (append, read back,
and the chunk's attention over it).

Each case is run either in its plain form (elementary torch operations in 32 bits, rounded once at
the end) or, with ``own`` set, through the library's entry points.  ``exact`` gives the same
outputs from the operators' definitions in 64 bits.
"""
import math

import torch

own = False

LAYER = {"H": 12, "Hkv": 12, "d": 128, "dtype": "bf16"}          # the Wan-shaped layer's heads
GROUPED = {"H": 16, "Hkv": 4, "d": 64, "dtype": "bf16"}          # narrow heads, shared keys
TOY = {"H": 2, "Hkv": 2, "d": 16, "dtype": "fp32"}               # the fp32 test configuration
RING = {"d_c": 192, "d_rope": 32, "frame_h": 30, "frame_w": 52}  # the Wan-shaped layer's frames
BASE = 10000.0
D_CQ = 512
GROUP = 16            # values that share one scale in the 4-bit ring
SCALE_BIAS = 107 * 8  # a scale's byte plus this, shifted left by 20, is its float32 pattern


def listed():
    return [
        # one query token against a text encoder's 512 states: where latency counts
        {"name": "cross_fwd_token", "op": "cross_fwd", **LAYER, "B": 1, "n_q": 1, "n_kv": 512},
        # a chunk of three latent frames against 512 states: one layer of one denoising step
        {"name": "cross_fwd_chunk", "op": "cross_fwd", **LAYER, "B": 1, "n_q": 4680, "n_kv": 512},
        # eight samples served together, prompts of different lengths
        {"name": "cross_fwd_batch8", "op": "cross_fwd", **LAYER, "B": 8, "n_q": 4680, "n_kv": 512},
        # narrow heads that share keys, odd sizes, ragged prompts of two encoders' states joined
        {"name": "cross_fwd_grouped", "op": "cross_fwd", **GROUPED, "B": 2, "n_q": 1333,
         "n_kv": 1501},
        # the fp32 test configuration: a frame of 16 tokens against a short prompt
        {"name": "cross_fwd_toy_fp32", "op": "cross_fwd", **TOY, "B": 1, "n_q": 16, "n_kv": 24},
        # training: the gradients of one chunk's call
        {"name": "cross_bwd_chunk", "op": "cross_bwd", **LAYER, "B": 1, "n_q": 4680, "n_kv": 512},
        # training: a batch of four chunks with prompts of different lengths
        {"name": "cross_bwd_batch4", "op": "cross_bwd", **LAYER, "B": 4, "n_q": 4680, "n_kv": 512},
        # training with shared keys: their gradients sum over the heads; odd sizes
        {"name": "cross_bwd_grouped", "op": "cross_bwd", **GROUPED, "B": 2, "n_q": 1333,
         "n_kv": 333},
        # a chunk's latents into the 4-bit ring, and the ring's values read back
        {"name": "q4_append_chunk", "op": "q4_append", **RING, "B": 1, "C": 3, "W": 6, "first": 6},
        # the same for eight samples with a longer window whose slots have wrapped
        {"name": "q4_append_batch8", "op": "q4_append", **RING, "B": 8, "C": 3, "W": 9,
         "first": 12},
        # a chunk's attention over a full window of six frames held in 4 bits
        {"name": "q4_attn_chunk", "op": "q4_attn", **RING, "B": 1, "C": 3, "W": 6, "first": 6,
         "from_cq": False},
        # two samples of small frames, a long window, query heads formed in the attention
        {"name": "q4_attn_small_frames", "op": "q4_attn", "d_c": 192, "d_rope": 32, "frame_h": 12,
         "frame_w": 21, "B": 2, "C": 3, "W": 21, "first": 60, "from_cq": True},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["cross_fwd", "cross_fwd", "cross_bwd", "cross_bwd", "q4_append", "q4_attn"])
    if op.startswith("cross"):
        shape = rng.choice([LAYER, LAYER, GROUPED, GROUPED, TOY])
        if shape is TOY:
            return {"op": op, **TOY, "B": rng.randint(1, 3), "n_q": _log_uniform(rng, 1, 64),
                    "n_kv": _log_uniform(rng, 1, 64)}
        most = 8 * 4680 if op == "cross_fwd" else 4 * 4680
        B = rng.randint(1, 4)
        return {"op": op, **shape, "B": B, "n_q": _log_uniform(rng, 1, most // (4 * B)),
                "n_kv": _log_uniform(rng, 1, 1600)}
    C = rng.randint(1, 3)
    W = rng.randint(C, 12)
    d_c, d_rope = rng.choice([(192, 32), (192, 32), (128, 32), (256, 64)])
    case = {"op": op, "d_c": d_c, "d_rope": d_rope, "frame_h": rng.randint(8, 16),
            "frame_w": rng.randint(8, 32), "B": rng.randint(1, 2), "C": C, "W": W,
            "first": C * rng.randint(0, 60)}
    if op == "q4_attn":
        case["from_cq"] = d_c <= 192 and rng.random() < 0.5
    return case


# ------------------------------------------------------------------------------------- inputs


def _dtype(case):
    return torch.float32 if case.get("dtype") == "fp32" else torch.bfloat16


def _normal(g, shape, dtype, std=1.0):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    return (x * std).to(dtype) if std != 1.0 else x.to(dtype)


def _ring_sizes(case):
    tpf = case["frame_h"] * case["frame_w"]
    return tpf, case["C"] * tpf, case["d_c"] + case["d_rope"], min(case["first"], case["W"])


def _rope_pairs(d_rope):
    n = d_rope // 2
    pt = n // 4
    ph = (n - pt) // 2
    return pt, ph, n - pt - ph


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    B = case["B"]
    if case["op"].startswith("cross"):
        H, Hkv, d, n_q, n_kv, dt = (case["H"], case["Hkv"], case["d"], case["n_q"], case["n_kv"],
                                    _dtype(case))
        s["scale"] = 1.0 / math.sqrt(d)
        # queries and keys of unit size, as a norm on both leaves them; the values likewise
        s["q"] = _normal(g, (B, n_q, H, d), dt)
        s["k"] = _normal(g, (B, n_kv, Hkv, d), dt)
        s["v"] = _normal(g, (B, n_kv, Hkv, d), dt)
        # valid states per sample: the first prompt fills the buffer, the others are shorter
        low = (n_kv + 3) // 4
        lens = torch.randint(low, n_kv + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        lens[0] = n_kv
        s["kv_len"] = lens
        s["out"] = torch.empty((B, n_q, H, d), device="cuda", dtype=dt)
        s["lse"] = torch.empty((B, H, n_q), device="cuda", dtype=torch.float32)
        if case["op"] == "cross_bwd":
            # what the forward call left for the backward
            out, lse = _cross_fwd(s)
            s["out"], s["lse"] = out, lse
            s["d_out"] = _normal(g, (B, n_q, H, d), dt)
            s["d_q"], s["d_k"], s["d_v"] = (torch.empty_like(s[n]) for n in "qkv")
        return s
    tpf, n_q, D, n_valid = _ring_sizes(case)
    W = case["W"]
    # the ring as earlier appends left it: every frame quantised, frame f in slot f mod W
    ring = _normal(g, (B, W * tpf, D), torch.bfloat16)
    s["codes"], s["scales"] = _q4_encode(ring)
    slot = torch.full((B, W), -1, dtype=torch.int32)
    for f in range(max(0, case["first"] - W), case["first"]):
        slot[:, f % W] = f
    s["slot_frame"] = slot.cuda()
    s["chunk"] = _normal(g, (B, n_q, D), torch.bfloat16)
    if case["op"] == "q4_append":
        s["values"] = torch.empty((B, W * tpf, D), device="cuda", dtype=torch.bfloat16)
        return s
    H, d_head = 12, 128
    s["scale"] = 1.0 / math.sqrt(d_head + case["d_rope"])
    if case["from_cq"]:
        s["c_q"] = _normal(g, (B, n_q, D_CQ), torch.bfloat16)
        s["w_qcat"] = _normal(g, (H, D, D_CQ), torch.bfloat16, 1.0 / math.sqrt(D_CQ))
    else:
        s["q"] = _normal(g, (B, n_q, H, D), torch.bfloat16)
    s["w_uv"] = _normal(g, (H, d_head, case["d_c"]), torch.bfloat16, 1.0 / math.sqrt(case["d_c"]))
    s["out"] = torch.empty((B, n_q, H * d_head), device="cuda", dtype=torch.bfloat16)
    s["lse"] = torch.empty((B, H, n_q), device="cuda", dtype=torch.float32)
    return s


# -------------------------------------------------------------------------------- plain forms


def _scores(s):
    """Scaled, masked scores [B, H, n_q, n_kv] in 32 bits; the keys and values per query head."""
    case = s["case"]
    rep = case["H"] // case["Hkv"]
    q = s["q"].float().transpose(1, 2)
    k = s["k"].float().transpose(1, 2).repeat_interleave(rep, dim=1)
    v = s["v"].float().transpose(1, 2).repeat_interleave(rep, dim=1)
    x = (q @ k.transpose(2, 3)) * s["scale"]
    col = torch.arange(case["n_kv"], device="cuda")
    x.masked_fill_(col[None, None, None, :] >= s["kv_len"][:, None, None, None], -math.inf)
    return q, k, v, x


def _softmax(x):
    """Probabilities and log-sum-exp of rows in 32 bits; a row of only -inf gives zeros."""
    m = x.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    e = torch.exp(x - m)
    t = e.sum(-1, keepdim=True)
    return e / torch.where(t > 0, t, torch.ones_like(t)), (m + torch.log(t)).squeeze(-1)


def _cross_fwd(s):
    _, _, v, x = _scores(s)
    p, lse = _softmax(x)
    return (p @ v).transpose(1, 2).to(s["q"].dtype).contiguous(), lse


def _cross_bwd(s):
    case = s["case"]
    q, k, v, x = _scores(s)
    p, _ = _softmax(x)
    g = s["d_out"].float().transpose(1, 2)
    dp = g @ v.transpose(2, 3)
    ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * s["scale"]
    d_q = ds @ k
    d_k, d_v = ds.transpose(2, 3) @ q, p.transpose(2, 3) @ g
    shared = (case["B"], case["Hkv"], case["H"] // case["Hkv"], case["n_kv"], case["d"])
    dt = s["q"].dtype
    return (d_q.transpose(1, 2).to(dt).contiguous(),
            d_k.reshape(shared).sum(2).transpose(1, 2).to(dt).contiguous(),
            d_v.reshape(shared).sum(2).transpose(1, 2).to(dt).contiguous())


def _q4_encode(x):
    """4-bit codes (two to a byte, the even column low, offset by 8) and one scale byte for every
    16 values: 5 exponent and 3 mantissa bits, the smallest such scale >= max|x| / 7."""
    g = x.float().unflatten(-1, (-1, GROUP))
    # the quotient in 64 bits: one that is a scale itself must not come out a hair above it
    r = (g.abs().amax(-1).double() / 7.0).float().view(torch.int32)
    byte = (((r + 0xFFFFF) >> 20) - SCALE_BIAS).clamp(0, 255)
    scale = ((byte + SCALE_BIAS) << 20).view(torch.float32)
    code = torch.round(g / scale[..., None]).clamp(-7, 7).to(torch.int32).flatten(-2) + 8
    return (code[..., 0::2] | (code[..., 1::2] << 4)).to(torch.uint8), byte.to(torch.uint8)


def _q4_decode(codes, scales):
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).to(torch.int32) - 8
    scale = ((scales.to(torch.int32) + SCALE_BIAS) << 20).view(torch.float32)
    return (c.unflatten(-1, (-1, GROUP)).float() * scale[..., None]).flatten(-2)


def _q4_append(s):
    case = s["case"]
    tpf, _, D, _ = _ring_sizes(case)
    B, C, W = case["B"], case["C"], case["W"]
    codes, scales = _q4_encode(s["chunk"])
    frames = case["first"] + torch.arange(C, device="cuda")
    slots = frames % W
    s["codes"].view(B, W, tpf, D // 2)[:, slots] = codes.view(B, C, tpf, D // 2)
    s["scales"].view(B, W, tpf, D // GROUP)[:, slots] = scales.view(B, C, tpf, D // GROUP)
    s["slot_frame"][:, slots] = frames.to(torch.int32)
    return _q4_decode(s["codes"], s["scales"]).to(torch.bfloat16), s["slot_frame"]


def _angles(case, frames):
    """Rotation angles [..., tokens, d_rope / 2] of whole frames, in 64 bits."""
    h = torch.arange(case["frame_h"], device="cuda").repeat_interleave(case["frame_w"])
    w = torch.arange(case["frame_w"], device="cuda").repeat(case["frame_h"])
    tpf = h.numel()
    t = frames.to(torch.float64)[..., None].expand(*frames.shape, tpf)
    h, w = (a.to(torch.float64).expand_as(t) for a in (h, w))
    bands = []
    for pos, n in zip((t, h, w), _rope_pairs(case["d_rope"])):
        freq = BASE ** (-torch.arange(n, device="cuda", dtype=torch.float64) / n)
        bands.append(pos[..., None] * freq)
    return torch.cat(bands, -1).flatten(-3, -2)


def _rotate(x, angle):
    sin, cos = torch.sin(angle).to(x.dtype), torch.cos(angle).to(x.dtype)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)


def _q4_attn(s):
    case = s["case"]
    tpf, n_q, _, n_valid = _ring_sizes(case)
    d_c, B, C = case["d_c"], case["B"], case["C"]
    here = _angles(case, (case["first"] + torch.arange(C, device="cuda"))[None])
    there = _angles(case, s["slot_frame"][:, :n_valid])
    ring = _q4_decode(s["codes"], s["scales"])[:, :n_valid * tpf]
    chunk = s["chunk"].float()
    value = torch.cat((ring[..., :d_c], chunk[..., :d_c]), 1)
    key = torch.cat((value, torch.cat((_rotate(ring[..., d_c:], there),
                                       _rotate(chunk[..., d_c:], here)), 1)), -1)
    if case["from_cq"]:
        q = s["c_q"].float()[:, None] @ s["w_qcat"].float().transpose(1, 2)
        q = torch.cat((q[..., :d_c], _rotate(q[..., d_c:], here[:, None])), -1)
    else:
        q = s["q"].float().transpose(1, 2)
    p, lse = _softmax((q @ key[:, None].transpose(2, 3)) * s["scale"])
    o = (p @ value[:, None]) @ s["w_uv"].float().transpose(1, 2)
    return o.transpose(1, 2).flatten(2).to(torch.bfloat16), lse


# -------------------------------------------------------------------------------- the library


def _handle(s):
    """The configuration and the workspace that a program keeps beside its buffers."""
    if "cfg" not in s:
        from mla_latent_kv_attn_b200 import api
        case = s["case"]
        if case["op"].startswith("cross"):
            s["cfg"] = api.make_cross_config(
                batch=case["B"], n_heads=case["H"], n_kv_heads=case["Hkv"], d_head=case["d"],
                n_q=case["n_q"], n_kv=case["n_kv"], softmax_scale=s["scale"], dtype=case["dtype"])
            need = api.mla_cross_attention_bwd_workspace_bytes(s["cfg"]) \
                if case["op"] == "cross_bwd" else 0
        else:
            from mla_latent_kv_attn_b200 import inputs
            s["cfg"] = api.make_config(inputs.MLAConfig(
                name="ring", dtype="bf16", d_model=1536, n_heads=12, d_head=128,
                d_c=case["d_c"], d_rope=case["d_rope"], d_cq=D_CQ,
                rope_pairs=_rope_pairs(case["d_rope"]), rope_base=BASE, frame_h=case["frame_h"],
                frame_w=case["frame_w"], chunk_frames=case["C"], window_frames=case["W"],
                batch=case["B"], n_chunks=1, measured_chunk=0))
            need = api.mla_attention_q4_workspace_bytes(s["cfg"], _ring_sizes(case)[3])
        s["workspace"] = torch.empty(max(need, 256), device="cuda", dtype=torch.uint8)
        s["dev_status"] = torch.zeros(1, device="cuda", dtype=torch.int32)
        s["api"] = api
    return s["api"], s["cfg"]


def _own(s):
    api, cfg = _handle(s)
    case = s["case"]
    if case["op"] == "cross_fwd":
        api.mla_cross_attention_fwd(cfg, s["q"], s["k"], s["v"], s["out"], lse=s["lse"],
                                    kv_len=s["kv_len"], dev_status=s["dev_status"])
        return s["out"], s["lse"]
    if case["op"] == "cross_bwd":
        api.mla_cross_attention_bwd(cfg, s["q"], s["k"], s["v"], s["out"], s["lse"], s["d_out"],
                                    s["d_q"], s["d_k"], s["d_v"], s["workspace"],
                                    kv_len=s["kv_len"], dev_status=s["dev_status"])
        return s["d_q"], s["d_k"], s["d_v"]
    if case["op"] == "q4_append":
        api.mla_cache_append_q4(cfg, s["chunk"], s["codes"], s["scales"], s["slot_frame"],
                                case["first"])
        api.mla_cache_read_q4(cfg, s["codes"], s["scales"], s["values"])
        return s["values"], s["slot_frame"]
    n_valid = _ring_sizes(case)[3]
    if case["from_cq"]:
        api.mla_attention_fwd_from_cq_q4(cfg, s["c_q"], s["w_qcat"], s["chunk"], s["codes"],
                                         s["scales"], s["slot_frame"], n_valid, case["first"],
                                         s["w_uv"], s["out"], s["lse"], s["workspace"],
                                         s["dev_status"])
    else:
        api.mla_attention_fwd_q4(cfg, s["q"], s["chunk"], s["codes"], s["scales"],
                                 s["slot_frame"], n_valid, case["first"], s["w_uv"], s["out"],
                                 s["lse"], s["workspace"], s["dev_status"])
    return s["out"], s["lse"]


def run(state):
    if own:
        return _own(state)
    return {"cross_fwd": _cross_fwd, "cross_bwd": _cross_bwd, "q4_append": _q4_append,
            "q4_attn": _q4_attn}[state["case"]["op"]](state)


def work(case):
    """Bytes of each input and output once, and the multiplications and additions of the
    definition (two products forward, five backward)."""
    B = case["B"]
    if case["op"].startswith("cross"):
        e = 4 if case["dtype"] == "fp32" else 2
        q = B * case["n_q"] * case["H"] * case["d"] * e
        kv = B * case["n_kv"] * case["Hkv"] * case["d"] * e
        stats = B * case["H"] * case["n_q"] * 4
        pairs = 2.0 * B * case["H"] * case["n_q"] * case["n_kv"] * case["d"]
        if case["op"] == "cross_fwd":
            return {"bytes": 2 * q + 2 * kv + stats, "flops": 2 * pairs}
        return {"bytes": 4 * q + 4 * kv + stats, "flops": 5 * pairs}
    tpf, n_q, D, n_valid = _ring_sizes(case)
    q4 = D // 2 + D // GROUP
    if case["op"] == "q4_append":
        return {"bytes": B * (n_q * (2 * D + q4) + case["W"] * tpf * (q4 + 2 * D)), "flops": 0}
    H, d_head, keys = 12, 128, n_valid * tpf + n_q
    flops = 2.0 * B * H * n_q * (keys * (D + case["d_c"]) + case["d_c"] * d_head)
    read = B * (n_valid * tpf * q4 + n_q * 2 * D) + 2 * H * d_head * case["d_c"]
    if case["from_cq"]:
        flops += 2.0 * B * H * n_q * D * D_CQ
        read += 2 * (B * n_q * D_CQ + H * D * D_CQ)
    else:
        read += 2 * B * n_q * H * D
    return {"bytes": read + B * n_q * H * (2 * d_head + 4), "flops": flops}


# ------------------------------------------------------------------- definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"cross_fwd": _exact_cross, "cross_bwd": _exact_cross, "q4_append": _exact_append,
            "q4_attn": _exact_attn}[case["op"]](s)


def _exact_cross(s):
    """Sample by sample and head by head, over the sample's valid states alone."""
    case = s["case"]
    fwd = case["op"] == "cross_fwd"
    f64 = lambda t: t.to(torch.float64)  # noqa: E731
    out = torch.zeros(s["q"].shape, device="cuda", dtype=torch.float64)
    lse = torch.full(s["lse"].shape, -math.inf, device="cuda", dtype=torch.float64)
    d_k, d_v = (torch.zeros(s[n].shape, device="cuda", dtype=torch.float64) for n in "kv")
    for b, n in enumerate(s["kv_len"].tolist()):
        for h in range(case["H"]):
            kh = h * case["Hkv"] // case["H"]
            q, k, v = f64(s["q"][b, :, h]), f64(s["k"][b, :n, kh]), f64(s["v"][b, :n, kh])
            x = torch.einsum("id,jd->ij", q, k) * s["scale"]
            lse[b, h] = torch.logsumexp(x, 1)
            p = torch.exp(x - lse[b, h][:, None])
            if fwd:
                out[b, :, h] = torch.einsum("ij,jd->id", p, v)
                continue
            g = f64(s["d_out"][b, :, h])
            dp = torch.einsum("id,jd->ij", g, v)
            ds = p * (dp - torch.einsum("ij,ij->i", p, dp)[:, None]) * s["scale"]
            out[b, :, h] = torch.einsum("ij,jd->id", ds, k)
            d_k[b, :n, kh] += torch.einsum("ij,id->jd", ds, q)
            d_v[b, :n, kh] += torch.einsum("ij,id->jd", p, g)
    return (out, lse) if fwd else (out, d_k, d_v)


def _exact_values(codes, scales):
    byte = scales.to(torch.float64)
    exponent = torch.floor(byte / 8)
    scale = torch.exp2(exponent - 20) * (1 + (byte - 8 * exponent) / 8)
    low = torch.remainder(codes.to(torch.float64), 16)
    high = (codes.to(torch.float64) - low) / 16
    flat = torch.stack((low, high), -1).flatten(-2) - 8
    return flat * scale.repeat_interleave(GROUP, dim=-1)


def _exact_append(s):
    case = s["case"]
    tpf, _, D, _ = _ring_sizes(case)
    B, W = case["B"], case["W"]
    x = s["chunk"].to(torch.float64).reshape(B, -1, D // GROUP, GROUP)
    least = x.abs().amax(-1, keepdim=True) / 7          # the scale that reaches the largest value
    _, e = torch.frexp(least.clamp_min(2.0 ** -20))     # least = f 2^e with f in [1/2, 1)
    step = torch.exp2(e.to(torch.float64) - 4)          # spacing of scales with 3 mantissa bits
    scale = (torch.ceil(least / step) * step).clamp(2.0 ** -20, 1.875 * 2.0 ** 11)
    new = (torch.round(x / scale).clamp(-7, 7) * scale).reshape(B, case["C"], tpf, D)
    values = _exact_values(s["codes"], s["scales"]).reshape(B, W, tpf, D)
    slot = s["slot_frame"].clone()
    for j in range(case["C"]):
        f = case["first"] + j
        values[:, f % W] = new[:, j]
        slot[:, f % W] = f
    return values.reshape(B, W * tpf, D), slot


def _exact_attn(s):
    """Sample by sample and head by head; rotations as products of complex numbers."""
    case = s["case"]
    tpf, n_q, D, n_valid = _ring_sizes(case)
    d_c, B, H = case["d_c"], case["B"], 12

    def turned(x, frames):
        z = torch.view_as_complex(x.reshape(*x.shape[:-1], -1, 2).contiguous())
        tok = torch.arange(x.shape[0], device="cuda")
        at = {0: frames.to(torch.float64)[tok // tpf],
              1: ((tok % tpf) // case["frame_w"]).to(torch.float64),
              2: ((tok % tpf) % case["frame_w"]).to(torch.float64)}
        angle = torch.stack([at[axis] * BASE ** (-i / n)
                             for axis, n in enumerate(_rope_pairs(case["d_rope"]))
                             for i in range(n)], -1)
        z = z * torch.polar(torch.ones_like(angle), angle)
        return torch.view_as_real(z).flatten(-2)

    out = torch.empty((B, n_q, H, 128), device="cuda", dtype=torch.float64)
    lse = torch.empty((B, H, n_q), device="cuda", dtype=torch.float64)
    now = case["first"] + torch.arange(case["C"], device="cuda")
    for b in range(B):
        ring = _exact_values(s["codes"][b, :n_valid * tpf], s["scales"][b, :n_valid * tpf])
        chunk = s["chunk"][b].to(torch.float64)
        c = torch.cat((ring[:, :d_c], chunk[:, :d_c]))
        r = turned(chunk[:, d_c:], now)
        if n_valid:
            r = torch.cat((turned(ring[:, d_c:], s["slot_frame"][b, :n_valid]), r))
        for h in range(H):
            if case["from_cq"]:
                q = s["c_q"][b].to(torch.float64) @ s["w_qcat"][h].to(torch.float64).T
                qc, qr = q[:, :d_c], turned(q[:, d_c:], now)
            else:
                q = s["q"][b, :, h].to(torch.float64)
                qc, qr = q[:, :d_c], q[:, d_c:]
            x = (qc @ c.T + qr @ r.T) * s["scale"]
            lse[b, h] = torch.logsumexp(x, 1)
            p = torch.exp(x - lse[b, h][:, None])
            out[b, :, h] = (p @ c) @ s["w_uv"][h].to(torch.float64).T
    return out.reshape(B, n_q, H * 128), lse
