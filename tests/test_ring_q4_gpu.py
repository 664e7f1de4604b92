"""The latent ring held in 4 bits on the GPU: codes, scales and values bit for bit against the
definition; attention over it against the float64 definition on the ring's values, element by
element within bounds derived from the roundings made, and a rollout against the oracle."""
import dataclasses

import numpy as np
import pytest
import torch

import oracle
from mla_latent_kv_attn_b200 import api, inputs, rollout
from parity_util import GpuRun, OracleRun, check_chunk, to_np

pytestmark = pytest.mark.gpu

SMALL = inputs.small_bf16_config()
TOY16 = inputs.with_latent_shape(inputs.CONFIGS[0], 16, 16)      # fp32, whole groups
PATHS = {"tc": api.MLA_PATH_AUTO, "pair": api.MLA_PATH_TC_PAIR, "simt": api.MLA_PATH_SIMT}


def _chunk(c, seed, std=1.0):
    n_q = c.chunk_frames * c.frame_h * c.frame_w
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((c.batch, n_q, c.d_c + c.d_rope), generator=g, device="cuda") * std
    return x.to(api.torch_dtype(c))


def _append(c, ring, lat, first):
    api.mla_cache_append_q4(c, lat, ring.codes, ring.scales, ring.slot_frame, first)


def _edge_values(lat):
    """Rows with what a group can hold at its edges."""
    x = lat.clone()
    x[0, 0] = 0
    x[0, 1, :16] = 1.75                       # max / 7 is a scale itself
    x[0, 2, :16] = 1e-8                       # below the smallest scale
    x[0, 3, 5] = 1e6                          # beyond the largest: saturates
    x[0, 4, :16] = torch.arange(-8, 8, device="cuda") / 2 * 0.25   # ties between codes
    x[0, 5, 3] = float("nan")
    x[0, 6, 3] = float("inf")
    x[0, 7, 3] = -float("inf")
    x[0, 8] = -0.0
    return x


@pytest.mark.parametrize("cfg", [SMALL, TOY16, inputs.with_latent_shape(SMALL, 256, 64),
                                 dataclasses.replace(SMALL, frame_h=3, frame_w=7, window_frames=5,
                                                     chunk_frames=2, batch=3)],
                         ids=["small", "fp32", "wide", "odd"])
def test_append_and_read_match_the_definition(cfg):
    c = api.make_config(cfg)
    tpf, W, D = cfg.tokens_per_frame, cfg.window_frames, cfg.d_latent
    ring = rollout.RingQ4(c)
    assert (ring.read() == 0).all()
    codes = np.full((cfg.batch, W, tpf, D // 2), 0x88, np.uint8)
    scales = np.zeros((cfg.batch, W, tpf, D // 16), np.uint8)
    slots = np.full((cfg.batch, W), -1, np.int32)
    for ch in range(4):                                    # wraps
        lat = _edge_values(_chunk(c, ch, std=10.0 ** (ch - 2)))
        first = ch * cfg.chunk_frames
        _append(c, ring, lat, first)
        # a NaN is stored as 0 and passed over by the group's maximum
        x = np.nan_to_num(to_np(lat), nan=0.0, posinf=1e30, neginf=-1e30)
        qc, qs = oracle.q4_encode(x)
        for f in range(cfg.chunk_frames):
            s = (first + f) % W
            codes[:, s], scales[:, s] = qc[:, f * tpf:(f + 1) * tpf], qs[:, f * tpf:(f + 1) * tpf]
            slots[:, s] = first + f
        assert np.array_equal(ring.codes.cpu().numpy().reshape(codes.shape), codes), ch
        assert np.array_equal(ring.scales.cpu().numpy().reshape(scales.shape), scales), ch
        assert np.array_equal(ring.slot_frame.cpu().numpy(), slots), ch
        assert np.array_equal(to_np(ring.read()).reshape(cfg.batch, W, tpf, D),
                              oracle.q4_decode(codes, scales)), ch


def _filled(cfg, path, chunks, seed=0):
    """A 4-bit ring after `chunks` appends, and a plain ring holding its values."""
    c = api.make_config(cfg, kernel_path=path)
    q4, plain = rollout.RingQ4(c), rollout.Ring(c)
    for ch in range(chunks):
        _append(c, q4, _chunk(c, seed + ch), ch * cfg.chunk_frames)
    plain.cache.copy_(q4.read())
    plain.slot_frame.copy_(q4.slot_frame)
    return c, q4, plain


def _query(c, seed):
    n_q = c.chunk_frames * c.frame_h * c.frame_w
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randn((c.batch, n_q, c.n_heads, c.d_c + c.d_rope), generator=g, device="cuda")
    w_uv = torch.randn((c.n_heads, c.d_head, c.d_c), generator=g, device="cuda") * c.d_c ** -0.5
    return q.to(api.torch_dtype(c)), w_uv.to(api.torch_dtype(c))


# The tensor-core attention over the 4-bit ring rounds its operands to fp16: P and the rotated keys
# by 2^-11 of themselves (P also by half of fp16's least step, beside a largest value of 1 or more),
# a formed query likewise; sines and cosines of these small angles are off by 2^-20; an exponential
# may come from a polynomial that is off by 1e-4.
F16 = 2.0 ** -11


def _reference(c, cfg, values, slots, lat, q, e_q, w_uv, first, n_valid):
    """out [B, n_q, H, d_head], lse, and the bounds on their errors, from the ring's values."""
    d = oracle.dims_from(cfg)
    res = []
    for b in range(cfg.batch):
        nc = n_valid * cfg.tokens_per_frame
        pos = np.concatenate([oracle.token_positions([int(t) for t in slots[b][:n_valid]], d),
                              oracle.token_positions(range(first, first + cfg.chunk_frames), d)]
                             ) if n_valid else oracle.token_positions(
                                 range(first, first + cfg.chunk_frames), d)
        rows = np.concatenate([values[b][:nc], lat[b]])
        raw = rows[:, cfg.d_c:]
        k_r = oracle.rope3d(raw, pos, d)
        size = np.abs(raw)[:, 0::2] + np.abs(raw)[:, 1::2]        # of a pair: bounds |rotated|
        e_k = F16 * np.abs(k_r) + 2.0 ** -20 * np.repeat(size, 2, axis=1) + 2.0 ** -25
        res.append(oracle.latent_attention(q[b], rows[:, :cfg.d_c], k_r, w_uv, cfg.softmax_scale,
                                           e_q[b], e_k, F16 + 1.1e-4, 2.0 ** -25))
    return [np.stack(x) for x in zip(*res)]


def _within(got, want, bound, r):
    err = np.abs(to_np(got) - want)
    limit = bound * (1 + r) + r * np.abs(want)
    assert np.isfinite(to_np(got)).all()
    assert (err <= limit).all(), float((err / limit).max())
    return err


@pytest.mark.parametrize("chunks", [0, 1, 5])
@pytest.mark.parametrize("path,d_c,d_rope", [("tc", 192, 32), ("tc", 128, 16), ("tc", 192, 64),
                                             ("tc", 256, 64), ("tc", 256, 32), ("tc", 256, 16),
                                             ("pair", 192, 32)])
def test_attention_matches_the_definition(path, d_c, d_rope, chunks):
    cfg = inputs.with_latent_shape(SMALL, d_c, d_rope)
    c, q4, plain = _filled(cfg, PATHS[path], chunks)
    first, n_valid = rollout.chunk_schedule(cfg.chunk_frames, cfg.window_frames, chunks)
    lat, (q, w_uv) = _chunk(c, 100), _query(c, 101)
    b = rollout.ChunkBuffers(c, q4=True)
    b.workspace.fill_(0xFF)                                # contents on entry must not matter
    need = max(api.mla_attention_q4_workspace_bytes(c, n_valid), 256)
    call = lambda w, out: api.mla_attention_fwd_q4(
        c, q, lat, q4.codes, q4.scales, q4.slot_frame, n_valid, first, w, out, b.lse,
        b.workspace[:need], b.dev_status)
    call(w_uv, b.o)
    torch.cuda.synchronize()
    rollout.check_device_status(b)
    assert (b.workspace[need:] == 0xFF).all()
    args = (c, cfg, to_np(plain.cache), plain.slot_frame.cpu().numpy(), to_np(lat), to_np(q),
            np.zeros(q.shape))
    out, lse, e_out, e_lse = _reference(*args, to_np(w_uv), first, n_valid)
    _within(b.o.view(*q.shape[:3], -1), out, e_out, 2.0 ** -8)
    err = _within(b.lse, lse, e_lse, 0.0)
    assert np.linalg.norm(err) <= 1e-5 * np.linalg.norm(lse)
    call(None, b.o_lat)
    eye = np.broadcast_to(np.eye(d_c), (cfg.n_heads, d_c, d_c))
    out, lse, e_out, e_lse = _reference(*args, eye, first, n_valid)
    _within(b.o_lat, out, e_out, 2.0 ** -8)
    _within(b.lse, lse, e_lse, 0.0)


@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** -20, 300.0, 2.0 ** 100])
@pytest.mark.parametrize("d_c,d_rope", [(192, 32), (256, 32)])
def test_queries_of_any_size(d_c, d_rope, size):
    """bf16's range of queries: rows far outside fp16's, with the score scale to match."""
    cfg = dataclasses.replace(inputs.with_latent_shape(SMALL, d_c, d_rope), n_heads=2)
    c, q4, plain = _filled(cfg, api.MLA_PATH_AUTO, 2)
    first, n_valid = rollout.chunk_schedule(cfg.chunk_frames, cfg.window_frames, 2)
    lat, (q, w_uv) = _chunk(c, 100), _query(c, 101)
    q[:, ::3] *= 2.0 ** -6                                  # rows of different sizes
    q[:, 1::3, :, ::2] *= 2.0 ** -9
    c.softmax_scale = c.softmax_scale / size
    big = (q.float() * size).bfloat16()
    b, plain_b = rollout.ChunkBuffers(c, q4=True), rollout.ChunkBuffers(c, q4=True)
    api.mla_attention_fwd_q4(c, big, lat, q4.codes, q4.scales, q4.slot_frame, n_valid, first, w_uv,
                             b.o, b.lse, b.workspace, b.dev_status)
    c.softmax_scale = cfg.softmax_scale
    api.mla_attention_fwd_q4(c, q, lat, q4.codes, q4.scales, q4.slot_frame, n_valid, first, w_uv,
                             plain_b.o, plain_b.lse, plain_b.workspace, plain_b.dev_status)
    for x, seen in ((b, to_np(big) / size), (plain_b, to_np(q))):     # (a big row is rounded anew)
        out, lse, e_out, e_lse = _reference(c, cfg, to_np(plain.cache),
                                            plain.slot_frame.cpu().numpy(), to_np(lat), seen,
                                            np.zeros(q.shape), to_np(w_uv), first, n_valid)
        _within(x.o.view(*q.shape[:3], -1), out, e_out, 2.0 ** -8)
        # (size / size in fp32 leaves 2^-23 of a score)
        _within(x.lse, lse, e_lse + 2.0 ** -20 * np.abs(lse).max(), 0.0)


@pytest.mark.parametrize("chunks", [0, 2, 5])
@pytest.mark.parametrize("d_c,d_rope", [(192, 32), (128, 64), (192, 16)])
def test_attention_from_cq_matches_the_definition(d_c, d_rope, chunks):
    cfg = inputs.with_latent_shape(SMALL, d_c, d_rope)
    c, q4, plain = _filled(cfg, api.MLA_PATH_AUTO, chunks)
    first, n_valid = rollout.chunk_schedule(cfg.chunk_frames, cfg.window_frames, chunks)
    lat, (_, w_uv) = _chunk(c, 100), _query(c, 101)
    g = torch.Generator(device="cuda").manual_seed(7)
    c_q = torch.randn((cfg.batch, cfg.n_q, c.d_cq), generator=g, device="cuda").bfloat16()
    w_q = (torch.randn((c.n_heads, cfg.d_latent, c.d_cq), generator=g, device="cuda")
           * c.d_cq ** -0.5).bfloat16()
    b = rollout.ChunkBuffers(c, q4=True)
    api.mla_attention_fwd_from_cq_q4(c, c_q, w_q, lat, q4.codes, q4.scales, q4.slot_frame, n_valid,
                                     first, w_uv, b.o, b.lse, b.workspace, b.dev_status)
    torch.cuda.synchronize()
    rollout.check_device_status(b)
    d = oracle.dims_from(cfg)
    pos = oracle.token_positions(range(first, first + cfg.chunk_frames), d)
    q = np.einsum("bnk,hdk->bnhd", to_np(c_q), to_np(w_q))
    size = np.einsum("bnk,hdk->bnhd", np.abs(to_np(c_q)), np.abs(to_np(w_q)))
    e_q = (c.d_cq + 4) * 2.0 ** -23 * size
    pair = np.abs(q[..., d_c::2]) + np.abs(q[..., d_c + 1::2])
    for x in range(cfg.batch):
        for h in range(cfg.n_heads):
            q[x, :, h, d_c:] = oracle.rope3d(q[x, :, h, d_c:], pos, d)
    e_r = e_q[..., d_c::2] + e_q[..., d_c + 1::2] + 2.0 ** -20 * pair
    e_q[..., d_c:] = np.repeat(e_r, 2, axis=-1)
    # fp16: 2^-11 of an element, or of a row whose largest is 2^13, half the least step 2^-24
    e_q += F16 * (np.abs(q) + e_q) + 2.0 ** -38 * np.abs(q).max(-1, keepdims=True)
    out, lse, e_out, e_lse = _reference(c, cfg, to_np(plain.cache), plain.slot_frame.cpu().numpy(),
                                        to_np(lat), q, e_q, to_np(w_uv), first, n_valid)
    _within(b.o.view(*q.shape[:3], -1), out, e_out, 2.0 ** -8)
    err = _within(b.lse, lse, e_lse, 0.0)
    assert np.linalg.norm(err) <= 1e-5 * np.linalg.norm(lse)


@pytest.mark.parametrize("scale", [1e-8, 1e-30, 1e-42])
@pytest.mark.parametrize("d_c,d_rope,from_cq", [(192, 32, False), (256, 32, False), (192, 32, True)])
def test_rows_of_zeros_and_the_smallest_scales(d_c, d_rope, from_cq, scale):
    """Scores of nothing: rows of zeros, of the least numbers and ordinary ones under scales down to
    fp32's subnormal ones weigh every key alike, in tiles with masked columns too."""
    cfg = dataclasses.replace(inputs.with_latent_shape(SMALL, d_c, d_rope), n_heads=2)
    c, q4, plain = _filled(cfg, api.MLA_PATH_AUTO, 2)
    first, n_valid = rollout.chunk_schedule(cfg.chunk_frames, cfg.window_frames, 2)
    lat, (q, w_uv) = _chunk(c, 100), _query(c, 101)
    c.softmax_scale = scale
    b = rollout.ChunkBuffers(c, q4=True)
    ring = (lat, q4.codes, q4.scales, q4.slot_frame, n_valid, first, w_uv, b.o, b.lse, b.workspace,
            b.dev_status)
    if from_cq:
        g = torch.Generator(device="cuda").manual_seed(7)
        c_q = torch.randn((cfg.batch, cfg.n_q, c.d_cq), generator=g, device="cuda").bfloat16()
        w_q = (torch.randn((c.n_heads, cfg.d_latent, c.d_cq), generator=g, device="cuda")
               * c.d_cq ** -0.5).bfloat16()
        c_q[:, ::3] = 0
        c_q[:, 1::3] *= 2.0 ** -120
        api.mla_attention_fwd_from_cq_q4(c, c_q, w_q, *ring)
        q = torch.einsum("bnk,hdk->bnhd", c_q.double(), w_q.double())    # (its rotation is nothing here)
    else:
        q[:, ::3] = 0
        q[:, 1::3] *= 2.0 ** -128
        api.mla_attention_fwd_q4(c, q, *ring)
    torch.cuda.synchronize()
    rollout.check_device_status(b)
    seen = to_np(q).astype(np.float64) * (c.softmax_scale / cfg.softmax_scale)
    out, lse, e_out, e_lse = _reference(c, cfg, to_np(plain.cache), plain.slot_frame.cpu().numpy(),
                                        to_np(lat), seen, F16 * np.abs(seen), to_np(w_uv), first,
                                        n_valid)
    _within(b.o.view(*q.shape[:3], -1), out, e_out, 2.0 ** -8)
    _within(b.lse, lse, e_lse, 0.0)


def test_chunk_latents_beyond_fp16():
    """The chunk's own latents enter the tensor-core attention held at fp16's limits; the ring holds
    no more than 26880 in any case."""
    c, q4, _ = _filled(SMALL, api.MLA_PATH_AUTO, 1)
    lat, (q, w_uv) = _chunk(c, 100), _query(c, 101)
    outs = []
    for top in (65504.0, 1e6, 3e38):
        x = lat.clone()
        x[0, 7, 5], x[0, 9, 150] = top, -top
        b = rollout.ChunkBuffers(c, q4=True)
        api.mla_attention_fwd_q4(c, q * 2.0 ** -12, x, q4.codes, q4.scales, q4.slot_frame, 3, 3, w_uv,
                                 b.o, b.lse, b.workspace, b.dev_status)
        outs.append(b.o)
        assert torch.isfinite(b.o).all()
    assert torch.equal(outs[1], outs[2])


@pytest.mark.parametrize("d_c,d_rope", [(192, 32), (256, 32)])
def test_chunk_values_beyond_fp16_are_taken_as_its_limits(d_c, d_rope):
    """Contents and rotated positional values beyond 65504 give the bits that 65504 gives, and the
    definition's results with such values held at 65504."""
    cfg = dataclasses.replace(inputs.with_latent_shape(SMALL, d_c, d_rope), n_heads=2)
    c, q4, plain = _filled(cfg, api.MLA_PATH_AUTO, 1)
    lat, (q, w_uv) = _chunk(c, 100), _query(c, 101)
    q = q * 2.0 ** -12

    def call(content, positional):
        x = lat.clone()
        x[0, 7, 5], x[0, 9, d_c - 1] = content, -content
        x[1, 100, d_c:] = 0
        x[1, 100, d_c::4] = positional             # alone in its pair: rotated to (x cos, x sin)
        b = rollout.ChunkBuffers(c, q4=True)
        api.mla_attention_fwd_q4(c, q, x, q4.codes, q4.scales, q4.slot_frame, 3, 3, w_uv, b.o, b.lse,
                                 b.workspace, b.dev_status)
        torch.cuda.synchronize()
        rollout.check_device_status(b)
        return x, b.o, b.lse

    # every nonzero sine and cosine here is above 1e-4, so from 1e9 on all such values are beyond
    runs = [call(*v) for v in ((65504.0, 1e9), (1e6, 1e20), (3e38, 3e38))]
    for _, o, lse in runs[1:]:
        assert torch.equal(o, runs[0][1]) and torch.equal(lse, runs[0][2])
    x, o, lse = call(1e6, 1e6)
    d = oracle.dims_from(cfg)
    slots = plain.slot_frame.cpu().numpy()
    for b in range(cfg.batch):
        pos = np.concatenate([oracle.token_positions([int(t) for t in slots[b][:3]], d),
                              oracle.token_positions(range(3, 3 + cfg.chunk_frames), d)])
        rows = np.concatenate([to_np(plain.cache)[b][:3 * cfg.tokens_per_frame], to_np(x)[b]])
        raw = rows[:, d_c:]
        k_r = oracle.rope3d(raw, pos, d)
        size = np.abs(raw)[:, 0::2] + np.abs(raw)[:, 1::2]
        e_rot = 2.0 ** -20 * np.repeat(size, 2, axis=1)
        e_k = np.where(np.abs(k_r) - e_rot > 65504, 0, F16 * np.abs(k_r) + e_rot + 2.0 ** -25)
        out, ls, e_out, e_lse = oracle.latent_attention(
            to_np(q)[b], np.clip(rows[:, :d_c], -65504, 65504), np.clip(k_r, -65504, 65504),
            to_np(w_uv), cfg.softmax_scale, np.zeros(q.shape[1:]), e_k, F16 + 1.1e-4, 2.0 ** -25)
        _within(o.view(*q.shape[:3], -1)[b], out, e_out, 2.0 ** -8)
        _within(lse[b], ls, e_lse, 0.0)


@pytest.mark.parametrize("fuse_uv", [True, False])
def test_cuda_cores_equal_the_call_on_the_rings_values(fuse_uv):
    c, q4, plain = _filled(SMALL, api.MLA_PATH_SIMT, 5)
    first, n_valid = rollout.chunk_schedule(SMALL.chunk_frames, SMALL.window_frames, 5)
    lat, (q, w_uv) = _chunk(c, 100), _query(c, 101)
    a, b = rollout.ChunkBuffers(c), rollout.ChunkBuffers(c, q4=True)
    w = w_uv if fuse_uv else None
    api.mla_attention_fwd(c, q, lat, plain.cache, plain.slot_frame, n_valid, first, w,
                          a.o if fuse_uv else a.o_lat, a.lse, a.workspace, a.dev_status)
    api.mla_attention_fwd_q4(c, q, lat, q4.codes, q4.scales, q4.slot_frame, n_valid, first, w,
                             b.o if fuse_uv else b.o_lat, b.lse, b.workspace, b.dev_status)
    assert torch.equal(a.lse, b.lse)
    assert torch.equal(a.o if fuse_uv else a.o_lat, b.o if fuse_uv else b.o_lat)


def test_fp32_ring_on_cuda_cores():
    c, q4, plain = _filled(TOY16, api.MLA_PATH_AUTO, 3)
    first, n_valid = rollout.chunk_schedule(TOY16.chunk_frames, TOY16.window_frames, 3)
    lat, (q, w_uv) = _chunk(c, 100), _query(c, 101)
    a, b = rollout.ChunkBuffers(c), rollout.ChunkBuffers(c, q4=True)
    api.mla_attention_fwd(c, q, lat, plain.cache, plain.slot_frame, n_valid, first, w_uv, a.o,
                          a.lse, a.workspace, a.dev_status)
    api.mla_attention_fwd_q4(c, q, lat, q4.codes, q4.scales, q4.slot_frame, n_valid, first, w_uv,
                             b.o, b.lse, b.workspace, b.dev_status)
    assert torch.equal(a.o, b.o) and torch.equal(a.lse, b.lse)


@pytest.mark.parametrize("fused_q", [True, False])
def test_rollout_matches_the_oracle_on_the_quantised_ring(fused_q):
    """A rollout whose ring wraps, with cross attention to a prompt between the chunks: every
    chunk's output against the oracle whose window holds the 4-bit ring's own values."""
    cfg = SMALL
    g, o = GpuRun(cfg), OracleRun(cfg, inputs.layer_weights(cfg))
    g.ring, g.buf = rollout.RingQ4(g.c), rollout.ChunkBuffers(g.c, q4=True)
    rows = np.arange(cfg.n_q)
    gen = torch.Generator(device="cuda").manual_seed(3)
    kv = torch.randn((2, cfg.batch, 50, cfg.n_heads, cfg.d_head), generator=gen, device="cuda")
    text = rollout.EncoderStates(kv[0].bfloat16(), kv[1].bfloat16(), n_heads=cfg.n_heads,
                                 kv_len=torch.tensor([50, 21], device="cuda", dtype=torch.int32))
    for ch in range(cfg.n_chunks):
        x = inputs.chunk_x(cfg, ch)
        g.load_x(x)
        out = rollout.attend_chunk(g.c, g.w, g.ring, g.buf, ch, fused_q=fused_q)
        q = out.unflatten(-1, (cfg.n_heads, cfg.d_head))
        cross = text.attend(q, torch.empty_like(q))
        rollout.append_chunk(g.c, g.ring, g.buf, ch)
        torch.cuda.synchronize()
        rollout.check_device_status(g.buf)
        ores = o.step(ch, x, rows)
        check_chunk(f"q4.chunk{ch}", cfg, dict(o=to_np(out), lse=to_np(g.buf.lse),
                                               c_q=to_np(g.buf.c_q),
                                               chunk_lat=to_np(g.buf.chunk_lat)), ores, rows)
        want, _, e, _ = oracle.cross_attention(to_np(q), to_np(text.k), to_np(text.v), [50, 21],
                                               cfg.d_head ** -0.5, p_rel=2.0 ** -8 + 1.1e-4)
        assert (np.abs(to_np(cross) - want) <= e * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)).all()
        # the oracle's window takes the values that the ring stands for
        values = to_np(g.ring.read())
        tpf = cfg.tokens_per_frame
        for b in range(cfg.batch):
            for rec in o.windows[b].frames:
                s = rec.t % cfg.window_frames
                v = values[b, s * tpf:(s + 1) * tpf]
                rec.c_kv, rec.k_r = v[:, :cfg.d_c], v[:, cfg.d_c:]
    assert int(text.dev_status) == 0


def test_layer_stack_and_graphs_over_4_bit_rings():
    """Layers that share one workspace, eager and captured, and a chunk graph: the same bits."""
    cfg = SMALL
    c = api.make_config(cfg)
    lws = [inputs.layer_weights(cfg, l) for l in range(2)]
    xs = {(ch, s, l): torch.from_numpy(inputs.chunk_x(cfg, ch, s, l)).to(torch.bfloat16).cuda()
          for ch in range(cfg.n_chunks) for s in range(2) for l in range(2)}
    eager = rollout.LayerStack(c, [rollout.upload_weights(c, lw) for lw in lws], q4=True)
    graphed = rollout.LayerStack(c, [rollout.upload_weights(c, lw) for lw in lws], q4=True)
    for ch in range(cfg.n_chunks):
        x_of = lambda s, l, ch=ch: xs[(ch, s, l)]
        eager.run_chunk(ch, 2, x_of)
        want = eager.buf.o.clone()
        graphed.capture_chunk(ch, 2, x_of).replay()
        torch.cuda.synchronize()
        assert torch.equal(graphed.buf.o, want), ch
        for a, b in zip(eager.rings, graphed.rings):
            assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
            assert torch.equal(a.slot_frame, b.slot_frame)
    rollout.check_device_status(graphed.buf)
    # the same rollout of layer 0 by hand and by chunk graphs
    w = rollout.upload_weights(c, lws[0])
    one, two = rollout.RingQ4(c), rollout.RingQ4(c)
    b1, b2 = rollout.ChunkBuffers(c, q4=True), rollout.ChunkBuffers(c, q4=True)
    for ch in range(cfg.n_chunks):
        b1.x.copy_(xs[(ch, 1, 0)])
        o1 = rollout.run_chunk(c, w, one, b1, ch)
        o2 = rollout.ChunkGraph(c, w, two, b2, ch, x=xs[(ch, 1, 0)]).replay()
        torch.cuda.synchronize()
        assert torch.equal(o1, o2)
    assert torch.equal(one.codes, two.codes) and torch.equal(one.codes, eager.rings[0].codes)
    saved = one.state_dict()
    three = rollout.RingQ4(c)
    three.load_state_dict(saved)
    assert torch.equal(three.read(), one.read())


def test_host_streamer_serves_4_bit_rings():
    """Two rollouts in turn through one streamer: outputs and rings of each as when run alone."""
    cfg = SMALL
    c = api.make_config(cfg)
    w = rollout.upload_weights(c, inputs.layer_weights(cfg))
    xs = [[torch.from_numpy(inputs.chunk_x(cfg, ch, layer=r)).to(torch.bfloat16)
           for ch in range(cfg.n_chunks)] for r in range(2)]
    buf = rollout.ChunkBuffers(c, q4=True)
    refs, rings = [], [rollout.RingQ4(c) for _ in range(2)]
    for r in range(2):
        refs.append([])
        for ch in range(cfg.n_chunks):
            buf.x.copy_(xs[r][ch])
            refs[r].append(rollout.run_chunk(c, w, rings[r], buf, ch).cpu().clone())
    served = [rollout.RingQ4(c) for _ in range(2)]
    st = rollout.HostStreamer(c, w, served[0])
    outs = [[torch.empty_like(refs[0][0]).pin_memory() for _ in range(cfg.n_chunks)]
            for _ in range(2)]
    for ch in range(cfg.n_chunks):
        for r in range(2):
            st.submit(ch, xs[r][ch].pin_memory(), outs[r][ch], ring=served[r])
    st.finish()
    torch.cuda.synchronize()
    st.check_device_status()
    for r in range(2):
        for ch in range(cfg.n_chunks):
            assert torch.equal(outs[r][ch], refs[r][ch]), (r, ch)
        assert torch.equal(served[r].codes, rings[r].codes), r
        assert torch.equal(served[r].scales, rings[r].scales), r


def test_ring_of_almost_2_to_31_values():
    """Appending to the last slots of the largest ring, and its values read back."""
    cfg = dataclasses.replace(inputs.CONFIGS[1], window_frames=(2 ** 31 - 1) // (1560 * 224) - 1)
    c = api.make_config(cfg)
    tpf, W, C = cfg.tokens_per_frame, cfg.window_frames, cfg.chunk_frames
    ring = rollout.RingQ4(c)
    lat = _chunk(c, 4)
    first = 2 * W - C                               # the window's last slots, once around
    _append(c, ring, lat, first)
    small = dataclasses.replace(cfg, window_frames=C)
    cs = api.make_config(small)
    want = rollout.RingQ4(cs)
    _append(cs, want, lat, 0)
    assert torch.equal(ring.codes[:, -C * tpf:], want.codes)
    assert torch.equal(ring.scales[:, -C * tpf:], want.scales)
    assert ring.slot_frame[0, -C:].tolist() == list(range(first, first + C))
    assert (ring.slot_frame[0, :-C] == -1).all() and (ring.codes[:, :-C * tpf] == 0x88).all()
    values = ring.read()
    assert torch.equal(values[:, -C * tpf:], want.read())
    assert not values[:, :-C * tpf].any()


def test_attention_over_a_ring_of_almost_2_to_31_values():
    """The last frame of the largest ring, whose keys outweigh ten million rows of zeros (each by e^40 or
    more), against the call on a ring of that frame alone."""
    cfg = dataclasses.replace(inputs.CONFIGS[1], n_heads=1, frame_h=8, frame_w=8, chunk_frames=1,
                              window_frames=(2 ** 31 - 1) // (64 * 224))
    W, tpf, d_c = cfg.window_frames, 64, cfg.d_c
    lat, last = torch.zeros((2, 1, tpf, cfg.d_latent), device="cuda", dtype=torch.bfloat16)
    g = torch.Generator(device="cuda").manual_seed(9)
    for x in (lat, last):                                  # (no positional values: no rotation)
        x[..., :d_c] = torch.randn((1, tpf, d_c), generator=g, device="cuda").bfloat16()
        x[..., 0] = 8
    w_uv = _query(api.make_config(cfg), 101)[1]
    q = torch.zeros((1, tpf, 1, cfg.d_latent), device="cuda", dtype=torch.bfloat16)
    q[..., :d_c] = torch.randn((1, tpf, 1, d_c), generator=g, device="cuda").bfloat16() / 8
    q[..., 0] = 8 / cfg.softmax_scale                      # a score of 64 with every other key
    res = []
    for c in (cfg, dataclasses.replace(cfg, window_frames=1)):
        cc = api.make_config(c)
        ring, buf = rollout.RingQ4(cc), rollout.ChunkBuffers(cc, q4=True)
        _append(cc, ring, last, W - 1)                     # (slot W - 1, and the one slot)
        ring.slot_frame.copy_(torch.arange(W - c.window_frames, W, dtype=torch.int32))
        api.mla_attention_fwd_q4(cc, q, lat, ring.codes, ring.scales, ring.slot_frame,
                                 c.window_frames, W, w_uv, buf.o, buf.lse, buf.workspace,
                                 buf.dev_status)
        torch.cuda.synchronize()
        rollout.check_device_status(buf)
        res.append((cc, c, buf, ring))
    cc, c, _, ring = res[1]
    out, lse, e_out, e_lse = _reference(cc, c, to_np(ring.read()), ring.slot_frame.cpu().numpy(),
                                        to_np(lat), to_np(q), np.zeros(q.shape), to_np(w_uv), W, 1)
    for _, _, buf, _ in res:
        _within(buf.o.view(1, tpf, 1, -1), out, e_out, 2.0 ** -8)
        _within(buf.lse, lse, e_lse, 0.0)


def test_prefill_on_a_side_stream():
    cfg = SMALL
    c = api.make_config(cfg)
    w = rollout.upload_weights(c, inputs.layer_weights(cfg))
    a, b = rollout.RingQ4(c), rollout.RingQ4(c)
    buf, other = rollout.ChunkBuffers(c, q4=True), rollout.ChunkBuffers(c, q4=True)
    side = torch.cuda.Stream()
    x = torch.from_numpy(inputs.chunk_x(cfg, 0)).to(torch.bfloat16).cuda()
    buf.x.copy_(x)
    other.x.copy_(x)
    rollout.run_chunk(c, w, a, buf, 0)
    side.wait_stream(torch.cuda.current_stream())
    rollout.prefill_chunk(c, w, b, other, 0, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)


@pytest.mark.parametrize("raw", [False, True])
def test_read_on_a_side_stream(raw):
    """The values are written into memory of the stream that writes them: a block just freed on the
    current stream, behind work that has yet to read and write it, is not taken."""
    c, ring, _ = _filled(SMALL, api.MLA_PATH_AUTO, 2)
    want = ring.read()
    side = torch.cuda.Stream()
    block = torch.full_like(want, 5.0)
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)                          # some 50 ms on the current stream
    kept = block.clone()
    block.fill_(7.0)
    del block
    got = ring.read(stream=side.cuda_stream if raw else side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert (kept == 5.0).all()


def test_bad_calls_are_refused():
    c, q4, _ = _filled(SMALL, api.MLA_PATH_AUTO, 1)
    buf = rollout.ChunkBuffers(c, q4=True)
    lat, (q, w_uv) = _chunk(c, 0), _query(c, 1)
    call = lambda ws=buf.workspace, codes=q4.codes, n_valid=3: api.mla_attention_fwd_q4(
        c, q, lat, codes, q4.scales, q4.slot_frame, n_valid, 3, w_uv, buf.o, buf.lse, ws,
        buf.dev_status)
    call()
    need = api.mla_attention_q4_workspace_bytes(c, 3)
    for bad in (dict(ws=buf.workspace[:need - 1]), dict(ws=None), dict(ws=buf.workspace[16:]),
                dict(n_valid=c.window_frames + 1), dict(codes=q4.codes.cpu())):
        with pytest.raises(api.MLAError):
            call(**bad)
    with pytest.raises(ValueError):
        call(codes=q4.codes[:, :-1])
    # a workspace sized for a plain ring does not serve
    with pytest.raises(api.MLAError):
        call(ws=rollout.ChunkBuffers(c).workspace)
