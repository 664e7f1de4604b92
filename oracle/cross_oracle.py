"""Float64 definitions of the cross attention to an encoder's states and of the 4-bit latent ring,
with bounds on how far results computed in a lower precision may lie from them."""
from __future__ import annotations

import numpy as np


# fp32 exponentials below the least normal number become 0, and one from a polynomial whose argument
# is held at -125 or more becomes 2^-125: a probability may be off by that, whatever its size.  (In
# the gradients it stands beside factors such as g.v, so even 0 <-> 2^-125 shows in results that
# should be 1e-41.)
TINY = 2.0 ** -125
F32 = 2.0 ** -23     # a step of fp32: a sum of n terms is off by at most n F32 sum |term|


def _score_error(q, k, scale, x, lse):
    """Bound on the error of x - lse when x = scale q.k comes from fp32 sums and lse is fp32."""
    return ((q.shape[1] + 4) * F32 * scale * (np.abs(q) @ np.abs(k).T) +
            4 * F32 * (np.abs(x) + np.abs(lse)[:, None] + 1))


def cross_attention(q, k, v, lens, scale, p_rel=0.0):
    """q [B, n_q, H, d], k, v [B, n_kv, Hkv, d], lens [B] -> out [B, n_q, H, d], lse [B, H, n_q],
    and bounds on their errors where sums are fp32 and the probabilities are off by p_rel of
    themselves (before out is rounded)."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    B, n_q, H, d = q.shape
    rep = H // k.shape[2]
    out, e_out = np.zeros((2, B, n_q, H, d))
    lse, e_lse = np.full((B, H, n_q), -np.inf), np.zeros((B, H, n_q))
    for b in range(B):
        n = int(min(max(lens[b], 0), k.shape[1]))
        for h in range(H if n else 0):
            qq, kk, vv = q[b, :, h], k[b, :n, h // rep], v[b, :n, h // rep]
            x = scale * qq @ kk.T
            m = x.max(1)
            lse[b, h] = m + np.log(np.exp(x - m[:, None]).sum(1))
            p = np.exp(x - lse[b, h][:, None])
            out[b, :, h] = p @ vv
            e_x = _score_error(qq, kk, scale, x, lse[b, h])
            e_lse[b, h] = (p * e_x).sum(1) + (n + 4) * F32 + 4 * F32 * np.abs(lse[b, h])
            # numerator and denominator: the weights' own errors, and those of the two sums
            e_p = p * (p_rel + e_x + (n + 4) * F32) + TINY
            e_out[b, :, h] = e_p @ np.abs(vv) + e_p.sum(1)[:, None] * np.abs(out[b, :, h])
    return out, lse, e_out, e_lse


def cross_attention_backward(q, k, v, lens, scale, g, p_rel=0.0, o_rel=0.0, ds_rel=0.0,
                             fwd_rel=0.0):
    """Gradients d_q, d_k, d_v of sum(g * out), and for each a bound on its error (before it is
    rounded): sums in fp32, the probabilities of dV off by p_rel of themselves, dS by ds_rel, and
    delta = g.o formed from a stored output that is off by o_rel and whose probabilities were off
    by fwd_rel.  Every error is taken at its largest with the worst sign."""
    q, k, v, g = (np.asarray(t, dtype=np.float64) for t in (q, k, v, g))
    B, n_q, H, d = q.shape
    Hkv = k.shape[2]
    rep = H // Hkv
    d_q, e_q = np.zeros_like(q), np.zeros_like(q)
    d_k, e_k, d_v, e_v = (np.zeros_like(k) for _ in range(4))
    out, lse, e_out, e_lse = cross_attention(q, k, v, lens, scale, fwd_rel)
    for b in range(B):
        n = int(min(max(lens[b], 0), k.shape[1]))
        for h in range(H if n else 0):
            kh = h // rep
            kk, vv, qq, gg = k[b, :n, kh], v[b, :n, kh], q[b, :, h], g[b, :, h]
            x = scale * qq @ kk.T
            p = np.exp(x - lse[b, h][:, None])
            dp = gg @ vv.T
            delta = (gg * out[b, :, h]).sum(1)[:, None]
            # one state: p = 1 and delta = dP, whatever the two sums round to
            ds = scale * p * (dp - delta) if n > 1 else np.zeros_like(dp)
            d_q[b, :, h] = ds @ kk
            d_k[b, :n, kh] += ds.T @ qq
            d_v[b, :n, kh] += p.T @ gg
            a_k, a_v, a_q, a_g = np.abs(kk), np.abs(vv), np.abs(qq), np.abs(gg)
            e_x = _score_error(qq, kk, scale, x, lse[b, h]) + e_lse[b, h][:, None]
            sums = (d + 4) * F32
            e_delta = (a_g * (o_rel * np.abs(out[b, :, h]) + (1 + o_rel) * e_out[b, :, h])).sum(1) \
                + sums * (a_g * np.abs(out[b, :, h])).sum(1)
            e_dp = sums * (a_g @ a_v.T)
            e_ds = (ds_rel + e_x + 4 * F32) * np.abs(ds) + \
                scale * p * (e_delta[:, None] + e_dp) * (1 + ds_rel) + \
                scale * TINY * (np.abs(dp - delta) + e_delta[:, None] + e_dp)
            if n == 1:
                e_ds = np.zeros_like(e_ds)
            e_q[b, :, h] = e_ds @ a_k + (n + 4) * F32 * (np.abs(ds) @ a_k)
            long = (rep * n_q + 4) * F32
            e_k[b, :n, kh] += e_ds.T @ a_q + long * (np.abs(ds).T @ a_q)
            e_v[b, :n, kh] += (p * (p_rel + e_x) + TINY).T @ a_g + long * (p.T @ a_g)
    return (d_q, d_k, d_v), (e_q, e_k, e_v)


Q4_GROUP = 16


def q4_scale(byte):
    byte = np.asarray(byte, dtype=np.int64)
    return 2.0 ** (byte // 8 - 20) * (1 + (byte % 8) / 8)


_Q4_SCALES = q4_scale(np.arange(256))     # increasing with the byte


def q4_encode(x):
    """codes [..., D/2] and scales [..., D/16] (uint8) of finite values x [..., D]."""
    x = np.asarray(x, dtype=np.float64)
    g = x.reshape(*x.shape[:-1], -1, Q4_GROUP)
    need = np.abs(g).max(-1) / 7
    byte = np.minimum(np.searchsorted(_Q4_SCALES, need, side="left"), 255)
    code = np.clip(np.rint(g / _Q4_SCALES[byte][..., None]), -7, 7).astype(np.int64) + 8
    code = code.reshape(x.shape)
    return (code[..., 0::2] + 16 * code[..., 1::2]).astype(np.uint8), byte.astype(np.uint8)


def q4_decode(codes, scales):
    codes = np.asarray(codes, dtype=np.int64)
    c = np.stack([codes % 16, codes // 16], -1).reshape(*codes.shape[:-1], -1) - 8
    return c * np.repeat(q4_scale(scales), Q4_GROUP, axis=-1)


def latent_attention(q, c, k_r, w_uv, scale, e_q, e_k, p_rel, p_abs):
    """One sample's attention of q [n_q, H, D] to content latents c [n_k, d_c] and rotated keys k_r
    [n_k, d_rope] (both unrounded) with w_uv [H, d_head, d_c]: out [n_q, H, d_head], lse [H, n_q],
    and bounds on their errors when the queries are off by e_q [n_q, H, D], the rotated keys by e_k
    of themselves (e_k [n_k, d_rope]), the exponentials by p_rel of themselves and p_abs of a row's
    largest, sums are fp32 and the latent output is held in 16 bits or more (before out is
    rounded)."""
    n_q, H, D = q.shape
    d_c, n = c.shape[1], c.shape[0]
    keys = np.concatenate([c, k_r], axis=1)
    e_keys = np.concatenate([np.zeros_like(c), e_k], axis=1)
    out, e_out = np.zeros((2, n_q, H, w_uv.shape[1]))
    lse, e_lse = np.zeros((2, H, n_q))
    for h in range(H):
        x = scale * q[:, h] @ keys.T
        m = x.max(1)
        lse[h] = m + np.log(np.exp(x - m[:, None]).sum(1))
        p = np.exp(x - lse[h][:, None])
        e_x = scale * (e_q[:, h] @ (np.abs(keys) + e_keys).T + np.abs(q[:, h]) @ e_keys.T) + \
            _score_error(q[:, h], keys, scale, x, lse[h])
        # the row sum takes the unrounded exponentials: p_rel is rounding and polynomial together
        e_lse[h] = (p * e_x).sum(1) + (p * e_x ** 2).sum(1) + 1.1e-4 + (n + 4) * F32 * \
            (1 + np.abs(lse[h]))
        e_p = p * (np.exp(e_x) * (1 + p_rel + (n + 4) * F32) - 1) + p_abs
        lat = p @ c
        e_lat = e_p @ np.abs(c) + e_p.sum(1)[:, None] * np.abs(lat) + 2.0 ** -16 * np.abs(lat)
        out[:, h] = lat @ w_uv[h].T
        e_out[:, h] = e_lat @ np.abs(w_uv[h]).T + \
            (d_c + 4) * F32 * (np.abs(lat) @ np.abs(w_uv[h]).T)
    return out, lse, e_out, e_lse
