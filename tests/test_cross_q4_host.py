"""Cross attention and the 4-bit ring on a machine without a GPU: the definitions that the GPU
tests compare with, and the refusals that the host makes before any launch."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from mla_latent_kv_attn_b200 import _lib, api, inputs


def _case(seed, B, n_q, n_kv, H, Hkv, d):
    r = np.random.default_rng(seed)
    return (r.standard_normal((B, n_q, H, d)), r.standard_normal((B, n_kv, Hkv, d)),
            r.standard_normal((B, n_kv, Hkv, d)), r.standard_normal((B, n_q, H, d)))


def test_gradients_match_differences():
    """Central differences of f = sum(g * out) along random directions: with step h the error is
    O(h^2 f''') ~ 1e-10 and the rounding 1e-16 |f| / h ~ 1e-10; 1e-7 relative leaves room."""
    q, k, v, g = _case(0, 2, 5, 7, 4, 2, 8)
    lens, scale = [7, 3], 0.3
    grads, _ = oracle.cross_attention_backward(q, k, v, lens, scale, g)
    f = lambda q, k, v: (g * oracle.cross_attention(q, k, v, lens, scale)[0]).sum()
    r = np.random.default_rng(1)
    for i, grad in enumerate(grads):
        t = [q, k, v]
        u = r.standard_normal(t[i].shape)
        h = 1e-5
        up, dn = list(t), list(t)
        up[i], dn[i] = t[i] + h * u, t[i] - h * u
        num = (f(*up) - f(*dn)) / (2 * h)
        assert abs(num - (grad * u).sum()) <= 1e-7 * max(1.0, abs(num))


def test_definition_matches_autograd_and_masks():
    q, k, v, g = _case(2, 2, 4, 6, 2, 1, 4)
    lens = [0, 5]
    out, lse, _, _ = oracle.cross_attention(q, k, v, lens, 0.5)
    assert (out[0] == 0).all() and np.isneginf(lse[0]).all()
    t = [torch.tensor(x, requires_grad=True) for x in (q, k, v)]
    kk, vv = (x[1, :5].expand(-1, 2, -1) for x in t[1:])
    p = torch.softmax(torch.einsum("ihd,jhd->hij", t[0][1], kk) * 0.5, -1)
    o = torch.einsum("hij,jhd->ihd", p, vv)
    assert np.abs(o.detach().numpy() - out[1]).max() < 1e-12
    (o * torch.tensor(g[1])).sum().backward()
    grads, _ = oracle.cross_attention_backward(q, k, v, lens, 0.5, g)
    for got, x in zip(grads, t):
        assert np.abs(got - x.grad.numpy()).max() < 1e-12


def test_q4_scales_are_the_least_that_hold_and_codes_the_nearest():
    r = np.random.default_rng(3)
    x = r.standard_normal((50, 64)) * 10.0 ** r.uniform(-5, 3, (50, 1))
    x = torch.tensor(x).to(torch.bfloat16).double().numpy()
    codes, scales = oracle.q4_encode(x)
    s = np.repeat(oracle.q4_scale(scales), 16, -1)
    y = oracle.q4_decode(codes, scales)
    assert (np.abs(x - y) <= s / 2).all()
    less = np.repeat(oracle.q4_scale(np.maximum(scales.astype(int) - 1, 0)), 16, -1)
    top = np.repeat(np.abs(x).reshape(50, 4, 16).max(-1), 16, -1)
    assert (top <= 7 * s).all() and (top[less < s] > 7 * less[less < s]).all()
    assert np.array_equal(torch.tensor(y).to(torch.bfloat16).double().numpy(), y)


def test_q4_edges():
    x = np.zeros((1, 32))
    codes, scales = oracle.q4_encode(x)
    assert (codes == 0x88).all() and (scales == 0).all()
    x[0, 3] = 1e9                                      # beyond the largest scale: saturates
    codes, scales = oracle.q4_encode(x)
    assert scales[0, 0] == 255 and oracle.q4_decode(codes, scales)[0, 3] == 7 * 3840
    assert oracle.q4_scale(255) == 3840 and oracle.q4_scale(0) == 2.0 ** -20
    x = np.full((1, 16), 1.75)                         # 1.75 / 7 is a scale itself
    assert oracle.q4_scale(oracle.q4_encode(x)[1])[0, 0] == 0.25


@pytest.mark.parametrize("field,value,status", [
    ("batch", 0, 1), ("n_heads", -1, 1), ("n_kv_heads", 5, 1), ("d_head", 0, 1),
    ("d_head", 257, 2), ("n_q", 0, 1), ("n_kv", 0, 1), ("softmax_scale", 0.0, 1),
    ("softmax_scale", float("nan"), 1), ("dtype", 2, 1), ("kernel_path", 2, 1),
    ("n_q", 2**30, 1), ("n_kv", 2**31 - 1, 1), ("batch", 70000, 1),
])
def test_bad_cross_configs_are_refused(field, value, status):
    cc = api.make_cross_config(batch=2, n_heads=12, d_head=128, n_q=100, n_kv=64)
    api.mla_cross_config_check(cc)
    assert api.mla_cross_attention_bwd_workspace_bytes(cc) > 0
    setattr(cc, field, value)
    with pytest.raises(api.MLAError) as e:
        api.mla_cross_config_check(cc)
    assert e.value.status == status and _lib.last_error()
    assert api.mla_cross_attention_bwd_workspace_bytes(cc) == 0
    st = _lib.lib().mla_cross_attention_fwd(ctypes.byref(cc), *[None, 0] * 3, *[None] * 5)
    assert st == status


def test_cross_strides_and_pointers_are_refused_on_the_host():
    cc = api.make_cross_config(batch=2, n_heads=4, d_head=16, n_q=8, n_kv=8)
    lib, ref = _lib.lib(), ctypes.byref(cc)
    for strides, status, word in (((63, 0, 0), 1, "row stride"), ((0, 65, 0), 3, "16 bytes"),
                                  ((0, 0, -64), 1, "row stride"), ((2**40, 0, 0), 1, "2^31"),
                                  ((0, 0, 0), 1, "null")):
        args = [a for s in strides for a in (None, s)]
        assert lib.mla_cross_attention_fwd(ref, *args, *[None] * 5) == status
        assert word in _lib.last_error()
        assert lib.mla_cross_attention_bwd(ref, *args, *[None] * 8, 0, None, None) == status
        assert word in _lib.last_error()


def test_cross_binding_checks_shapes_types_and_strides():
    cc = api.make_cross_config(batch=2, n_heads=4, d_head=16, n_q=8, n_kv=6)
    q = torch.zeros(2, 8, 4, 16, dtype=torch.bfloat16)
    k = torch.zeros(2, 6, 4, 16, dtype=torch.bfloat16)
    out = torch.zeros_like(q)
    call = lambda q=q, k=k, v=k, out=out, **kw: api.mla_cross_attention_fwd(cc, q, k, v, out, **kw)
    with pytest.raises(TypeError):
        call(q=q.float())
    with pytest.raises(ValueError):
        call(k=k[:, :5])
    with pytest.raises(ValueError):
        call(q=q.transpose(1, 2).contiguous().transpose(1, 2))      # heads not dense
    with pytest.raises(ValueError):
        call(k=torch.zeros(2, 7, 4, 16, dtype=torch.bfloat16)[:, :6])   # a gap between samples
    with pytest.raises(ValueError):
        call(k=k[:1].expand(2, -1, -1, -1))                         # samples share rows
    with pytest.raises(ValueError):
        call(out=torch.zeros(2, 8, 8, 16, dtype=torch.bfloat16)[:, :, ::2])
    with pytest.raises(TypeError):
        call(kv_len=torch.zeros(2, dtype=torch.int64))
    wide = torch.zeros(2, 6, 3, 4, 16, dtype=torch.bfloat16)
    assert api._rows(wide[:, :, 1], "k", torch.bfloat16, (2, 6, 4, 16)) == (wide[:, :, 1].data_ptr(),
                                                                            192)
    one = torch.zeros(2, 1, 3, 4, 16, dtype=torch.bfloat16)[:, :, 2]
    assert api._rows(one, "k", torch.bfloat16, (2, 1, 4, 16))[1] == 192


def test_q4_refusals_without_a_device():
    lib = _lib.lib()
    toy = api.make_config(inputs.CONFIGS[0])                        # d_rope 8: half a group
    st = lib.mla_cache_append_q4(ctypes.byref(toy), *[None] * 4, 0, None)
    assert st == _lib.MLA_ERR_UNSUPPORTED and "multiples of 16" in _lib.last_error()
    assert lib.mla_cache_read_q4(ctypes.byref(toy), *[None] * 4) == _lib.MLA_ERR_UNSUPPORTED
    c = api.make_config(inputs.CONFIGS[1])
    ref = ctypes.byref(c)
    assert lib.mla_cache_append_q4(ref, *[None] * 4, -1, None) == 1
    assert "first_frame" in _lib.last_error()
    assert lib.mla_cache_append_q4(ref, *[None] * 4, 0, None) == 1 and "null" in _lib.last_error()
    args = [None] * 5 + [7, 0] + [None] * 4 + [0, None, None]
    assert lib.mla_attention_fwd_q4(ref, *args) == 1 and "n_valid" in _lib.last_error()
    wide = api.make_config(inputs.with_latent_shape(inputs.CONFIGS[1], 256, 32))
    args = [None] * 6 + [0, 0] + [None] * 4 + [0, None, None]
    assert lib.mla_attention_fwd_from_cq_q4(ctypes.byref(wide), *args) == _lib.MLA_ERR_UNSUPPORTED
    assert api.mla_attention_q4_workspace_bytes(c, 7) == 0
    # the rotated keys as for a bf16 ring, and the contents of slots and chunk in 16 bits
    tpf, D, d_c = 1560, 224, 192
    keys = -(-api.mla_attention_workspace_bytes(c, 6) // 256) * 256
    assert api.mla_attention_q4_workspace_bytes(c, 6) == keys + (6 + 3) * tpf * d_c * 2
    # CUDA cores: the slots' values beside the caller's chunk
    simt = api.make_config(inputs.CONFIGS[1], kernel_path=api.MLA_PATH_SIMT)
    assert api.mla_attention_q4_workspace_bytes(simt, 6) == keys + 6 * tpf * D * 2
