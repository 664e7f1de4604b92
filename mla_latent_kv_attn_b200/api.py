"""Python binding of the C ABI: the same entry points, taking torch tensors.

Every function here only marshals arguments (shape/dtype checks, raw device pointers, the
current CUDA stream) and calls the library; all arithmetic runs in the CUDA kernels.  A non-zero
status raises MLAError with the library's message.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Tuple

import torch

from . import _lib
from ._lib import (MLA_APPEND, MLA_BF16, MLA_FP32, MLA_PATH_AUTO, MLA_PATH_SIMT,
                   MLA_PATH_TC_PAIR, MLA_PATH_TC_SINGLE, MLA_PROJECT, MLA_PROJECT_AND_APPEND, MLAConfigC,
                   MLACrossConfigC, MLAError)

__all__ = [
    "make_config", "torch_dtype", "mla_config_check", "mla_cache_append", "mla_rope3d",
    "mla_key_positions", "mla_compose_query_weights", "mla_query_proj", "mla_project_chunk",
    "mla_attention_workspace_bytes", "mla_attention_fwd", "mla_attention_fwd_static_scratch",
    "mla_project_latents", "mla_project_latents_rotated", "mla_attention_fwd_from_cq",
    "mla_rotate_ring_keys", "mla_attention_fwd_cached_ring", "mla_attention_uses_tensor_cores",
    "mla_attention_bwd_workspace_bytes", "mla_attention_bwd",
    "mla_out_proj", "mla_cache_append_q4", "mla_cache_read_q4", "mla_attention_q4_workspace_bytes",
    "mla_attention_fwd_q4", "mla_attention_fwd_from_cq_q4", "make_cross_config",
    "mla_cross_config_check", "mla_cross_attention_fwd", "mla_cross_attention_bwd_workspace_bytes",
    "mla_cross_attention_bwd", "MLAError",
    "MLA_PROJECT", "MLA_APPEND", "MLA_PROJECT_AND_APPEND", "MLA_PATH_AUTO", "MLA_PATH_SIMT",
    "MLA_PATH_TC_SINGLE", "MLA_PATH_TC_PAIR",
]


def make_config(cfg, kernel_path: int = MLA_PATH_AUTO, batch: Optional[int] = None) -> MLAConfigC:
    """struct mla_config from a workload preset (mla_latent_kv_attn_b200.inputs.MLAConfig)."""
    pt, ph, pw = cfg.rope_pairs
    return MLAConfigC(
        d_model=cfg.d_model, n_heads=cfg.n_heads, d_head=cfg.d_head, d_c=cfg.d_c,
        d_rope=cfg.d_rope, d_cq=cfg.d_cq, rope_pairs_t=pt, rope_pairs_h=ph, rope_pairs_w=pw,
        rope_base=cfg.rope_base, softmax_scale=cfg.softmax_scale, frame_h=cfg.frame_h,
        frame_w=cfg.frame_w, chunk_frames=cfg.chunk_frames, window_frames=cfg.window_frames,
        batch=cfg.batch if batch is None else batch,
        dtype=MLA_FP32 if cfg.dtype == "fp32" else MLA_BF16, kernel_path=kernel_path)


def torch_dtype(c: MLAConfigC) -> torch.dtype:
    return torch.float32 if c.dtype == MLA_FP32 else torch.bfloat16


def _ptr(t: Optional[torch.Tensor], name: str, dtype=None, shape=None) -> Optional[int]:
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if (shape is None or t.shape == shape) and (dtype is None or t.dtype is dtype) and \
            t.is_contiguous():
        return t.data_ptr()
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        # The handle of torch.cuda.current_stream(), whose Python object costs 4 us a call, as much
        # as the smallest launches.  Before CUDA is initialised there is only the default stream.
        if not torch.cuda.is_initialized():
            return None
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _geom(c: MLAConfigC):
    tpf = c.frame_h * c.frame_w
    return tpf, c.chunk_frames * tpf, c.d_c + c.d_rope


def mla_config_check(c: MLAConfigC) -> None:
    _lib.check("mla_config_check", _lib.lib().mla_config_check(ctypes.byref(c)))


def mla_cache_append(c: MLAConfigC, x, w_dkv_kr, chunk_lat, cache, slot_frame, first_frame: int,
                     mode: int, stream=None) -> None:
    tpf, n_q, D = _geom(c)
    dt = torch_dtype(c)
    B = c.batch
    st = _lib.lib().mla_cache_append(
        ctypes.byref(c), _ptr(x, "x", dt, (B, n_q, c.d_model)),
        _ptr(w_dkv_kr, "w_dkv_kr", dt, (D, c.d_model)), _ptr(chunk_lat, "chunk_lat", dt, (B, n_q, D)),
        _ptr(cache, "cache", dt, (B, c.window_frames * tpf, D)),
        _ptr(slot_frame, "slot_frame", torch.int32, (B, c.window_frames)), first_frame, mode,
        _stream(stream))
    _lib.check("mla_cache_append", st)


def mla_rope3d(c: MLAConfigC, data, n_vec: int, col_offset: int, vec_stride: int,
               frame_table=None, first_frame: int = 0, stream=None) -> None:
    """Rotates data [n_samples, rows, row_width] in place (see include/mla.h)."""
    if data.dim() != 3:
        raise ValueError("data must be [n_samples, rows, row_width]")
    n_s, rows, width = data.shape
    fstride = frame_table.shape[1] if frame_table is not None else 0
    st = _lib.lib().mla_rope3d(
        ctypes.byref(c), _ptr(data, "data", torch_dtype(c)), n_s, rows, width, col_offset, n_vec,
        vec_stride, _ptr(frame_table, "frame_table", torch.int32), fstride, first_frame,
        _stream(stream))
    _lib.check("mla_rope3d", st)


def mla_key_positions(c: MLAConfigC, slot_frame, n_valid_frames: int, first_frame: int,
                      pos_out, stream=None) -> None:
    tpf, n_q, _ = _geom(c)
    n_keys = n_valid_frames * tpf + n_q
    st = _lib.lib().mla_key_positions(
        ctypes.byref(c), _ptr(slot_frame, "slot_frame", torch.int32, (c.batch, c.window_frames)),
        n_valid_frames, first_frame, _ptr(pos_out, "pos_out", torch.int32, (c.batch, n_keys, 3)),
        _stream(stream))
    _lib.check("mla_key_positions", st)


def mla_compose_query_weights(c: MLAConfigC, w_uq, w_uk, w_qr, w_qcat, stream=None) -> None:
    dt = torch_dtype(c)
    H, D = c.n_heads, c.d_c + c.d_rope
    st = _lib.lib().mla_compose_query_weights(
        ctypes.byref(c), _ptr(w_uq, "w_uq", dt, (H, c.d_head, c.d_cq)),
        _ptr(w_uk, "w_uk", dt, (H, c.d_head, c.d_c)), _ptr(w_qr, "w_qr", dt, (H, c.d_rope, c.d_cq)),
        _ptr(w_qcat, "w_qcat", dt, (H, D, c.d_cq)), _stream(stream))
    _lib.check("mla_compose_query_weights", st)


def mla_query_proj(c: MLAConfigC, x, w_dq, w_qcat, c_q, q, first_frame: int, stream=None) -> None:
    tpf, n_q, D = _geom(c)
    dt = torch_dtype(c)
    B, H = c.batch, c.n_heads
    st = _lib.lib().mla_query_proj(
        ctypes.byref(c), _ptr(x, "x", dt, (B, n_q, c.d_model)),
        _ptr(w_dq, "w_dq", dt, (c.d_cq, c.d_model)), _ptr(w_qcat, "w_qcat", dt, (H, D, c.d_cq)),
        _ptr(c_q, "c_q", dt, (B, n_q, c.d_cq)), _ptr(q, "q", dt, (B, n_q, H, D)), first_frame,
        _stream(stream))
    _lib.check("mla_query_proj", st)


def mla_project_chunk(c: MLAConfigC, x, w_x, w_qcat, c_q, q, chunk_lat, first_frame: int,
                      stream=None) -> None:
    tpf, n_q, D = _geom(c)
    dt = torch_dtype(c)
    B, H = c.batch, c.n_heads
    st = _lib.lib().mla_project_chunk(
        ctypes.byref(c), _ptr(x, "x", dt, (B, n_q, c.d_model)),
        _ptr(w_x, "w_x", dt, (c.d_cq + D, c.d_model)), _ptr(w_qcat, "w_qcat", dt, (H, D, c.d_cq)),
        _ptr(c_q, "c_q", dt, (B, n_q, c.d_cq)), _ptr(q, "q", dt, (B, n_q, H, D)),
        _ptr(chunk_lat, "chunk_lat", dt, (B, n_q, D)), first_frame, _stream(stream))
    _lib.check("mla_project_chunk", st)


def mla_project_latents(c: MLAConfigC, x, w_x, c_q, chunk_lat, stream=None) -> None:
    tpf, n_q, D = _geom(c)
    dt = torch_dtype(c)
    B = c.batch
    st = _lib.lib().mla_project_latents(
        ctypes.byref(c), _ptr(x, "x", dt, (B, n_q, c.d_model)),
        _ptr(w_x, "w_x", dt, (c.d_cq + D, c.d_model)), _ptr(c_q, "c_q", dt, (B, n_q, c.d_cq)),
        _ptr(chunk_lat, "chunk_lat", dt, (B, n_q, D)), _stream(stream))
    _lib.check("mla_project_latents", st)


def mla_project_latents_rotated(c: MLAConfigC, x, w_x, c_q, chunk_lat, cache, slot_frame,
                                n_valid_frames: int, first_frame: int, workspace,
                                rotate_ring: bool = True, dev_status=None, stream=None) -> None:
    """mla_project_latents that also writes the chunk attention's rotated positional keys into
    `workspace` (the ring's too with rotate_ring), for mla_attention_fwd_from_cq(...,
    prerotated=True)."""
    tpf, n_q, D = _geom(c)
    dt = torch_dtype(c)
    B = c.batch
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = _lib.lib().mla_project_latents_rotated(
        ctypes.byref(c), _ptr(x, "x", dt, (B, n_q, c.d_model)),
        _ptr(w_x, "w_x", dt, (c.d_cq + D, c.d_model)), _ptr(c_q, "c_q", dt, (B, n_q, c.d_cq)),
        _ptr(chunk_lat, "chunk_lat", dt, (B, n_q, D)),
        _ptr(cache, "cache", dt, (B, c.window_frames * tpf, D)),
        _ptr(slot_frame, "slot_frame", torch.int32, (B, c.window_frames)), n_valid_frames,
        first_frame, 1 if rotate_ring else 0, _ptr(workspace, "workspace"), ws_bytes,
        _ptr(dev_status, "dev_status", torch.int32), _stream(stream))
    _lib.check("mla_project_latents_rotated", st)


def mla_attention_uses_tensor_cores(c: MLAConfigC, with_w_uv: bool = True) -> bool:
    r = int(_lib.lib().mla_attention_uses_tensor_cores(ctypes.byref(c), 1 if with_w_uv else 0))
    if r < 0:
        raise MLAError("mla_attention_uses_tensor_cores", _lib.MLA_ERR_INVALID_ARG, _lib.last_error())
    return bool(r)


def mla_attention_workspace_bytes(c: MLAConfigC, n_valid_frames: int) -> int:
    return int(_lib.lib().mla_attention_workspace_bytes(ctypes.byref(c), n_valid_frames))


def _attention(fn_name: str, c: MLAConfigC, q, chunk_lat, cache, slot_frame, n_valid_frames: int,
               first_frame: int, w_uv, out, lse, workspace, dev_status, stream) -> None:
    tpf, n_q, D = _geom(c)
    dt = torch_dtype(c)
    B, H = c.batch, c.n_heads
    out_shape = (B, n_q, H * c.d_head) if w_uv is not None else (B, n_q, H, c.d_c)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = getattr(_lib.lib(), fn_name)(
        ctypes.byref(c), _ptr(q, "q", dt, (B, n_q, H, D)), _ptr(chunk_lat, "chunk_lat", dt, (B, n_q, D)),
        _ptr(cache, "cache", dt, (B, c.window_frames * tpf, D)),
        _ptr(slot_frame, "slot_frame", torch.int32, (B, c.window_frames)), n_valid_frames,
        first_frame, _ptr(w_uv, "w_uv", dt, (H, c.d_head, c.d_c)), _ptr(out, "out", dt, out_shape),
        _ptr(lse, "lse", torch.float32, (B, H, n_q)), _ptr(workspace, "workspace"), ws_bytes,
        _ptr(dev_status, "dev_status", torch.int32), _stream(stream))
    _lib.check(fn_name, st)


def mla_attention_fwd(c: MLAConfigC, q, chunk_lat, cache, slot_frame, n_valid_frames: int,
                      first_frame: int, w_uv, out, lse=None, workspace=None, dev_status=None,
                      stream=None) -> None:
    _attention("mla_attention_fwd", c, q, chunk_lat, cache, slot_frame, n_valid_frames,
               first_frame, w_uv, out, lse, workspace, dev_status, stream)


def mla_attention_fwd_from_cq(c: MLAConfigC, c_q, w_qcat, chunk_lat, cache, slot_frame,
                              n_valid_frames: int, first_frame: int, w_uv, out, lse=None,
                              workspace=None, dev_status=None, stream=None,
                              cached_ring: bool = False, prerotated: bool = False) -> None:
    """mla_attention_fwd with the query heads (and their 3D-RoPE) formed inside the attention
    kernel from the query latent c_q and the composed weights w_qcat.  cached_ring: the
    workspace already holds the ring's rotated keys (mla_rotate_ring_keys); prerotated: it holds
    every rotated key of the call (mla_project_latents_rotated), so no rotation pass runs."""
    if cached_ring and prerotated:
        raise ValueError("cached_ring and prerotated are exclusive")
    fn = ("mla_attention_fwd_from_cq_prerotated" if prerotated else
          "mla_attention_fwd_from_cq_cached_ring" if cached_ring else "mla_attention_fwd_from_cq")
    tpf, n_q, D = _geom(c)
    dt = torch_dtype(c)
    B, H = c.batch, c.n_heads
    out_shape = (B, n_q, H * c.d_head) if w_uv is not None else (B, n_q, H, c.d_c)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = getattr(_lib.lib(), fn)(
        ctypes.byref(c), _ptr(c_q, "c_q", dt, (B, n_q, c.d_cq)),
        _ptr(w_qcat, "w_qcat", dt, (H, D, c.d_cq)), _ptr(chunk_lat, "chunk_lat", dt, (B, n_q, D)),
        _ptr(cache, "cache", dt, (B, c.window_frames * tpf, D)),
        _ptr(slot_frame, "slot_frame", torch.int32, (B, c.window_frames)), n_valid_frames,
        first_frame, _ptr(w_uv, "w_uv", dt, (H, c.d_head, c.d_c)), _ptr(out, "out", dt, out_shape),
        _ptr(lse, "lse", torch.float32, (B, H, n_q)), _ptr(workspace, "workspace"), ws_bytes,
        _ptr(dev_status, "dev_status", torch.int32), _stream(stream))
    _lib.check(fn, st)


def mla_attention_fwd_cached_ring(c: MLAConfigC, q, chunk_lat, cache, slot_frame,
                                  n_valid_frames: int, first_frame: int, w_uv, out, lse=None,
                                  workspace=None, dev_status=None, stream=None) -> None:
    """mla_attention_fwd for a workspace whose ring part mla_rotate_ring_keys has filled for the
    same (unchanged) ring; only the chunk's positional keys are rotated."""
    _attention("mla_attention_fwd_cached_ring", c, q, chunk_lat, cache, slot_frame,
               n_valid_frames, first_frame, w_uv, out, lse, workspace, dev_status, stream)


def mla_rotate_ring_keys(c: MLAConfigC, cache, slot_frame, n_valid_frames: int, workspace,
                         stream=None) -> None:
    tpf, n_q, D = _geom(c)
    dt = torch_dtype(c)
    B = c.batch
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = _lib.lib().mla_rotate_ring_keys(
        ctypes.byref(c), _ptr(cache, "cache", dt, (B, c.window_frames * tpf, D)),
        _ptr(slot_frame, "slot_frame", torch.int32, (B, c.window_frames)), n_valid_frames,
        _ptr(workspace, "workspace"), ws_bytes, _stream(stream))
    _lib.check("mla_rotate_ring_keys", st)


def mla_attention_bwd_workspace_bytes(c: MLAConfigC, n_valid_frames: int) -> int:
    return int(_lib.lib().mla_attention_bwd_workspace_bytes(ctypes.byref(c), n_valid_frames))


def mla_attention_bwd(c: MLAConfigC, q, chunk_lat, cache, slot_frame, n_valid_frames: int,
                      first_frame: int, o_lat, lse, d_o_lat, d_q, d_chunk_lat, d_cache, workspace,
                      dev_status=None, stream=None) -> None:
    """Gradients of the latent attention call (see include/mla.h)."""
    tpf, n_q, D = _geom(c)
    dt = torch_dtype(c)
    B, H = c.batch, c.n_heads
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = _lib.lib().mla_attention_bwd(
        ctypes.byref(c), _ptr(q, "q", dt, (B, n_q, H, D)), _ptr(chunk_lat, "chunk_lat", dt, (B, n_q, D)),
        _ptr(cache, "cache", dt, (B, c.window_frames * tpf, D)),
        _ptr(slot_frame, "slot_frame", torch.int32, (B, c.window_frames)), n_valid_frames,
        first_frame, _ptr(o_lat, "o_lat", dt, (B, n_q, H, c.d_c)),
        _ptr(lse, "lse", torch.float32, (B, H, n_q)), _ptr(d_o_lat, "d_o_lat", dt, (B, n_q, H, c.d_c)),
        _ptr(d_q, "d_q", dt, (B, n_q, H, D)), _ptr(d_chunk_lat, "d_chunk_lat", dt, (B, n_q, D)),
        _ptr(d_cache, "d_cache", dt, (B, c.window_frames * tpf, D)), _ptr(workspace, "workspace"),
        ws_bytes, _ptr(dev_status, "dev_status", torch.int32), _stream(stream))
    _lib.check("mla_attention_bwd", st)


def mla_out_proj(c: MLAConfigC, o_lat, w_uv, o, w_o=None, y=None, stream=None) -> None:
    tpf, n_q, D = _geom(c)
    dt = torch_dtype(c)
    B, H = c.batch, c.n_heads
    st = _lib.lib().mla_out_proj(
        ctypes.byref(c), _ptr(o_lat, "o_lat", dt, (B, n_q, H, c.d_c)),
        _ptr(w_uv, "w_uv", dt, (H, c.d_head, c.d_c)), _ptr(w_o, "w_o", dt, (c.d_model, H * c.d_head)),
        _ptr(o, "o", dt, (B, n_q, H * c.d_head)), _ptr(y, "y", dt, (B, n_q, c.d_model)),
        _stream(stream))
    _lib.check("mla_out_proj", st)


def mla_attention_fwd_static_scratch(c: MLAConfigC, q, chunk_lat, cache, slot_frame,
                                     n_valid_frames: int, first_frame: int, w_uv, out, lse=None,
                                     dev_status=None, stream=None) -> None:
    """mla_attention_fwd for callers that cannot allocate: the scratch lives in the library's
    built-in 16 MiB device array (one per device, shared by all calls; order calls on one
    stream).  The first call on a device should come before any stream capture."""
    tpf, n_q, D = _geom(c)
    dt = torch_dtype(c)
    B, H = c.batch, c.n_heads
    out_shape = (B, n_q, H * c.d_head) if w_uv is not None else (B, n_q, H, c.d_c)
    st = _lib.lib().mla_attention_fwd_static_scratch(
        ctypes.byref(c), _ptr(q, "q", dt, (B, n_q, H, D)), _ptr(chunk_lat, "chunk_lat", dt, (B, n_q, D)),
        _ptr(cache, "cache", dt, (B, c.window_frames * tpf, D)),
        _ptr(slot_frame, "slot_frame", torch.int32, (B, c.window_frames)), n_valid_frames,
        first_frame, _ptr(w_uv, "w_uv", dt, (H, c.d_head, c.d_c)), _ptr(out, "out", dt, out_shape),
        _ptr(lse, "lse", torch.float32, (B, H, n_q)), _ptr(dev_status, "dev_status", torch.int32),
        _stream(stream))
    _lib.check("mla_attention_fwd_static_scratch", st)


# ---- the latent ring held in 4 bits -----------------------------------------------------------


def _q4_ring(codes, scales, B: int, rows: int, D: int):
    return (_ptr(codes, "codes", torch.uint8, (B, rows, D // 2)),
            _ptr(scales, "scales", torch.uint8, (B, rows, D // 16)))


def mla_cache_append_q4(c: MLAConfigC, chunk_lat, codes, scales, slot_frame, first_frame: int,
                        stream=None) -> None:
    tpf, n_q, D = _geom(c)
    B, W = c.batch, c.window_frames
    st = _lib.lib().mla_cache_append_q4(
        ctypes.byref(c), _ptr(chunk_lat, "chunk_lat", torch_dtype(c), (B, n_q, D)),
        *_q4_ring(codes, scales, B, W * tpf, D),
        _ptr(slot_frame, "slot_frame", torch.int32, (B, W)), first_frame, _stream(stream))
    if st:
        _lib.check("mla_cache_append_q4", st)


def mla_cache_read_q4(c: MLAConfigC, codes, scales, cache, stream=None) -> None:
    tpf, _, D = _geom(c)
    B, rows = c.batch, c.window_frames * tpf
    st = _lib.lib().mla_cache_read_q4(
        ctypes.byref(c), *_q4_ring(codes, scales, B, rows, D),
        _ptr(cache, "cache", torch_dtype(c), (B, rows, D)), _stream(stream))
    if st:
        _lib.check("mla_cache_read_q4", st)


def mla_attention_q4_workspace_bytes(c: MLAConfigC, n_valid_frames: int) -> int:
    return int(_lib.lib().mla_attention_q4_workspace_bytes(ctypes.byref(c), n_valid_frames))


def _attention_q4(fn_name: str, c: MLAConfigC, query, chunk_lat, codes, scales, slot_frame,
                  n_valid_frames: int, first_frame: int, w_uv, out, lse, workspace, dev_status,
                  stream) -> None:
    tpf, n_q, D = _geom(c)
    dt = torch_dtype(c)
    B, H = c.batch, c.n_heads
    out_shape = (B, n_q, H * c.d_head) if w_uv is not None else (B, n_q, H, c.d_c)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = getattr(_lib.lib(), fn_name)(
        ctypes.byref(c), *query, _ptr(chunk_lat, "chunk_lat", dt, (B, n_q, D)),
        *_q4_ring(codes, scales, B, c.window_frames * tpf, D),
        _ptr(slot_frame, "slot_frame", torch.int32, (B, c.window_frames)), n_valid_frames,
        first_frame, _ptr(w_uv, "w_uv", dt, (H, c.d_head, c.d_c)), _ptr(out, "out", dt, out_shape),
        _ptr(lse, "lse", torch.float32, (B, H, n_q)), _ptr(workspace, "workspace"), ws_bytes,
        _ptr(dev_status, "dev_status", torch.int32), _stream(stream))
    _lib.check(fn_name, st)


def mla_attention_fwd_q4(c: MLAConfigC, q, chunk_lat, codes, scales, slot_frame,
                         n_valid_frames: int, first_frame: int, w_uv, out, lse=None,
                         workspace=None, dev_status=None, stream=None) -> None:
    """mla_attention_fwd over a ring held in 4 bits."""
    _, n_q, D = _geom(c)
    query = (_ptr(q, "q", torch_dtype(c), (c.batch, n_q, c.n_heads, D)),)
    _attention_q4("mla_attention_fwd_q4", c, query, chunk_lat, codes, scales, slot_frame,
                  n_valid_frames, first_frame, w_uv, out, lse, workspace, dev_status, stream)


def mla_attention_fwd_from_cq_q4(c: MLAConfigC, c_q, w_qcat, chunk_lat, codes, scales, slot_frame,
                                 n_valid_frames: int, first_frame: int, w_uv, out, lse=None,
                                 workspace=None, dev_status=None, stream=None) -> None:
    """mla_attention_fwd_from_cq over a ring held in 4 bits."""
    _, n_q, D = _geom(c)
    dt = torch_dtype(c)
    query = (_ptr(c_q, "c_q", dt, (c.batch, n_q, c.d_cq)),
             _ptr(w_qcat, "w_qcat", dt, (c.n_heads, D, c.d_cq)))
    _attention_q4("mla_attention_fwd_from_cq_q4", c, query, chunk_lat, codes, scales, slot_frame,
                  n_valid_frames, first_frame, w_uv, out, lse, workspace, dev_status, stream)


# ---- cross attention to an encoder's states ---------------------------------------------------


def make_cross_config(batch: int, n_heads: int, d_head: int, n_q: int, n_kv: int,
                      n_kv_heads: Optional[int] = None, softmax_scale: Optional[float] = None,
                      dtype: str = "bf16", kernel_path: int = MLA_PATH_AUTO) -> MLACrossConfigC:
    """struct mla_cross_config; softmax_scale defaults to 1/sqrt(d_head), n_kv_heads to n_heads."""
    if dtype not in ("bf16", "fp32"):
        raise ValueError(f"unknown dtype {dtype!r}")
    return MLACrossConfigC(
        batch=batch, n_heads=n_heads, n_kv_heads=n_heads if n_kv_heads is None else n_kv_heads,
        d_head=d_head, n_q=n_q, n_kv=n_kv,
        softmax_scale=1.0 / math.sqrt(d_head) if softmax_scale is None else softmax_scale,
        dtype=MLA_FP32 if dtype == "fp32" else MLA_BF16, kernel_path=kernel_path)


def mla_cross_config_check(cc: MLACrossConfigC) -> None:
    _lib.check("mla_cross_config_check", _lib.lib().mla_cross_config_check(ctypes.byref(cc)))


def _rows(t: torch.Tensor, name: str, dtype, shape) -> Tuple[int, int]:
    """Pointer and row stride of a [B, n, H, d] tensor whose tokens' heads are dense and whose
    samples' tokens follow one another (a dense tensor, or part of the rows of one)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.is_contiguous():
        return t.data_ptr(), 0
    B, n, H, d = shape
    sb, sn, sh, sd = t.stride()
    row = sn if n > 1 else sb if B > 1 else H * d      # (the stride of a dimension of 1 says nothing)
    if (d > 1 and sd != 1) or (H > 1 and sh != d) or (B > 1 and sb != n * row) or row < H * d:
        raise ValueError(f"{name} must have dense heads and tokens at one stride: got strides "
                         f"{t.stride()} for shape {tuple(t.shape)}")
    return t.data_ptr(), row


def _cross_inputs(cc: MLACrossConfigC, q, k, v, kv_len):
    """The calls' common arguments, then T and the shapes of q and of k (each field of cc is read
    once: a ctypes field costs as much as a tensor's shape)."""
    dt = torch.float32 if cc.dtype == MLA_FP32 else torch.bfloat16
    B, d = cc.batch, cc.d_head
    rows, kv = (B, cc.n_q, cc.n_heads, d), (B, cc.n_kv, cc.n_kv_heads, d)
    return (*_rows(q, "q", dt, rows), *_rows(k, "k", dt, kv), *_rows(v, "v", dt, kv),
            _ptr(kv_len, "kv_len", torch.int32, (B,))), dt, rows, kv


def mla_cross_attention_fwd(cc: MLACrossConfigC, q, k, v, out, lse=None, kv_len=None,
                            dev_status=None, stream=None) -> None:
    """Attention of q [B, n_q, H, d] to the first kv_len[b] of an encoder's states k, v
    [B, n_kv, H_kv, d].  q, k and v may be parts of wider rows (see include/mla.h)."""
    inputs, dt, rows, _ = _cross_inputs(cc, q, k, v, kv_len)
    B, n_q, H, _ = rows
    st = _lib.lib().mla_cross_attention_fwd(
        ctypes.byref(cc), *inputs, _ptr(out, "out", dt, rows),
        _ptr(lse, "lse", torch.float32, (B, H, n_q)), _ptr(dev_status, "dev_status", torch.int32),
        _stream(stream))
    if st:
        _lib.check("mla_cross_attention_fwd", st)


def mla_cross_attention_bwd_workspace_bytes(cc: MLACrossConfigC) -> int:
    return int(_lib.lib().mla_cross_attention_bwd_workspace_bytes(ctypes.byref(cc)))


def mla_cross_attention_bwd(cc: MLACrossConfigC, q, k, v, out, lse, d_out, d_q, d_k, d_v,
                            workspace, kv_len=None, dev_status=None, stream=None) -> None:
    """Gradients of mla_cross_attention_fwd, given its out and lse (see include/mla.h)."""
    inputs, dt, rows, kv = _cross_inputs(cc, q, k, v, kv_len)
    B, n_q, H, _ = rows
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = _lib.lib().mla_cross_attention_bwd(
        ctypes.byref(cc), *inputs, _ptr(out, "out", dt, rows),
        _ptr(lse, "lse", torch.float32, (B, H, n_q)), _ptr(d_out, "d_out", dt, rows),
        _ptr(d_q, "d_q", dt, rows), _ptr(d_k, "d_k", dt, kv), _ptr(d_v, "d_v", dt, kv),
        _ptr(workspace, "workspace"), ws_bytes, _ptr(dev_status, "dev_status", torch.int32),
        _stream(stream))
    if st:
        _lib.check("mla_cross_attention_bwd", st)
