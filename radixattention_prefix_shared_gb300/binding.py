"""Thin ctypes binding of libsgl_attn.so (names follow the C ABI).

Argument marshalling only: every step runs in the library's CUDA kernels.
Tensors are torch CUDA tensors (PyTorch provides device memory and streams);
bf16 tensors are ``torch.bfloat16``, indices ``torch.int32``.  A call that
the library rejects raises ``SglError``.  If the library is missing it is
built from source with nvcc; if that is impossible the import fails loudly --
there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import functools
import os

from . import build as _build

c_i32, c_i64, c_f32, c_size, c_vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t, ctypes.c_void_p

STATUS = {0: "SGL_OK", 1: "SGL_ERR_INVALID_ARG", 2: "SGL_ERR_UNSUPPORTED", 3: "SGL_ERR_WORKSPACE",
          4: "SGL_ERR_CUDA", 5: "SGL_ERR_INDEX"}


class SglError(RuntimeError):
    def __init__(self, func: str, code: int):
        super().__init__(f"{func} failed: {STATUS.get(code, code)}")
        self.code = code


class sgl_attn_dims(ctypes.Structure):
    _fields_ = [("num_q_heads", c_i32), ("num_kv_heads", c_i32), ("head_dim", c_i32),
                ("pool_size", c_i64), ("sm_scale", c_f32)]


_P = ctypes.POINTER
_SIGS = {
    "sgl_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "sgl_version": (ctypes.c_char_p, []),
    "sgl_set_device_wait_limit_ns": (ctypes.c_uint64, [ctypes.c_uint64]),
    "sgl_store_kv": (ctypes.c_int, [c_vp, c_vp, c_vp, c_i32, c_vp, c_vp, _P(sgl_attn_dims), c_vp]),
    "sgl_extend_attention": (ctypes.c_int, [c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_i32, c_i32, c_vp, c_vp,
                                            c_vp, c_i32, c_i32, c_i32, c_i32, c_vp, c_vp, c_size,
                                            _P(sgl_attn_dims), c_vp]),
    "sgl_decode_attention": (ctypes.c_int, [c_vp, c_vp, c_vp, c_vp, c_i32, c_i32, c_vp, c_vp, c_i32,
                                            c_i32, c_vp, c_vp, c_size, _P(sgl_attn_dims), c_vp]),
    "sgl_decode_attention_noalloc": (ctypes.c_int, [c_vp, c_vp, c_vp, c_vp, c_i32, c_i32, c_vp, c_vp, c_i32,
                                                    c_i32, c_vp, _P(sgl_attn_dims), c_vp]),
    "sgl_mixed_attention": (ctypes.c_int, [c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_i32, c_i32, c_i32, c_i32,
                                           c_vp, c_vp, c_size, c_vp, c_vp, c_vp, c_i32, c_i32, c_vp, c_vp,
                                           c_size, c_vp, c_vp, c_vp, c_i32, c_i32, c_i32, _P(sgl_attn_dims),
                                           c_vp]),
    "sgl_extend_workspace_bytes": (c_size, [c_i32, c_i32, _P(sgl_attn_dims)]),
    "sgl_decode_workspace_bytes": (c_size, [c_i32, c_i32, _P(sgl_attn_dims)]),
    "sgl_check_store_kv_indices": (ctypes.c_int, [c_vp, c_i32, c_i64, c_vp, c_size, c_vp, c_vp]),
    "sgl_check_extend_indices": (ctypes.c_int, [c_vp, c_i32, c_i32, c_vp, c_vp, c_vp, c_i32, c_i32, c_i32,
                                                c_i32, c_i64, c_vp, c_vp]),
    "sgl_check_decode_indices": (ctypes.c_int, [c_vp, c_i32, c_i32, c_vp, c_vp, c_i32, c_i32, c_i64,
                                                c_vp, c_vp]),
    "sgl_cascade_decode_attention": (ctypes.c_int, [c_vp, c_vp, c_vp, c_vp, c_i32, c_i32, c_vp, c_vp,
                                                    c_i32, c_i32, c_vp, c_vp, c_vp, c_vp, c_vp, c_i32,
                                                    c_i32, c_i32, c_vp, c_vp, c_size, _P(sgl_attn_dims),
                                                    c_vp]),
    "sgl_cascade_decode_workspace_bytes": (c_size, [c_i32, c_i32, c_i32, _P(sgl_attn_dims)]),
    "sgl_radix_create": (c_vp, []),
    "sgl_radix_destroy": (None, [c_vp]),
    "sgl_radix_match_prefix": (c_i32, [c_vp, c_vp, c_i32, c_vp, c_i32, _P(c_i64)]),
    "sgl_radix_insert": (c_i32, [c_vp, c_vp, c_vp, c_i32]),
    "sgl_radix_inc_lock_ref": (ctypes.c_int, [c_vp, c_i64]),
    "sgl_radix_dec_lock_ref": (ctypes.c_int, [c_vp, c_i64]),
    "sgl_radix_evict": (c_i32, [c_vp, c_i32, c_vp, c_i32]),
    "sgl_radix_evictable_tokens": (c_i64, [c_vp]),
    "sgl_radix_protected_tokens": (c_i64, [c_vp]),
    "sgl_radix_groups": (c_i32, [c_vp, c_vp, c_i32, c_vp, c_vp, c_vp, c_vp, c_vp, c_i32, c_i32, _P(c_i32)]),
    "sgl_store_kv_fp8": (ctypes.c_int, [c_vp, c_vp, c_vp, c_i32, c_vp, c_vp, c_f32, c_f32,
                                        _P(sgl_attn_dims), c_vp]),
    "sgl_decode_attention_fp8": (ctypes.c_int, [c_vp, c_vp, c_vp, c_f32, c_f32, c_vp, c_i32, c_i32, c_vp,
                                                c_vp, c_i32, c_i32, c_vp, c_vp, c_size, _P(sgl_attn_dims),
                                                c_vp]),
    "sgl_extend_attention_fp8": (ctypes.c_int, [c_vp, c_vp, c_vp, c_f32, c_f32, c_vp, c_i32, c_i32, c_vp,
                                                c_vp, c_vp, c_i32, c_i32, c_i32, c_i32, c_vp, c_vp, c_size,
                                                _P(sgl_attn_dims), c_vp]),
    "sgl_cascade_decode_attention_fp8": (ctypes.c_int, [c_vp, c_vp, c_vp, c_f32, c_f32, c_vp, c_i32, c_i32,
                                                        c_vp, c_vp, c_i32, c_i32, c_vp, c_vp, c_vp, c_vp,
                                                        c_vp, c_i32, c_i32, c_i32, c_vp, c_vp, c_size,
                                                        _P(sgl_attn_dims), c_vp]),
    "sgl_check_extend_fp8_indices": (ctypes.c_int, [c_vp, c_i32, c_i32, c_vp, c_vp, c_vp, c_i32, c_i32,
                                                    c_i32, c_i32, c_i64, c_vp, c_vp]),
    "sgl_decode_window_workspace_bytes": (c_size, [c_i32, c_i32, c_i32, c_i32, _P(sgl_attn_dims)]),
    "sgl_extend_window_workspace_bytes": (c_size, [c_i32] * 6 + [_P(sgl_attn_dims)]),
    "sgl_decode_attention_window": (ctypes.c_int, [c_vp] * 4 + [c_i32, c_i32, c_vp, c_vp] + [c_i32] * 4
                                    + [c_vp, c_vp, c_size, _P(sgl_attn_dims), c_vp]),
    "sgl_decode_attention_window_fp8": (ctypes.c_int, [c_vp] * 3 + [c_f32, c_f32, c_vp, c_i32, c_i32, c_vp, c_vp]
                                        + [c_i32] * 4 + [c_vp, c_vp, c_size, _P(sgl_attn_dims), c_vp]),
    "sgl_extend_attention_window": (ctypes.c_int, [c_vp] * 4 + [c_i32, c_i32, c_vp, c_vp, c_vp] + [c_i32] * 6
                                    + [c_vp, c_vp, c_size, _P(sgl_attn_dims), c_vp]),
    "sgl_extend_attention_window_fp8": (ctypes.c_int, [c_vp] * 3 + [c_f32, c_f32, c_vp, c_i32, c_i32, c_vp, c_vp,
                                                                    c_vp] + [c_i32] * 6
                                        + [c_vp, c_vp, c_size, _P(sgl_attn_dims), c_vp]),
    "sgl_check_decode_window_indices": (ctypes.c_int, [c_vp, c_i32, c_i32, c_vp, c_vp] + [c_i32] * 4
                                        + [c_i64, c_vp, c_vp]),
    "sgl_check_extend_window_indices": (ctypes.c_int, [c_vp, c_i32, c_i32, c_vp, c_vp, c_vp] + [c_i32] * 6
                                        + [c_i64, c_vp, c_vp]),
    "sgl_qk_norm_rope_store_kv": (ctypes.c_int, [c_vp, c_i64] * 3 + [c_vp, c_vp, c_f32, c_vp, c_i32, c_vp, c_vp,
                                                                     c_i32, c_i32, c_vp, c_i32, c_vp, c_vp, c_vp,
                                                                     _P(sgl_attn_dims), c_vp]),
    "sgl_qk_norm_rope_store_kv_fp8": (ctypes.c_int, [c_vp, c_i64] * 3
                                      + [c_vp, c_vp, c_f32, c_vp, c_i32, c_vp, c_vp, c_i32, c_i32, c_vp, c_i32,
                                         c_vp, c_vp, c_vp, c_f32, c_f32, _P(sgl_attn_dims), c_vp]),
    "sgl_check_cascade_scratch_bytes": (c_size, [c_i32, c_i32]),
    "sgl_check_cascade_groups": (ctypes.c_int, [c_vp, c_i32, c_i32, c_vp, c_vp, c_i32, c_vp, c_vp, c_vp,
                                                c_vp, c_vp, c_i32, c_i32, c_i32, c_vp, c_size, c_vp,
                                                c_vp]),
}

_lib = None


def lib() -> ctypes.CDLL:
    """Load (building first if needed) the C-ABI library."""
    global _lib
    if _lib is None:
        path = _build.LIB_PATH
        if not os.path.exists(path) or os.environ.get("SGL_ATTN_REBUILD"):
            path = _build.build()
        cdll = ctypes.CDLL(path)
        for name, (res, args) in _SIGS.items():
            f = getattr(cdll, name)
            f.restype = res
            f.argtypes = args
        _lib = cdll
    return _lib


def lib_path() -> str:
    return _build.LIB_PATH


def _check(name: str, code: int) -> None:
    if code != 0:
        raise SglError(name, code)


def make_dims(num_q_heads, num_kv_heads, head_dim, pool_size, sm_scale=0.0) -> sgl_attn_dims:
    return sgl_attn_dims(int(num_q_heads), int(num_kv_heads), int(head_dim), int(pool_size), float(sm_scale))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _dims_for(q_or_new, pool_k, sm_scale):
    return make_dims(q_or_new.shape[1] if q_or_new is not None else pool_k.shape[1],
                     pool_k.shape[1], pool_k.shape[2], pool_k.shape[0], sm_scale)


# ----------------------------------------------------------------- calls

def sgl_store_kv(k_new, v_new, slots, pool_k, pool_v, stream=None):
    """pool_k[slots[i]] = k_new[i]; pool_v[slots[i]] = v_new[i]."""
    d = make_dims(pool_k.shape[1], pool_k.shape[1], pool_k.shape[2], pool_k.shape[0])
    _check("sgl_store_kv", lib().sgl_store_kv(_ptr(k_new), _ptr(v_new), _ptr(slots), int(slots.shape[0]),
                                              _ptr(pool_k), _ptr(pool_v), ctypes.byref(d), _stream(stream)))


def extend_workspace_bytes(batch, total_extend, dims: sgl_attn_dims) -> int:
    return int(lib().sgl_extend_workspace_bytes(int(batch), int(total_extend), ctypes.byref(dims)))


def decode_workspace_bytes(batch, max_seq_len, dims: sgl_attn_dims) -> int:
    return int(lib().sgl_decode_workspace_bytes(int(batch), int(max_seq_len), ctypes.byref(dims)))


def new_workspace(nbytes: int, device):
    """A zero-filled device byte buffer (16-byte aligned by the allocator)."""
    import torch
    return torch.zeros(max(16, int(nbytes)), dtype=torch.uint8, device=device)


def sgl_extend_attention(q, k_new, v_new, pool_k, pool_v, req_to_token, req_pool_idx, prefix_lens,
                         extend_lens, out=None, *, max_extend, max_prefix=0, total_extend=None,
                         workspace=None, sm_scale=0.0, stream=None):
    """Attention of the suffix tokens over cached prefix + causal suffix.

    ``max_extend``/``max_prefix``/``total_extend`` are host-side values (the
    library never reads device memory on the host)."""
    import torch
    T = int(q.shape[0]) if total_extend is None else int(total_extend)
    d = _dims_for(q, pool_k, sm_scale)
    if out is None:
        out = torch.empty_like(q)
    B = int(req_pool_idx.shape[0])
    if workspace is None:
        workspace = new_workspace(extend_workspace_bytes(B, T, d), q.device)
    _check("sgl_extend_attention", lib().sgl_extend_attention(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(pool_k), _ptr(pool_v), _ptr(req_to_token),
        int(req_to_token.shape[0]), int(req_to_token.shape[1]), _ptr(req_pool_idx), _ptr(prefix_lens),
        _ptr(extend_lens), B, T, int(max_extend), int(max_prefix), _ptr(out), _ptr(workspace),
        int(workspace.numel() * workspace.element_size()), ctypes.byref(d), _stream(stream)))
    return out


def sgl_mixed_attention(q_ext, k_new, v_new, ext_req_pool_idx, prefix_lens, extend_lens, q_dec,
                        dec_req_pool_idx, seq_lens, pool_k, pool_v, req_to_token, out_ext=None, out_dec=None, *,
                        max_extend, max_prefix=0, max_seq_len, total_extend=None, ext_workspace=None,
                        dec_workspace=None, extend_sms=0, sm_scale=0.0, stream=None):
    """An extend batch and a decode batch over the same pools in one launch
    (outputs equal to sgl_extend_attention's and sgl_decode_attention's)."""
    import torch
    T = int(q_ext.shape[0]) if total_extend is None else int(total_extend)
    d = _dims_for(q_ext, pool_k, sm_scale)
    Be, Bd = int(ext_req_pool_idx.shape[0]), int(q_dec.shape[0])
    if out_ext is None:
        out_ext = torch.empty_like(q_ext)
    if out_dec is None:
        out_dec = torch.empty_like(q_dec)
    if ext_workspace is None:
        ext_workspace = new_workspace(extend_workspace_bytes(Be, T, d), q_ext.device)
    if dec_workspace is None:
        dec_workspace = new_workspace(decode_workspace_bytes(Bd, max_seq_len, d), q_dec.device)
    _check("sgl_mixed_attention", lib().sgl_mixed_attention(
        _ptr(q_ext), _ptr(k_new), _ptr(v_new), _ptr(ext_req_pool_idx), _ptr(prefix_lens), _ptr(extend_lens),
        Be, T, int(max_extend), int(max_prefix), _ptr(out_ext), _ptr(ext_workspace),
        int(ext_workspace.numel() * ext_workspace.element_size()), _ptr(q_dec), _ptr(dec_req_pool_idx),
        _ptr(seq_lens), Bd, int(max_seq_len), _ptr(out_dec), _ptr(dec_workspace),
        int(dec_workspace.numel() * dec_workspace.element_size()), _ptr(pool_k), _ptr(pool_v),
        _ptr(req_to_token), int(req_to_token.shape[0]), int(req_to_token.shape[1]), int(extend_sms),
        ctypes.byref(d), _stream(stream)))
    return out_ext, out_dec


def sgl_decode_attention(q, pool_k, pool_v, req_to_token, req_pool_idx, seq_lens, out=None, *,
                         max_seq_len, workspace=None, sm_scale=0.0, stream=None):
    """One query per request over all ``seq_len`` keys of its row."""
    import torch
    d = _dims_for(q, pool_k, sm_scale)
    if out is None:
        out = torch.empty_like(q)
    B = int(q.shape[0])
    if workspace is None:
        workspace = new_workspace(decode_workspace_bytes(B, max_seq_len, d), q.device)
    _check("sgl_decode_attention", lib().sgl_decode_attention(
        _ptr(q), _ptr(pool_k), _ptr(pool_v), _ptr(req_to_token), int(req_to_token.shape[0]),
        int(req_to_token.shape[1]), _ptr(req_pool_idx), _ptr(seq_lens), B, int(max_seq_len), _ptr(out),
        _ptr(workspace), int(workspace.numel() * workspace.element_size()), ctypes.byref(d),
        _stream(stream)))
    return out


def sgl_check_store_kv_indices(slots, pool_size, d_error, bitmap=None, stream=None):
    import torch
    need = ((int(pool_size) + 31) // 32 * 4 + 15) // 16 * 16
    if bitmap is None:
        bitmap = torch.empty(need, dtype=torch.uint8, device=slots.device)
    _check("sgl_check_store_kv_indices", lib().sgl_check_store_kv_indices(
        _ptr(slots), int(slots.shape[0]), int(pool_size), _ptr(bitmap),
        int(bitmap.numel()), _ptr(d_error), _stream(stream)))


def sgl_check_extend_indices(req_to_token, req_pool_idx, prefix_lens, extend_lens, *, total_extend,
                             max_extend, max_prefix, pool_size, d_error, stream=None, fp8=False):
    """``fp8``: the e4m3 extend's check (suffix positions' slots too)."""
    name = "sgl_check_extend_fp8_indices" if fp8 else "sgl_check_extend_indices"
    _check(name, getattr(lib(), name)(
        _ptr(req_to_token), int(req_to_token.shape[0]), int(req_to_token.shape[1]), _ptr(req_pool_idx),
        _ptr(prefix_lens), _ptr(extend_lens), int(req_pool_idx.shape[0]), int(total_extend),
        int(max_extend), int(max_prefix), int(pool_size), _ptr(d_error), _stream(stream)))


def sgl_check_decode_indices(req_to_token, req_pool_idx, seq_lens, *, max_seq_len, pool_size, d_error,
                             stream=None):
    _check("sgl_check_decode_indices", lib().sgl_check_decode_indices(
        _ptr(req_to_token), int(req_to_token.shape[0]), int(req_to_token.shape[1]), _ptr(req_pool_idx),
        _ptr(seq_lens), int(req_pool_idx.shape[0]), int(max_seq_len), int(pool_size), _ptr(d_error),
        _stream(stream)))


# ----------------------------------------------------------------- cascade

def cascade_decode_workspace_bytes(batch, max_seq_len, max_depth, dims: sgl_attn_dims) -> int:
    return int(lib().sgl_cascade_decode_workspace_bytes(int(batch), int(max_seq_len), int(max_depth),
                                                        ctypes.byref(dims)))


def sgl_cascade_decode_attention(q, pool_k, pool_v, req_to_token, req_pool_idx, seq_lens,
                                 group_start, group_len, group_depth, group_member_off, group_members,
                                 out=None, *, max_seq_len, max_group_members, max_depth,
                                 workspace=None, sm_scale=0.0, stream=None, kv_scales=None):
    """Decode attention with shared-prefix groups read once per group.

    ``group_*`` are int32 device tensors (CSR members); ``max_seq_len``,
    ``max_group_members`` and ``max_depth`` are host values.  A new workspace
    is zero-filled; a reused one must keep its first 256 bytes zero.
    ``kv_scales=(k_scale, v_scale)`` selects the e4m3-pool entry point."""
    import torch
    d = _dims_for(q, pool_k, sm_scale)
    if out is None:
        out = torch.empty_like(q)
    B = int(q.shape[0])
    G = int(group_start.shape[0])
    if workspace is None:
        workspace = new_workspace(cascade_decode_workspace_bytes(B, max_seq_len, max_depth, d), q.device)
    if kv_scales is None:
        name, head = "sgl_cascade_decode_attention", (_ptr(q), _ptr(pool_k), _ptr(pool_v))
    else:
        name = "sgl_cascade_decode_attention_fp8"
        head = (_ptr(q), _ptr(pool_k), _ptr(pool_v), float(kv_scales[0]), float(kv_scales[1]))
    _check(name, getattr(lib(), name)(
        *head, _ptr(req_to_token), int(req_to_token.shape[0]),
        int(req_to_token.shape[1]), _ptr(req_pool_idx), _ptr(seq_lens), B, int(max_seq_len),
        _ptr(group_start), _ptr(group_len), _ptr(group_depth), _ptr(group_member_off), _ptr(group_members),
        G, int(max_group_members), int(max_depth), _ptr(out), _ptr(workspace),
        int(workspace.numel() * workspace.element_size()), ctypes.byref(d), _stream(stream)))
    return out


def sgl_check_cascade_groups(req_to_token, req_pool_idx, seq_lens, group_start, group_len, group_depth,
                             group_member_off, group_members, *, max_group_members, max_depth, d_error,
                             scratch=None, stream=None):
    import torch
    B = int(req_pool_idx.shape[0])
    need = int(lib().sgl_check_cascade_scratch_bytes(B, int(max_depth)))
    if scratch is None:
        scratch = torch.empty(need, dtype=torch.uint8, device=req_to_token.device)
    _check("sgl_check_cascade_groups", lib().sgl_check_cascade_groups(
        _ptr(req_to_token), int(req_to_token.shape[0]), int(req_to_token.shape[1]), _ptr(req_pool_idx),
        _ptr(seq_lens), B, _ptr(group_start), _ptr(group_len), _ptr(group_depth), _ptr(group_member_off),
        _ptr(group_members), int(group_start.shape[0]), int(max_group_members), int(max_depth),
        _ptr(scratch), int(scratch.numel()), _ptr(d_error), _stream(stream)))


# ----------------------------------------------------------------- FP8 pool

def sgl_store_kv_fp8(k_new, v_new, slots, pool_k, pool_v, k_scale, v_scale, stream=None):
    """pool[slots[i]] = e4m3(new[i] / scale) for K and V (pools: torch.uint8 [S, Hkv, D])."""
    d = make_dims(pool_k.shape[1], pool_k.shape[1], pool_k.shape[2], pool_k.shape[0])
    _check("sgl_store_kv_fp8", lib().sgl_store_kv_fp8(
        _ptr(k_new), _ptr(v_new), _ptr(slots), int(slots.shape[0]), _ptr(pool_k), _ptr(pool_v),
        float(k_scale), float(v_scale), ctypes.byref(d), _stream(stream)))


def sgl_decode_attention_fp8(q, pool_k, pool_v, k_scale, v_scale, req_to_token, req_pool_idx, seq_lens,
                             out=None, *, max_seq_len, workspace=None, sm_scale=0.0, stream=None):
    """Decode attention over an e4m3 pool (values are code * scale)."""
    import torch
    d = _dims_for(q, pool_k, sm_scale)
    if out is None:
        out = torch.empty_like(q)
    B = int(q.shape[0])
    if workspace is None:
        workspace = new_workspace(decode_workspace_bytes(B, max_seq_len, d), q.device)
    _check("sgl_decode_attention_fp8", lib().sgl_decode_attention_fp8(
        _ptr(q), _ptr(pool_k), _ptr(pool_v), float(k_scale), float(v_scale), _ptr(req_to_token),
        int(req_to_token.shape[0]), int(req_to_token.shape[1]), _ptr(req_pool_idx), _ptr(seq_lens), B,
        int(max_seq_len), _ptr(out), _ptr(workspace), int(workspace.numel() * workspace.element_size()),
        ctypes.byref(d), _stream(stream)))
    return out


def sgl_extend_attention_fp8(q, pool_k, pool_v, k_scale, v_scale, req_to_token, req_pool_idx, prefix_lens,
                             extend_lens, out=None, *, max_extend, max_prefix=0, total_extend=None,
                             workspace=None, sm_scale=0.0, stream=None):
    """Extend attention over an e4m3 pool: prefix AND suffix keys are read
    from the pool through ``req_to_token`` (the suffix stored first)."""
    import torch
    T = int(q.shape[0]) if total_extend is None else int(total_extend)
    d = _dims_for(q, pool_k, sm_scale)
    if out is None:
        out = torch.empty_like(q)
    B = int(req_pool_idx.shape[0])
    if workspace is None:
        workspace = new_workspace(extend_workspace_bytes(B, T, d), q.device)
    _check("sgl_extend_attention_fp8", lib().sgl_extend_attention_fp8(
        _ptr(q), _ptr(pool_k), _ptr(pool_v), float(k_scale), float(v_scale), _ptr(req_to_token),
        int(req_to_token.shape[0]), int(req_to_token.shape[1]), _ptr(req_pool_idx), _ptr(prefix_lens),
        _ptr(extend_lens), B, T, int(max_extend), int(max_prefix), _ptr(out), _ptr(workspace),
        int(workspace.numel() * workspace.element_size()), ctypes.byref(d), _stream(stream)))
    return out


# ----------------------------------------------------------------- sliding window

@functools.lru_cache(maxsize=256)
def _dims_ref(num_q_heads, num_kv_heads, head_dim, pool_size, sm_scale):
    return ctypes.byref(make_dims(num_q_heads, num_kv_heads, head_dim, pool_size, sm_scale))


def _need(name, ok, what):
    if not ok:
        raise ValueError(f"{name}: {what}")


def _need_dense(name, dtype, **tensors):
    """Dense tensors of one type on the current device (None passes)."""
    import torch
    dev = torch.cuda.current_device()
    for arg, t in tensors.items():
        if t is not None and not (t.dtype is dtype and t.is_contiguous() and t.get_device() == dev):
            raise ValueError(f"{name}: {arg} must be a dense {dtype} tensor on the current CUDA device")


_I32 = 2**31 - 1


def _need_i32(name, **values):
    """Host values that the library takes as int32; ctypes would cut longer ones."""
    for arg, v in values.items():
        _need(name, -_I32 <= v <= _I32, f"{arg} = {v} is not an int32")


class _Torch:
    """What the calls below look up in torch at every call (bound at the first)."""

    def __init__(self):
        import torch
        self.bf16, self.i32, self.u8, self.f32 = torch.bfloat16, torch.int32, torch.uint8, torch.float32
        self.current_device = torch.cuda.current_device
        # the handle alone: torch.cuda.current_stream() builds an object around it
        self.current_stream = torch._C._cuda_getCurrentRawStream
        self.empty = torch.empty
        self.empty_like = torch.empty_like


@functools.lru_cache(maxsize=1)
def _torch():
    return _Torch()


def _raw_stream(stream):
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _stream_object(stream):
    """The torch stream of a call's ``stream`` argument: itself, or the one
    around a handle (0: the default stream, which ExternalStream does not take)."""
    import torch
    if isinstance(stream, torch.cuda.Stream):
        return stream
    handle = int(getattr(stream, "cuda_stream", stream))
    return torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()


def _on(stream):
    """Context whose allocations belong to the stream that a call runs on, so
    that a scratch buffer dropped on return is not handed out again before
    the call's kernels are done with it."""
    import contextlib

    import torch
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(_stream_object(stream))


def _in_use(stream, *tensors):
    """Tensors of a call on a stream of the caller's choice: dropped by the
    caller, their memory is not handed out again before the call's kernels are
    done with it.  (That the stream waits for what fills them is the caller's
    to see to.)"""
    if stream is not None:
        s = _stream_object(stream)
        for t in tensors:
            if t is not None:
                t.record_stream(s)


def decode_window_workspace_bytes(batch, max_seq_len, window, sinks, dims: sgl_attn_dims) -> int:
    _need_i32("decode_window_workspace_bytes", batch=batch, max_seq_len=max_seq_len, window=window, sinks=sinks)
    return int(lib().sgl_decode_window_workspace_bytes(int(batch), int(max_seq_len), int(window), int(sinks),
                                                       ctypes.byref(dims)))


def extend_window_workspace_bytes(batch, total_extend, max_extend, max_prefix, window, sinks,
                                  dims: sgl_attn_dims) -> int:
    _need_i32("extend_window_workspace_bytes", batch=batch, total_extend=total_extend, max_extend=max_extend,
              max_prefix=max_prefix, window=window, sinks=sinks)
    return int(lib().sgl_extend_window_workspace_bytes(int(batch), int(total_extend), int(max_extend),
                                                       int(max_prefix), int(window), int(sinks),
                                                       ctypes.byref(dims)))


def _refuse_window(name, q, pool_k, pool_v, kv_dtype, req_to_token, lens, out, workspace):
    """Names what a sliding-window call cannot take (its checks failed)."""
    import torch
    _need_dense(name, torch.bfloat16, q=q, out=out)
    _need_dense(name, kv_dtype, pool_k=pool_k, pool_v=pool_v)
    _need_dense(name, torch.int32, req_to_token=req_to_token, **lens)
    _need(name, q.dim() == 3 and pool_k.dim() == 3 and pool_v.shape == pool_k.shape
          and q.shape[2] == pool_k.shape[2], "q [T, Hq, D] and pools [S, Hkv, D]")
    _need(name, req_to_token.dim() == 2, "req_to_token [rows, stride]")
    _need(name, out is None or out.shape == q.shape, "out of q's shape")
    _need(name, workspace is None or (workspace.is_contiguous() and workspace.get_device() == q.get_device()),
          "workspace: a dense buffer on q's device")
    raise ValueError(f"{name}: one entry a request in {', '.join(lens)}"
                     + ("" if "prefix_lens" in lens else ", one query a request"))


# The calls check their tensors in one expression and look for what was wrong
# only when it fails: a decode step's kernels last a few microseconds.

def _decode_window(name, q, pool_k, pool_v, scales, req_to_token, req_pool_idx, seq_lens, out, max_seq_len,
                   window, sinks, workspace, sm_scale, stream):
    T = _torch()
    bf16, i32, dev = T.bf16, T.i32, T.current_device()
    kv = T.u8 if scales else bf16
    qs, ks, ts = q.shape, pool_k.shape, req_to_token.shape
    if not (q.dtype is bf16 and q.is_contiguous() and q.get_device() == dev and len(qs) == 3
            and pool_k.dtype is kv and pool_k.is_contiguous() and pool_k.get_device() == dev and len(ks) == 3
            and pool_v.dtype is kv and pool_v.is_contiguous() and pool_v.get_device() == dev
            and pool_v.shape == ks and qs[2] == ks[2]
            and req_to_token.dtype is i32 and req_to_token.is_contiguous() and req_to_token.get_device() == dev
            and len(ts) == 2
            and req_pool_idx.dtype is i32 and req_pool_idx.is_contiguous() and req_pool_idx.get_device() == dev
            and seq_lens.dtype is i32 and seq_lens.is_contiguous() and seq_lens.get_device() == dev
            and req_pool_idx.shape == qs[:1] and seq_lens.shape == qs[:1]
            and (out is None or (out.dtype is bf16 and out.is_contiguous() and out.get_device() == dev
                                 and out.shape == qs))
            and (workspace is None or (workspace.is_contiguous() and workspace.get_device() == dev))):
        _refuse_window(name, q, pool_k, pool_v, kv, req_to_token, dict(req_pool_idx=req_pool_idx, seq_lens=seq_lens),
                       out, workspace)
    if not (-_I32 <= window <= _I32 and -_I32 <= sinks <= _I32 and -_I32 <= max_seq_len <= _I32):
        _need_i32(name, window=window, sinks=sinks, max_seq_len=max_seq_len)
    dims = _dims_ref(qs[1], ks[1], ks[2], ks[0], float(sm_scale))
    if out is None or workspace is None:
        with _on(stream):
            if out is None:
                out = T.empty_like(q)
            if workspace is None:
                workspace = T.empty(max(16, lib().sgl_decode_window_workspace_bytes(
                    qs[0], int(max_seq_len), int(window), int(sinks), dims)), dtype=T.u8, device=q.device)
    code = getattr(lib(), name)(
        q.data_ptr(), pool_k.data_ptr(), pool_v.data_ptr(), *scales, req_to_token.data_ptr(), ts[0], ts[1],
        req_pool_idx.data_ptr(), seq_lens.data_ptr(), qs[0], int(max_seq_len), int(window), int(sinks), out.data_ptr(),
        workspace.data_ptr(), workspace.nbytes, dims,
        T.current_stream(dev) if stream is None else _raw_stream(stream))
    _in_use(stream, q, pool_k, pool_v, req_to_token, req_pool_idx, seq_lens, out, workspace)
    if code != 0:
        raise SglError(name, code)
    return out


def sgl_decode_attention_window(q, pool_k, pool_v, req_to_token, req_pool_idx, seq_lens, out=None, *,
                                max_seq_len, window, sinks=0, workspace=None, sm_scale=0.0, stream=None):
    """One query per request over its last ``window`` keys (the new token's
    among them) and its first ``sinks``; rows of length 0 are left as they were."""
    return _decode_window("sgl_decode_attention_window", q, pool_k, pool_v, (), req_to_token, req_pool_idx,
                          seq_lens, out, max_seq_len, window, sinks, workspace, sm_scale, stream)


def sgl_decode_attention_window_fp8(q, pool_k, pool_v, k_scale, v_scale, req_to_token, req_pool_idx, seq_lens,
                                    out=None, *, max_seq_len, window, sinks=0, workspace=None, sm_scale=0.0,
                                    stream=None):
    """``sgl_decode_attention_window`` over an e4m3 pool (values are code * scale)."""
    return _decode_window("sgl_decode_attention_window_fp8", q, pool_k, pool_v, (float(k_scale), float(v_scale)),
                          req_to_token, req_pool_idx, seq_lens, out, max_seq_len, window, sinks, workspace,
                          sm_scale, stream)


def _extend_window(name, q, pool_k, pool_v, scales, req_to_token, req_pool_idx, prefix_lens, extend_lens, out,
                   max_extend, max_prefix, window, sinks, total_extend, workspace, sm_scale, stream):
    T = _torch()
    bf16, i32, dev = T.bf16, T.i32, T.current_device()
    kv = T.u8 if scales else bf16
    qs, ks, ts, bs = q.shape, pool_k.shape, req_to_token.shape, req_pool_idx.shape
    if not (q.dtype is bf16 and q.is_contiguous() and q.get_device() == dev and len(qs) == 3
            and pool_k.dtype is kv and pool_k.is_contiguous() and pool_k.get_device() == dev and len(ks) == 3
            and pool_v.dtype is kv and pool_v.is_contiguous() and pool_v.get_device() == dev
            and pool_v.shape == ks and qs[2] == ks[2]
            and req_to_token.dtype is i32 and req_to_token.is_contiguous() and req_to_token.get_device() == dev
            and len(ts) == 2
            and req_pool_idx.dtype is i32 and req_pool_idx.is_contiguous() and req_pool_idx.get_device() == dev
            and prefix_lens.dtype is i32 and prefix_lens.is_contiguous() and prefix_lens.get_device() == dev
            and extend_lens.dtype is i32 and extend_lens.is_contiguous() and extend_lens.get_device() == dev
            and len(bs) == 1 and prefix_lens.shape == bs and extend_lens.shape == bs
            and (out is None or (out.dtype is bf16 and out.is_contiguous() and out.get_device() == dev
                                 and out.shape == qs))
            and (workspace is None or (workspace.is_contiguous() and workspace.get_device() == dev))):
        _refuse_window(name, q, pool_k, pool_v, kv, req_to_token,
                       dict(req_pool_idx=req_pool_idx, prefix_lens=prefix_lens, extend_lens=extend_lens), out,
                       workspace)
    total = qs[0] if total_extend is None else int(total_extend)
    _need(name, total <= qs[0], "total_extend within q's rows")
    if not (-_I32 <= window <= _I32 and -_I32 <= sinks <= _I32 and -_I32 <= max_extend <= _I32
            and -_I32 <= max_prefix <= _I32 and -_I32 <= total):
        _need_i32(name, window=window, sinks=sinks, max_extend=max_extend, max_prefix=max_prefix, total_extend=total)
    dims = _dims_ref(qs[1], ks[1], ks[2], ks[0], float(sm_scale))
    if out is None or workspace is None:
        with _on(stream):
            if out is None:
                out = T.empty_like(q)
            if workspace is None:
                workspace = new_workspace(lib().sgl_extend_window_workspace_bytes(
                    bs[0], total, int(max_extend), int(max_prefix), int(window), int(sinks), dims), q.device)
    code = getattr(lib(), name)(
        q.data_ptr(), pool_k.data_ptr(), pool_v.data_ptr(), *scales, req_to_token.data_ptr(), ts[0], ts[1],
        req_pool_idx.data_ptr(), prefix_lens.data_ptr(), extend_lens.data_ptr(), bs[0], total, int(max_extend),
        int(max_prefix), int(window), int(sinks), out.data_ptr(), workspace.data_ptr(), workspace.nbytes, dims,
        T.current_stream(dev) if stream is None else _raw_stream(stream))
    _in_use(stream, q, pool_k, pool_v, req_to_token, req_pool_idx, prefix_lens, extend_lens, out, workspace)
    if code != 0:
        raise SglError(name, code)
    return out


def sgl_extend_attention_window(q, pool_k, pool_v, req_to_token, req_pool_idx, prefix_lens, extend_lens, out=None,
                                *, max_extend, max_prefix, window, sinks=0, total_extend=None, workspace=None,
                                sm_scale=0.0, stream=None):
    """Attention of the suffix tokens over their last ``window`` keys and the
    request's first ``sinks``; prefix AND suffix keys are read from the pool
    through ``req_to_token`` (the suffix stored first)."""
    return _extend_window("sgl_extend_attention_window", q, pool_k, pool_v, (), req_to_token, req_pool_idx,
                          prefix_lens, extend_lens, out, max_extend, max_prefix, window, sinks, total_extend,
                          workspace, sm_scale, stream)


def sgl_extend_attention_window_fp8(q, pool_k, pool_v, k_scale, v_scale, req_to_token, req_pool_idx, prefix_lens,
                                    extend_lens, out=None, *, max_extend, max_prefix, window, sinks=0,
                                    total_extend=None, workspace=None, sm_scale=0.0, stream=None):
    """``sgl_extend_attention_window`` over an e4m3 pool (values are code * scale)."""
    return _extend_window("sgl_extend_attention_window_fp8", q, pool_k, pool_v, (float(k_scale), float(v_scale)),
                          req_to_token, req_pool_idx, prefix_lens, extend_lens, out, max_extend, max_prefix,
                          window, sinks, total_extend, workspace, sm_scale, stream)


def sgl_check_decode_window_indices(req_to_token, req_pool_idx, seq_lens, *, max_seq_len, window, sinks=0,
                                    pool_size, d_error, stream=None):
    _need_i32("sgl_check_decode_window_indices", max_seq_len=max_seq_len, window=window, sinks=sinks)
    _check("sgl_check_decode_window_indices", lib().sgl_check_decode_window_indices(
        _ptr(req_to_token), int(req_to_token.shape[0]), int(req_to_token.shape[1]), _ptr(req_pool_idx),
        _ptr(seq_lens), int(req_pool_idx.shape[0]), int(max_seq_len), int(window), int(sinks), int(pool_size),
        _ptr(d_error), _stream(stream)))
    _in_use(stream, req_to_token, req_pool_idx, seq_lens, d_error)


def sgl_check_extend_window_indices(req_to_token, req_pool_idx, prefix_lens, extend_lens, *, total_extend,
                                    max_extend, max_prefix, window, sinks=0, pool_size, d_error, stream=None):
    _need_i32("sgl_check_extend_window_indices", total_extend=total_extend, max_extend=max_extend,
              max_prefix=max_prefix, window=window, sinks=sinks)
    _check("sgl_check_extend_window_indices", lib().sgl_check_extend_window_indices(
        _ptr(req_to_token), int(req_to_token.shape[0]), int(req_to_token.shape[1]), _ptr(req_pool_idx),
        _ptr(prefix_lens), _ptr(extend_lens), int(req_pool_idx.shape[0]), int(total_extend), int(max_extend),
        int(max_prefix), int(window), int(sinks), int(pool_size), _ptr(d_error), _stream(stream)))
    _in_use(stream, req_to_token, req_pool_idx, prefix_lens, extend_lens, d_error)


# ----------------------------------------------------------------- norms, rotary positions, store

def _refuse_rope(name, q, k, v, positions, inv_freq, slots, pool_k, pool_v, kv_dtype, q_weight, k_weight, freq_axis,
                 q_out):
    """Names what the call cannot take (its checks failed)."""
    import torch
    bf16, dev = torch.bfloat16, torch.cuda.current_device()
    _need_dense(name, kv_dtype, pool_k=pool_k, pool_v=pool_v)
    _need(name, pool_k.dim() == 3 and pool_v.shape == pool_k.shape, "pools [S, Hkv, D]")
    for arg, t in (("q", q), ("k", k), ("v", v)):
        _need(name, t.dim() == 3 and t.dtype is bf16 and t.get_device() == dev and t.shape[0] == q.shape[0]
              and t.shape[2] == pool_k.shape[2] and (arg == "q" or t.shape[1] == pool_k.shape[1])
              and t.stride(2) == 1 and (t.shape[1] == 1 or t.stride(1) == t.shape[2]),
              f"{arg}: bf16 [n, heads, D] with dense rows on the current CUDA device")
    _need_dense(name, bf16, q_weight=q_weight, k_weight=k_weight, q_out=q_out)
    _need_dense(name, torch.int32, positions=positions, slots=slots, freq_axis=freq_axis)
    _need_dense(name, torch.float32, inv_freq=inv_freq)
    for arg, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        _need(name, w is None or w.shape == pool_k.shape[2:], f"{arg} [D]")
    _need(name, q_out is None or q_out.shape == q.shape, "q_out of q's shape")
    raise ValueError(f"{name}: one slot a token, positions [n] or [axes, n], inv_freq [rot / 2] and, with several "
                     "axes, freq_axis [rot / 2]")


def _qk_norm_rope_store(name, q, k, v, positions, inv_freq, slots, pool_k, pool_v, scales, q_weight, k_weight,
                        eps, freq_axis, interleaved, q_out, stream):
    T = _torch()
    bf16, i32, dev = T.bf16, T.i32, T.current_device()
    kv = T.u8 if scales else bf16
    qs, ps, qt, kt, vt = q.shape, pool_k.shape, q.stride(), k.stride(), v.stride()
    rot, axes, new, width = 0, 1, None, None
    if len(qs) == 3 == len(ps):
        new, width = (qs[0], ps[1], ps[2]), ps[2:]
    # dense rows; tokens may lie apart (parts of a packed projection)
    ok = (new is not None and q.dtype is bf16 and k.dtype is bf16 and v.dtype is bf16 and qs[2] == ps[2]
          and k.shape == new and v.shape == new and qt[2] == kt[2] == vt[2] == 1
          and (qt[1] == ps[2] or qs[1] == 1) and (kt[1] == vt[1] == ps[2] or ps[1] == 1)
          and q.get_device() == dev and k.get_device() == dev and v.get_device() == dev
          and pool_k.dtype is kv and pool_k.is_contiguous() and pool_k.get_device() == dev
          and pool_v.dtype is kv and pool_v.is_contiguous() and pool_v.get_device() == dev and pool_v.shape == ps
          and slots.dtype is i32 and slots.is_contiguous() and slots.get_device() == dev and slots.shape == qs[:1])
    if ok and inv_freq is not None:
        fs, xs = inv_freq.shape, positions.shape if positions is not None else ()
        if len(xs) == 2:
            axes = xs[0]
        ok = (len(fs) == 1 and inv_freq.dtype is T.f32 and inv_freq.is_contiguous() and inv_freq.get_device() == dev
              and 0 < len(xs) <= 2 and xs[-1] == qs[0] and axes > 0
              and positions.dtype is i32 and positions.is_contiguous() and positions.get_device() == dev
              and (axes == 1 or (freq_axis is not None and freq_axis.dtype is i32 and freq_axis.shape == fs
                                 and freq_axis.is_contiguous() and freq_axis.get_device() == dev)))
        rot = 2 * fs[0] if ok else 0
    if ok and q_weight is not None:
        ok = (q_weight.dtype is bf16 and q_weight.shape == width and q_weight.is_contiguous()
              and q_weight.get_device() == dev)
    if ok and k_weight is not None:
        ok = (k_weight.dtype is bf16 and k_weight.shape == width and k_weight.is_contiguous()
              and k_weight.get_device() == dev)
    if ok and q_out is not None:
        ok = q_out.dtype is bf16 and q_out.is_contiguous() and q_out.get_device() == dev and q_out.shape == qs
    if not ok:
        _refuse_rope(name, q, k, v, positions, inv_freq, slots, pool_k, pool_v, kv, q_weight, k_weight, freq_axis,
                     q_out)
    n, hq, d = qs
    if q_out is None:
        with _on(stream):
            q_out = T.empty(qs, dtype=bf16, device=q.device)
    if n > 1:
        qt, kt, vt = qt[0], kt[0], vt[0]
    else:   # the stride of a single token means nothing
        qt, kt, vt = hq * d, ps[1] * d, ps[1] * d
    code = getattr(lib(), name)(
        q.data_ptr(), qt, k.data_ptr(), kt, v.data_ptr(), vt,
        None if q_weight is None else q_weight.data_ptr(), None if k_weight is None else k_weight.data_ptr(),
        float(eps), positions.data_ptr() if rot else None, axes, inv_freq.data_ptr() if rot else None,
        freq_axis.data_ptr() if axes > 1 else None, rot, 1 if interleaved else 0, slots.data_ptr(), n,
        q_out.data_ptr(), pool_k.data_ptr(), pool_v.data_ptr(), *scales, _dims_ref(hq, ps[1], d, ps[0], 0.0),
        T.current_stream(dev) if stream is None else _raw_stream(stream))
    _in_use(stream, q, k, v, positions, inv_freq, slots, pool_k, pool_v, q_weight, k_weight, freq_axis, q_out)
    if code != 0:
        raise SglError(name, code)
    return q_out


def sgl_qk_norm_rope_store_kv(q, k, v, positions, inv_freq, slots, pool_k, pool_v, *, q_weight=None, k_weight=None,
                              eps=1e-6, freq_axis=None, interleaved=False, q_out=None, stream=None):
    """Head norms of Q and K, rotary positions, and the store of K and V into
    their slots, in one pass; returns the finished queries.

    ``q`` [n, Hq, D], ``k`` and ``v`` [n, Hkv, D] may be parts of one packed
    projection.  ``inv_freq`` [rot / 2] (None: no rotation) turns the first
    ``rot`` values of each row by ``positions`` [n], or [axes, n] with
    ``freq_axis`` naming each frequency's axis.  Tokens whose slot lies
    outside the pool are padding and leave everything as it was."""
    return _qk_norm_rope_store("sgl_qk_norm_rope_store_kv", q, k, v, positions, inv_freq, slots, pool_k, pool_v,
                               (), q_weight, k_weight, eps, freq_axis, interleaved, q_out, stream)


def sgl_qk_norm_rope_store_kv_fp8(q, k, v, positions, inv_freq, slots, pool_k, pool_v, k_scale, v_scale, *,
                                  q_weight=None, k_weight=None, eps=1e-6, freq_axis=None, interleaved=False,
                                  q_out=None, stream=None):
    """``sgl_qk_norm_rope_store_kv`` into an e4m3 pool (code = e4m3(row / scale))."""
    return _qk_norm_rope_store("sgl_qk_norm_rope_store_kv_fp8", q, k, v, positions, inv_freq, slots, pool_k, pool_v,
                               (float(k_scale), float(v_scale)), q_weight, k_weight, eps, freq_axis, interleaved,
                               q_out, stream)


# ----------------------------------------------------------------- radix tree

class RadixTree:
    """The library's radix tree of cached token runs (host side, C++).

    Token ids and slots are int sequences; node handles are ints."""

    def __init__(self):
        self._t = lib().sgl_radix_create()
        if not self._t:
            raise MemoryError("sgl_radix_create failed")

    def __del__(self):
        if getattr(self, "_t", None):
            lib().sgl_radix_destroy(self._t)
            self._t = None

    @staticmethod
    def _arr(xs):
        import numpy as np
        return np.ascontiguousarray(np.asarray(xs, dtype=np.int32))

    def match_prefix(self, tokens):
        """(matched length, slots along the path, last node handle)."""
        toks = self._arr(tokens)
        out = self._arr([0] * max(1, toks.size))
        node = c_i64(0)
        m = lib().sgl_radix_match_prefix(self._t, toks.ctypes.data, int(toks.size), out.ctypes.data,
                                         int(out.size), ctypes.byref(node))
        if m < 0:
            raise SglError("sgl_radix_match_prefix", 1)
        return int(m), out[:m].tolist(), int(node.value)

    def insert(self, tokens, slots):
        toks, sl = self._arr(tokens), self._arr(slots)
        if toks.size != sl.size:
            raise ValueError("one slot per token")
        m = lib().sgl_radix_insert(self._t, toks.ctypes.data, sl.ctypes.data, int(toks.size))
        if m < 0:
            raise SglError("sgl_radix_insert", 1)
        return int(m)

    def inc_lock_ref(self, node):
        _check("sgl_radix_inc_lock_ref", lib().sgl_radix_inc_lock_ref(self._t, int(node)))

    def dec_lock_ref(self, node):
        _check("sgl_radix_dec_lock_ref", lib().sgl_radix_dec_lock_ref(self._t, int(node)))

    def evict(self, num_tokens):
        cap = int(self.evictable_tokens) + 1
        out = self._arr([0] * cap)
        n = lib().sgl_radix_evict(self._t, int(num_tokens), out.ctypes.data, cap)
        if n < 0:
            raise SglError("sgl_radix_evict", 1)
        return out[:n].tolist()

    @property
    def evictable_tokens(self):
        return int(lib().sgl_radix_evictable_tokens(self._t))

    @property
    def protected_tokens(self):
        return int(lib().sgl_radix_protected_tokens(self._t))

    def groups(self, nodes):
        """Shared-prefix groups of a batch: (start, len, depth, member_off, members) int32 arrays."""
        import numpy as np
        hs = np.ascontiguousarray(np.asarray(nodes, dtype=np.int64))
        nm = c_i32(0)
        ng = lib().sgl_radix_groups(self._t, hs.ctypes.data, int(hs.size), None, None, None, None, None,
                                    0, 0, ctypes.byref(nm))
        if ng < 0:
            raise SglError("sgl_radix_groups", 1)
        start, length, depth = (np.zeros(ng, np.int32) for _ in range(3))
        off, mem = np.zeros(ng + 1, np.int32), np.zeros(max(1, nm.value), np.int32)
        ng2 = lib().sgl_radix_groups(self._t, hs.ctypes.data, int(hs.size), start.ctypes.data,
                                     length.ctypes.data, depth.ctypes.data, off.ctypes.data, mem.ctypes.data,
                                     ng, int(mem.size), ctypes.byref(nm))
        assert ng2 == ng
        return start, length, depth, off, mem[: nm.value]
