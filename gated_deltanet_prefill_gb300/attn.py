"""ctypes binding of the attention-layer operators (include/gdn2_attn.h): the
per-head norm with the rotary position embedding, the append to a paged
key/value cache and the attention over it.

Argument marshalling only, as in ``gdn2``: every step runs in the library's
CUDA kernels, outputs and workspaces are allocated with torch when the caller
does not pass them, and there is no CPU path.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import gdn2
from .gdn2 import GDN2_OK, Gdn2Error, device_status  # noqa: F401  (status reader of these calls too)

EXPORTS = ("gdn2_attn_dims_init", "gdn2_qk_norm_rope", "gdn2_kv_append_workspace_bytes", "gdn2_kv_append",
           "gdn2_paged_attn_workspace_bytes", "gdn2_paged_attn_fwd")
_DTYPE_CODE = {torch.bfloat16: gdn2.DTYPE_BF16, torch.float16: gdn2.DTYPE_F16}
_i32, _i64, _f32, _vp, _sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t


class AttnDims(ctypes.Structure):
    _fields_ = [("T_tot", _i64), ("num_pages", _i64), ("q_stride", _i64 * 2), ("k_stride", _i64 * 2),
                ("v_stride", _i64 * 2), ("qo_stride", _i64 * 2), ("ko_stride", _i64 * 2),
                ("kc_stride", _i64 * 3), ("vc_stride", _i64 * 3), ("table_stride", _i64), ("N", _i32),
                ("HQ", _i32), ("HKV", _i32), ("D", _i32), ("page_size", _i32), ("max_pages", _i32),
                ("dtype", _i32), ("cu_seqlens_i64", _i32), ("positions_i64", _i32), ("norm", _i32),
                ("rot_dim", _i32), ("rope_interleaved", _i32), ("causal", _i32), ("window_left", _i32),
                ("norm_eps", _f32), ("rope_factor", _f32)]


_bound = None


def load():
    """The library of ``gdn2.load()`` with these entry points' signatures set."""
    global _bound
    lib = gdn2.load()
    if lib is not _bound:
        dims = ctypes.POINTER(AttnDims)
        lib.gdn2_attn_dims_init.argtypes = [dims, _i64, _i32, _i32, _i32, _i32, _i64, _i32, _i32]
        lib.gdn2_attn_dims_init.restype = ctypes.c_int
        lib.gdn2_qk_norm_rope.argtypes = [_vp] * 8 + [dims, _vp]
        lib.gdn2_qk_norm_rope.restype = ctypes.c_int
        lib.gdn2_kv_append_workspace_bytes.argtypes = [dims]
        lib.gdn2_kv_append_workspace_bytes.restype = _sz
        lib.gdn2_kv_append.argtypes = [_vp] * 13 + [dims, _vp, _sz, _vp]
        lib.gdn2_kv_append.restype = ctypes.c_int
        lib.gdn2_paged_attn_workspace_bytes.argtypes = [dims]
        lib.gdn2_paged_attn_workspace_bytes.restype = _sz
        lib.gdn2_paged_attn_fwd.argtypes = [_vp] * 6 + [_f32, _vp, _vp, dims, _vp, _sz, _vp]
        lib.gdn2_paged_attn_fwd.restype = ctypes.c_int
        _bound = lib
    return lib


def rope_frequencies(rot_dim, base=10000.0, scaling="none", factor=1.0, trained_len=0, beta_fast=32.0,
                     beta_slow=1.0, device="cuda"):
    """(inv_freq, rope_factor) for ``qk_norm_rope`` and ``append_kv``: the angle
    per position of each of the rot_dim / 2 pairs (float64 tensor), and the
    factor on cos and sin.  ``scaling`` extends the context ``factor`` times:

    * ``"none"``    base^(-2 i / rot_dim)
    * ``"linear"``  every frequency divided by ``factor`` (position interpolation)
    * ``"base"``    the base raised so that the slowest pair is slowed by ``factor``
    * ``"parts"``   pairs that turn fewer than ``beta_slow`` times in the
      ``trained_len`` tokens are slowed by ``factor``, those that turn more than
      ``beta_fast`` times are left, a linear ramp between; rope_factor is
      0.1 ln(factor) + 1
    """
    if rot_dim <= 0 or rot_dim % 2:
        raise ValueError("rot_dim must be positive and even")
    if scaling not in ("none", "linear", "base", "parts"):
        raise ValueError("scaling must be none, linear, base or parts")
    if scaling != "none" and not factor > 0:
        raise ValueError("factor must be positive")
    if scaling == "base" and rot_dim > 2:
        base = base * factor ** (rot_dim / (rot_dim - 2))
    f = base ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64) / rot_dim)
    rope_factor = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "parts":
        if trained_len <= 0 or not beta_fast > beta_slow:
            raise ValueError("parts needs trained_len > 0 and beta_fast > beta_slow")
        kept = ((trained_len * f / (2.0 * math.pi) - beta_slow) / (beta_fast - beta_slow)).clamp(0.0, 1.0)
        f = f * kept + f / factor * (1.0 - kept)
        rope_factor = 0.1 * math.log(factor) + 1.0
    return f.to(device), rope_factor


def _code(ref, *tensors):
    """dtype code of the call: the tensors' one 16-bit dtype (99: refused by the library)."""
    for t in tensors:
        if t is not None and t.dtype != ref.dtype:
            return 99
    return _DTYPE_CODE.get(ref.dtype, 99)


def _rows(name, t):
    """(token, head) strides of a [T, heads, D] tensor on the device."""
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    s = t.stride()
    if len(s) != 3 or s[2] != 1:
        raise ValueError("%s must be [tokens, heads, channels] with contiguous channels" % name)
    return s[:2]


def _same_shape(name, t, shape):
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s" % (name, tuple(shape)))


def _flat(name, t, dtypes, n=None):
    """A contiguous device tensor of one of the dtypes, with n elements."""
    if not t.is_cuda or t.dtype not in dtypes or not t.is_contiguous() or (n is not None and t.numel() != n):
        raise ValueError("%s must be a contiguous CUDA tensor of %s%s" % (
            name, " or ".join(str(d) for d in dtypes), "" if n is None else " with %d elements" % n))
    return t.data_ptr()


def _weights(norm, D, ref, q_weight, k_weight):
    if not norm and (q_weight is not None or k_weight is not None):
        raise ValueError("a norm weight was given, but norm is off")
    return [None if w is None else _flat("norm weight", w, (ref.dtype,), D) for w in (q_weight, k_weight)]


def _rotation(inv_freq, positions, T, need_positions):
    """(rot_dim, inv_freq pointer, positions pointer, positions are int64)."""
    if inv_freq is None:
        return 0, None, None, 0
    f = _flat("inv_freq", inv_freq, (torch.float64,))
    if positions is None:
        if need_positions:
            raise ValueError("positions are required with inv_freq")
        return 2 * inv_freq.numel(), f, None, 0
    p = _flat("positions", positions, (torch.int32, torch.int64), T)
    return 2 * inv_freq.numel(), f, p, 1 if positions.dtype == torch.int64 else 0


def _paged(k_cache, v_cache, block_table, kv_lens, cu_seqlens):
    """Shapes, strides and pointers of the cache and its tables."""
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape or not k_cache.is_cuda or not v_cache.is_cuda:
        raise ValueError("k_cache and v_cache must be CUDA tensors [pages, page_size, heads, channels] of one shape")
    kc, vc = k_cache.stride(), v_cache.stride()
    if kc[3] != 1 or vc[3] != 1:
        raise ValueError("k_cache and v_cache: channels must be contiguous")
    n = cu_seqlens.numel() - 1
    if not block_table.is_cuda or block_table.dtype != torch.int32 or block_table.dim() != 2 \
            or block_table.shape[0] != n or (block_table.shape[1] > 1 and block_table.stride(1) != 1):
        raise ValueError("block_table must be an int32 CUDA tensor [sequences, pages] with contiguous rows")
    cu = _flat("cu_seqlens", cu_seqlens, (torch.int32, torch.int64))
    lens = _flat("kv_lens", kv_lens, (torch.int32,), n)
    width = block_table.shape[1]
    return n, kc[:3], vc[:3], max(block_table.stride(0), width), width, cu, lens


def _stream(t, stream):
    return torch.cuda.current_stream(t.device).cuda_stream if stream is None else stream


def qk_norm_rope(q, k=None, positions=None, inv_freq=None, rope_factor=1.0, interleaved=False, norm=True,
                 q_weight=None, k_weight=None, eps=1e-6, q_out=None, k_out=None, stream=None):
    """RMS norm of every query and key head and the rotary position embedding
    through ``gdn2_qk_norm_rope``, in one pass.

    q [T, HQ, D], k [T, HK, D] (or None) at bf16 or fp16, D 64 or 128, views of
    a packed projection included; q_weight, k_weight [D] at the same dtype or
    None for ones; positions [T] int32/int64; inv_freq [rot_dim / 2] float64
    (``rope_frequencies``), None for no rotation.  The first rot_dim channels
    are rotated, in pairs (i, i + rot_dim / 2), or (2 i, 2 i + 1) with
    ``interleaved``.  q_out, k_out may be q, k (in place).  Returns (q_out,
    k_out).
    """
    lib = load()
    T, HQ, D = q.shape
    HK = 0
    if k is not None:
        HK = k.shape[1]
        _same_shape("k", k, (T, HK, D))
    q_out = torch.empty((T, HQ, D), dtype=q.dtype, device=q.device) if q_out is None else q_out
    _same_shape("q_out", q_out, (T, HQ, D))
    if k is None:
        if k_out is not None:
            raise ValueError("k_out was given without k")
    else:
        k_out = torch.empty((T, HK, D), dtype=k.dtype, device=k.device) if k_out is None else k_out
        _same_shape("k_out", k_out, (T, HK, D))
    wq, wk = _weights(norm, D, q, q_weight, k_weight)
    rot, f, pos, pos64 = _rotation(inv_freq, positions, T, True)
    ks, kos = (_rows("k", k), _rows("k_out", k_out)) if k is not None else ((0, 0), (0, 0))
    dims = AttnDims(T, 0, _rows("q", q), ks, (0, 0), _rows("q_out", q_out), kos, (0, 0, 0), (0, 0, 0), 0, 0, HQ, HK,
                    D, 0, 0, _code(q, k, q_out, k_out), 0, pos64, 1 if norm else 0, rot, 1 if interleaved else 0, 1,
                    -1, eps, rope_factor)
    st = lib.gdn2_qk_norm_rope(q.data_ptr(), None if k is None else k.data_ptr(), wq, wk, f, pos, q_out.data_ptr(),
                               None if k is None else k_out.data_ptr(), dims, _stream(q, stream))
    if st != GDN2_OK:
        raise Gdn2Error(st, "gdn2_qk_norm_rope")
    return q_out, k_out


def append_kv(k, v, k_cache, v_cache, block_table, kv_lens, cu_seqlens, q=None, positions=None, inv_freq=None,
              rope_factor=1.0, interleaved=False, norm=True, q_weight=None, k_weight=None, eps=1e-6, q_out=None,
              workspace=None, stream=None):
    """Append the new tokens' keys (normed and rotated as in ``qk_norm_rope``)
    and values to a paged cache through ``gdn2_kv_append``; with q, the queries
    are normed and rotated into q_out in the same launch.

    k, v [T, HKV, D]; k_cache, v_cache [pages, page_size, HKV, D] (any strides;
    pass a transposed view for head-major pages); block_table [N, max_pages]
    int32; cu_seqlens [N + 1] int32/int64; kv_lens [N] int32, the cached tokens
    of each sequence with the new ones.  The rotation's positions are the
    tokens' places in the cached sequences unless given.  ``device_status`` on
    the workspace reports a bad length, place or table entry.  Returns q_out
    (None without q).
    """
    lib = load()
    T, HKV, D = k.shape
    _same_shape("v", v, (T, HKV, D))
    n, kc, vc, ts, width, cu, lens = _paged(k_cache, v_cache, block_table, kv_lens, cu_seqlens)
    pages, page = k_cache.shape[:2]
    _same_shape("k_cache", k_cache, (pages, page, HKV, D))
    HQ, qs, qos = 0, (0, 0), (0, 0)
    if q is not None:
        HQ = q.shape[1]
        _same_shape("q", q, (T, HQ, D))
        q_out = torch.empty((T, HQ, D), dtype=q.dtype, device=q.device) if q_out is None else q_out
        _same_shape("q_out", q_out, (T, HQ, D))
        qs, qos = _rows("q", q), _rows("q_out", q_out)
    elif q_out is not None:
        raise ValueError("q_out was given without q")
    wq, wk = _weights(norm, D, k, q_weight, k_weight)
    rot, f, pos, pos64 = _rotation(inv_freq, positions, T, False)
    if workspace is None:
        workspace = torch.empty(64, dtype=torch.uint8, device=k.device)
    dims = AttnDims(T, pages, qs, _rows("k", k), _rows("v", v), qos, (0, 0), kc, vc, ts, n, HQ, HKV, D, page, width,
                    _code(k, v, q, q_out, k_cache, v_cache), 1 if cu_seqlens.dtype == torch.int64 else 0, pos64,
                    1 if norm else 0, rot, 1 if interleaved else 0, 1, -1, eps, rope_factor)
    st = lib.gdn2_kv_append(None if q is None else q.data_ptr(), k.data_ptr(), v.data_ptr(), wq, wk, f, pos, cu, lens,
                            block_table.data_ptr(), None if q is None else q_out.data_ptr(), k_cache.data_ptr(),
                            v_cache.data_ptr(), dims, workspace.data_ptr(), workspace.numel(), _stream(k, stream))
    if st != GDN2_OK:
        raise Gdn2Error(st, "gdn2_kv_append")
    return q_out


def paged_attn_fwd(q, k_cache, v_cache, block_table, kv_lens, cu_seqlens, scale=None, causal=True, window_left=-1,
                   out=None, lse=None, return_lse=False, workspace=None, stream=None):
    """Attention of the new tokens over the paged cache, which holds their keys
    and values already, through ``gdn2_paged_attn_fwd``.

    q [T, HQ, D] (HQ a multiple of the cache's heads); cache and tables as in
    ``append_kv``.  With ``causal`` a token attends to the keys up to its own
    place, with ``window_left`` >= 0 to at most that many before it; scale None
    means 1/sqrt(D).  Returns out [T, HQ, D], or (out, lse [T, HQ] fp32) with
    ``return_lse``; a token with no key gets zeros and lse -inf.
    """
    lib = load()
    T, HQ, D = q.shape
    n, kc, vc, ts, width, cu, lens = _paged(k_cache, v_cache, block_table, kv_lens, cu_seqlens)
    pages, page, HKV, dk = k_cache.shape
    if dk != D:
        raise ValueError("the cache's channels differ from q's")
    out = torch.empty((T, HQ, D), dtype=q.dtype, device=q.device) if out is None else out
    _same_shape("out", out, (T, HQ, D))
    if lse is None:
        lse = torch.empty((T, HQ), dtype=torch.float32, device=q.device) if return_lse else None
    lse_ptr = None if lse is None else _flat("lse", lse, (torch.float32,), T * HQ)
    dims = AttnDims(T, pages, _rows("q", q), (0, 0), (0, 0), _rows("out", out), (0, 0), kc, vc, ts, n, HQ, HKV, D,
                    page, width, _code(q, out, k_cache, v_cache), 1 if cu_seqlens.dtype == torch.int64 else 0, 0, 0,
                    0, 0, 1 if causal else 0, window_left, 0.0, 1.0)
    if workspace is None:
        need = lib.gdn2_paged_attn_workspace_bytes(dims)
        workspace = torch.empty(max(need, 64), dtype=torch.uint8, device=q.device)
    st = lib.gdn2_paged_attn_fwd(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), cu, lens,
                                 block_table.data_ptr(), 0.0 if scale is None else scale, out.data_ptr(), lse_ptr,
                                 dims, workspace.data_ptr(), workspace.numel(), _stream(q, stream))
    if st != GDN2_OK:
        raise Gdn2Error(st, "gdn2_paged_attn_fwd")
    return (out, lse) if return_lse else out
