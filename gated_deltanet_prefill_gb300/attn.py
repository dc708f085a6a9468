"""ctypes binding of the attention-layer operators (include/gdn2_attn.h): the
per-head norm with the rotary position embedding, the append to a paged
key/value cache and the attention over it.

Argument marshalling only, as in ``gdn2``: every step runs in the library's
CUDA kernels, outputs and workspaces are allocated with torch when the caller
does not pass them, and there is no CPU path.

A decode step calls these functions with a few microseconds of GPU work per
call.  So what depends on the tensors' metadata alone is worked out here, once
per set of shapes, strides, dtypes and options (the checks and the dims struct,
``_norm_rope_dims`` and its like), and the calls for known metadata are made by
a compiled module (csrc/gdn2_attn_call.cpp).  Nothing is kept by address or
content.
"""
from __future__ import annotations

import ctypes
import importlib.util
import math
import os

import torch

from . import build, gdn2
from .gdn2 import Gdn2Error, device_status  # noqa: F401  (status reader of these calls too)

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
_call = None  # the compiled module, bound to the library


def _raise(status, call):
    raise Gdn2Error(status, call)


def load():
    """The library of ``gdn2.load()`` with these entry points' signatures set,
    and the compiled module bound to it."""
    global _bound, _call
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
        path = build.call_path()
        if not os.path.exists(path):
            raise RuntimeError("%s is not built; run __graft_entry__.build()" % os.path.basename(path))
        spec = importlib.util.spec_from_file_location("gdn2_attn_call", path)
        call = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(call)
        call.bind(*(ctypes.cast(f, _vp).value for f in (lib.gdn2_qk_norm_rope, lib.gdn2_kv_append,
                                                        lib.gdn2_paged_attn_workspace_bytes, lib.gdn2_paged_attn_fwd)),
                  _raise)
        _call, _bound = call, lib
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
      0.1 ln(factor) + 1.  The ramp is linear in the turns; where it is linear
      in the pairs' index, frequencies inside it differ: pass such a table itself
      (the kernels take any)
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


def _rows(t):
    """Metadata of a strided tensor."""
    return None if t is None else (t.shape, t.stride(), t.dtype, t.is_cuda)


def _flat(t):
    """Metadata of a tensor that has to be contiguous."""
    return None if t is None else (t.numel(), t.dtype, t.is_cuda and t.is_contiguous())


def _code(*metas):
    """dtype code of the call: the tensors' one 16-bit dtype (99: refused by the library)."""
    dtypes = {m[2] for m in metas if m is not None}
    return _DTYPE_CODE.get(dtypes.pop(), 99) if len(dtypes) == 1 else 99


def _check_rows(name, m, shape=None):
    """(token, head) strides of a [T, heads, D] tensor on the device."""
    size, stride, _, cuda = m
    if not cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if len(size) != 3 or stride[2] != 1:
        raise ValueError("%s must be [tokens, heads, channels] with contiguous channels" % name)
    if shape is not None and tuple(size) != tuple(shape):
        raise ValueError("%s must have shape %s" % (name, tuple(shape)))
    return stride[:2]


def _check_flat(name, m, dtypes, n=None):
    if not m[2] or m[1] not in dtypes or (n is not None and m[0] != n):
        raise ValueError("%s must be a contiguous CUDA tensor of %s%s" % (
            name, " or ".join(str(d) for d in dtypes), "" if n is None else " with %d elements" % n))


def _check_rope(norm, ref, D, T, q_weight, k_weight, inv_freq, positions, need_positions):
    """(rot_dim, positions are int64)."""
    for w in (q_weight, k_weight):
        if w is not None:
            if not norm:
                raise ValueError("a norm weight was given, but norm is off")
            _check_flat("norm weight", w, (ref[2],), D)
    if inv_freq is None:
        return 0, 0
    _check_flat("inv_freq", inv_freq, (torch.float64,))
    if positions is None:
        if need_positions:
            raise ValueError("positions are required with inv_freq")
        return 2 * inv_freq[0], 0
    _check_flat("positions", positions, (torch.int32, torch.int64), T)
    return 2 * inv_freq[0], 1 if positions[1] == torch.int64 else 0


def _check_paged(k_cache, v_cache, table, lens, cu):
    """(sequences, strides of k_cache and v_cache, row stride and width of the table, cu is int64)."""
    if len(k_cache[0]) != 4 or k_cache[0] != v_cache[0] or not k_cache[3] or not v_cache[3]:
        raise ValueError("k_cache and v_cache must be CUDA tensors [pages, page_size, heads, channels] of one shape")
    kc, vc = k_cache[1], v_cache[1]
    if kc[3] != 1 or vc[3] != 1:
        raise ValueError("k_cache and v_cache: channels must be contiguous")
    n = cu[0] - 1
    size, stride, dtype, cuda = table
    if not cuda or dtype != torch.int32 or len(size) != 2 or size[0] != n or (size[1] > 1 and stride[1] != 1):
        raise ValueError("block_table must be an int32 CUDA tensor [sequences, pages] with contiguous rows")
    if n > 1 and stride[0] < size[1]:
        raise ValueError("block_table: the rows lie on top of one another (one row expanded to all sequences?)")
    _check_flat("cu_seqlens", cu, (torch.int32, torch.int64))
    _check_flat("kv_lens", lens, (torch.int32,), n)
    return n, kc[:3], vc[:3], stride[0] if n > 1 else size[1], size[1], 1 if cu[1] == torch.int64 else 0


def _norm_rope_dims(q, k, q_out, k_out, q_weight, k_weight, inv_freq, positions, norm, interleaved, eps, rope_factor):
    q, k, q_out, k_out = _rows(q), _rows(k), _rows(q_out), _rows(k_out)
    q_weight, k_weight, inv_freq, positions = _flat(q_weight), _flat(k_weight), _flat(inv_freq), _flat(positions)
    if len(q[0]) != 3:
        raise ValueError("q must be [tokens, heads, channels]")
    T, HQ, D = q[0]
    qs = _check_rows("q", q)
    qo = (HQ * D, D) if q_out is None else _check_rows("q_out", q_out, (T, HQ, D))
    HK, ks, ko = 0, (0, 0), (0, 0)
    if k is not None:
        ks = _check_rows("k", k)
        HK = k[0][1]
        _check_rows("k", k, (T, HK, D))
        ko = (HK * D, D) if k_out is None else _check_rows("k_out", k_out, (T, HK, D))
    elif k_out is not None:
        raise ValueError("k_out was given without k")
    rot, pos64 = _check_rope(norm, q, D, T, q_weight, k_weight, inv_freq, positions, True)
    return AttnDims(T, 0, qs, ks, (0, 0), qo, ko, (0, 0, 0), (0, 0, 0), 0, 0, HQ, HK, D, 0, 0,
                    _code(q, k, q_out, k_out), 0, pos64, 1 if norm else 0, rot, 1 if interleaved else 0, 1, -1, eps,
                    rope_factor)


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
    if _call is None:
        load()
    args = (q, k, positions, inv_freq, rope_factor, interleaved, norm, q_weight, k_weight, eps, q_out, k_out, stream)
    r = _call.qk_norm_rope(*args)
    if r is NotImplemented:
        r = _call.qk_norm_rope(*args, bytes(_norm_rope_dims(q, k, q_out, k_out, q_weight, k_weight, inv_freq, positions,
                                                            norm, interleaved, eps, rope_factor)))
    return r


def _append_dims(q, k, v, q_out, k_cache, v_cache, table, lens, cu, q_weight, k_weight, inv_freq, positions, norm,
                 interleaved, eps, rope_factor):
    q, k, v, q_out, k_cache, v_cache, table = [_rows(t) for t in (q, k, v, q_out, k_cache, v_cache, table)]
    lens, cu, q_weight, k_weight, inv_freq, positions = [
        _flat(t) for t in (lens, cu, q_weight, k_weight, inv_freq, positions)]
    ks = _check_rows("k", k)
    T, HKV, D = k[0]
    vs = _check_rows("v", v, (T, HKV, D))
    n, kc, vc, ts, width, cu64 = _check_paged(k_cache, v_cache, table, lens, cu)
    pages, page = k_cache[0][:2]
    if tuple(k_cache[0]) != (pages, page, HKV, D):
        raise ValueError("k_cache must have shape %s" % ((pages, page, HKV, D),))
    HQ, qs, qo = 0, (0, 0), (0, 0)
    if q is not None:
        qs = _check_rows("q", q)
        HQ = q[0][1]
        _check_rows("q", q, (T, HQ, D))
        qo = (HQ * D, D) if q_out is None else _check_rows("q_out", q_out, (T, HQ, D))
    elif q_out is not None:
        raise ValueError("q_out was given without q")
    rot, pos64 = _check_rope(norm, k, D, T, q_weight, k_weight, inv_freq, positions, False)
    return AttnDims(T, pages, qs, ks, vs, qo, (0, 0), kc, vc, ts, n, HQ, HKV, D, page, width,
                    _code(k, v, q, q_out, k_cache, v_cache), cu64, pos64, 1 if norm else 0, rot,
                    1 if interleaved else 0, 1, -1, eps, rope_factor)


def append_kv(k, v, k_cache, v_cache, block_table, kv_lens, cu_seqlens, q=None, positions=None, inv_freq=None,
              rope_factor=1.0, interleaved=False, norm=True, q_weight=None, k_weight=None, eps=1e-6, q_out=None,
              workspace=None, stream=None):
    """Append the new tokens' keys (normed and rotated as in ``qk_norm_rope``)
    and values to a paged cache through ``gdn2_kv_append``; with q, the queries
    are normed and rotated into q_out in the same launch.

    k, v [T, HKV, D]; k_cache, v_cache [pages, page_size, HKV, D] (any strides;
    pass a transposed view for head-major pages); block_table [N, max_pages]
    int32, its rows apart; cu_seqlens [N + 1] int32/int64; kv_lens [N] int32, the
    cached tokens of each sequence with the new ones.  The rotation's positions are the
    tokens' places in the cached sequences unless given.  ``device_status`` on
    the workspace (contiguous, on the inputs' device) reports a bad length,
    place or table entry.  Returns q_out (None without q).
    """
    if _call is None:
        load()
    args = (k, v, k_cache, v_cache, block_table, kv_lens, cu_seqlens, q, positions, inv_freq, rope_factor, interleaved,
            norm, q_weight, k_weight, eps, q_out, workspace, stream)
    r = _call.append_kv(*args)
    if r is NotImplemented:
        r = _call.append_kv(*args, bytes(_append_dims(q, k, v, q_out, k_cache, v_cache, block_table, kv_lens,
                                                      cu_seqlens, q_weight, k_weight, inv_freq, positions, norm,
                                                      interleaved, eps, rope_factor)))
    return r


def _attn_dims(q, k_cache, v_cache, table, lens, cu, out, lse, causal, window_left):
    q, k_cache, v_cache, table, out = _rows(q), _rows(k_cache), _rows(v_cache), _rows(table), _rows(out)
    lens, cu, lse = _flat(lens), _flat(cu), _flat(lse)
    qs = _check_rows("q", q)
    T, HQ, D = q[0]
    n, kc, vc, ts, width, cu64 = _check_paged(k_cache, v_cache, table, lens, cu)
    pages, page, HKV, dk = k_cache[0]
    if dk != D:
        raise ValueError("the cache's channels differ from q's")
    out_stride = (HQ * D, D) if out is None else _check_rows("out", out, (T, HQ, D))
    if lse is not None:
        _check_flat("lse", lse, (torch.float32,), T * HQ)
    return AttnDims(T, pages, qs, (0, 0), (0, 0), out_stride, (0, 0), kc, vc, ts, n, HQ, HKV, D, page, width,
                    _code(q, out, k_cache, v_cache), cu64, 0, 0, 0, 0, 1 if causal else 0,
                    min(window_left, 2 ** 31 - 1), 0.0, 1.0)


def paged_attn_fwd(q, k_cache, v_cache, block_table, kv_lens, cu_seqlens, scale=None, causal=True, window_left=-1,
                   out=None, lse=None, return_lse=False, workspace=None, stream=None):
    """Attention of the new tokens over the paged cache, which holds their keys
    and values already, through ``gdn2_paged_attn_fwd``.

    q [T, HQ, D] (HQ a multiple of the cache's heads); cache and tables as in
    ``append_kv``.  With ``causal`` a token attends to the keys up to its own
    place, with ``window_left`` >= 0 to at most that many before it (pages wholly
    before the first new token's window are not read); scale is positive, None
    means 1/sqrt(D).  Returns out [T, HQ, D], or (out, lse [T, HQ] fp32) with
    ``return_lse``; a token with no key gets zeros and lse -inf.
    """
    if _call is None:
        load()
    args = (q, k_cache, v_cache, block_table, kv_lens, cu_seqlens, scale, causal, window_left, out, lse, return_lse,
            workspace, stream)
    r = _call.paged_attn_fwd(*args)
    if r is NotImplemented:
        r = _call.paged_attn_fwd(*args, bytes(_attn_dims(q, k_cache, v_cache, block_table, kv_lens, cu_seqlens, out, lse,
                                                         causal, window_left)))
    return r
