"""ctypes binding of the attention layer's operators (argument marshalling only, as ``_lib``).

Every tensor of a call lives on one CUDA device; the call runs on that device, on ``stream`` or the
device's current stream, and allocates its outputs and workspace there.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from ._lib import GDN2_BF16, GDN2_F32, _check, _dt, raw

# flags of gdn2_qk_rope (gdn2_rope_flags in include/gdn2.h)
ROPE_RMSNORM, ROPE_INTERLEAVED = 1, 2
# gdn2_cache_type
CACHE_BF16, CACHE_E4M3 = 0, 1

_NONE = ctypes.c_void_p(None)


def _ptr(t):
    return _NONE if t is None else ctypes.c_void_p(t.data_ptr())


def _bytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def _need(name, t, dtype, shape, dev):
    """`t` is a contiguous tensor of this dtype, shape (None: any) and device, or None."""
    if t is None:
        return
    if t.device != dev or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor on {dev}, is on {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, has {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


@contextlib.contextmanager
def _elsewhere(dev, stream):
    with torch.cuda.device(dev), torch.cuda.stream(stream):
        yield


_HERE = contextlib.nullcontext()


def _on(t, stream):
    """The device and stream of a call, for its allocations and its launches."""
    if not t.is_cuda:
        raise ValueError("q, k, v must be CUDA tensors")
    if stream is None and t.device.index == torch.cuda.current_device():
        return _HERE
    return _elsewhere(t.device, torch.cuda.current_stream(t.device) if stream is None else stream)


def _current():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _workspace(ws, nbytes, dev):
    if ws is None and nbytes > 0:
        return torch.empty(nbytes, dtype=torch.uint8, device=dev)
    if ws is not None and ws.device != dev:
        raise ValueError(f"workspace must be on {dev}")
    return ws


def _scale(scale, D):
    return D ** -0.5 if scale is None else float(scale)


# ------------------------------------------------------------------ norm and rotation
def _rope_args(q, k, q_weight, k_weight, positions, inv_freq, flags):
    if q.dim() < 2 or k.dim() != q.dim() or k.shape[:-2] != q.shape[:-2] or k.shape[-1] != q.shape[-1]:
        raise ValueError("q and k are [.., H, D] and [.., Hkv, D] over the same rows")
    dev, H, Hkv, D = q.device, q.shape[-2], k.shape[-2], q.shape[-1]
    N = q.numel() // (H * D) if H * D else 0
    _need("q", q, q.dtype, None, dev)
    _need("k", k, q.dtype, None, dev)
    _need("q_weight", q_weight, torch.float32, (D,), dev)
    _need("k_weight", k_weight, torch.float32, (D,), dev)
    rot = 0
    if inv_freq is not None:
        _need("inv_freq", inv_freq, torch.float32, None, dev)
        rot = 2 * inv_freq.numel()
        if positions is None:
            raise ValueError("inv_freq needs positions")
        _need("positions", positions, torch.int32, None, dev)
        if positions.numel() != N:
            raise ValueError(f"positions must hold one entry for each of the {N} rows")
    return dev, N, H, Hkv, D, rot


def gdn2_qk_rope(q, k, q_weight=None, k_weight=None, positions=None, inv_freq=None, *, flags=ROPE_RMSNORM, eps=1e-6,
                 rot_scale=1.0, q_out=None, k_out=None, stream=None):
    """Per-head RMS norm of q [.., H, D] and k [.., Hkv, D] (with ROPE_RMSNORM) and the rotation of
    their first 2 * len(inv_freq) channels by positions (int32, one per row).  Returns (q_out, k_out);
    q_out may be q and k_out k."""
    dev, N, H, Hkv, D, rot = _rope_args(q, k, q_weight, k_weight, positions, inv_freq, flags)
    with _on(q, stream):
        q_out = torch.empty_like(q) if q_out is None else q_out
        k_out = torch.empty_like(k) if k_out is None else k_out
        _need("q_out", q_out, q.dtype, q.shape, dev)
        _need("k_out", k_out, q.dtype, k.shape, dev)
        st = raw().gdn2_qk_rope(flags, _dt(q), N, H, Hkv, D, rot, _ptr(q), _ptr(k), _ptr(q_weight), _ptr(k_weight),
                                _ptr(positions), _ptr(inv_freq), eps, rot_scale, _ptr(q_out), _ptr(k_out), _current())
    _check("gdn2_qk_rope", st)
    return q_out, k_out


def gdn2_qk_rope_bwd(q, k, q_weight, k_weight, positions, inv_freq, d_q_out, d_k_out, *, flags=ROPE_RMSNORM, eps=1e-6,
                     rot_scale=1.0, out=None, workspace=None, stream=None):
    """The gradients of gdn2_qk_rope: dict(dq, dk, dq_weight, dk_weight).  The weight gradients (fp32
    [D]) are None without ROPE_RMSNORM.  Of a given ``out`` a weight gradient may be None."""
    dev, N, H, Hkv, D, rot = _rope_args(q, k, q_weight, k_weight, positions, inv_freq, flags)
    _need("d_q_out", d_q_out, q.dtype, q.shape, dev)
    _need("d_k_out", d_k_out, q.dtype, k.shape, dev)
    norm = bool(flags & ROPE_RMSNORM)
    with _on(q, stream):
        if out is None:
            w = torch.empty(2, D, dtype=torch.float32, device=dev) if norm else (None, None)
            out = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dq_weight": w[0], "dk_weight": w[1]}
        else:
            _need("dq", out["dq"], q.dtype, q.shape, dev)
            _need("dk", out["dk"], q.dtype, k.shape, dev)
            _need("dq_weight", out["dq_weight"], torch.float32, (D,), dev)
            _need("dk_weight", out["dk_weight"], torch.float32, (D,), dev)
        if norm and (out["dq_weight"] is not None or out["dk_weight"] is not None):
            workspace = _workspace(workspace, int(raw().gdn2_qk_rope_workspace_size(flags, _dt(q), N, H, Hkv, D)), dev)
        st = raw().gdn2_qk_rope_bwd(flags, _dt(q), N, H, Hkv, D, rot, _ptr(q), _ptr(k), _ptr(q_weight), _ptr(k_weight),
                                    _ptr(positions), _ptr(inv_freq), eps, rot_scale, _ptr(d_q_out), _ptr(d_k_out),
                                    _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dq_weight"]), _ptr(out["dk_weight"]),
                                    _ptr(workspace), _bytes(workspace), _current())
    _check("gdn2_qk_rope_bwd", st)
    return out


# ------------------------------------------------------------------ attention over whole sequences
def _attn_args(q, k, v, packed):
    rank = 3 if packed else 4
    if q.dim() != rank or k.dim() != rank:
        raise ValueError("q and k, v are " + ("[total_T, H, D] and [total_T, Hkv, D]" if packed else
                                              "[B, T, H, D] and [B, T, Hkv, D]"))
    dev = q.device
    _need("q", q, q.dtype, None, dev)
    _need("k", k, q.dtype, q.shape[:-2] + k.shape[-2:-1] + q.shape[-1:], dev)
    _need("v", v, q.dtype, k.shape, dev)
    return dev, q.shape[-2], k.shape[-2], q.shape[-1]


def _attn_fwd(q, k, v, cu_seqlens, window, scale, o, lse, want_lse, stream):
    packed = cu_seqlens is not None
    dev, H, Hkv, D = _attn_args(q, k, v, packed)
    with _on(q, stream):
        o = torch.empty_like(q) if o is None else o
        if lse is None and want_lse:
            lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=dev)
        _need("o", o, q.dtype, q.shape, dev)
        _need("lse", lse, torch.float32, q.shape[:-1], dev)
        tail = (_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _current())
        if packed:
            _need("cu_seqlens", cu_seqlens, torch.int32, None, dev)
            st = raw().gdn2_attn_fwd_varlen(_dt(q), cu_seqlens.numel() - 1, q.shape[0], H, Hkv, D, window,
                                            _scale(scale, D), _ptr(cu_seqlens), *tail)
        else:
            st = raw().gdn2_attn_fwd(_dt(q), q.shape[0], q.shape[1], H, Hkv, D, window, _scale(scale, D), *tail)
    _check("gdn2_attn_fwd_varlen" if packed else "gdn2_attn_fwd", st)
    return o, lse


def gdn2_attn_fwd(q, k, v, *, window=0, scale=None, o=None, lse=None, want_lse=True, stream=None):
    """Causal attention of q [B, T, H, D] over k, v [B, T, Hkv, D]; window > 0 limits a query to the last
    `window` keys, its own among them; scale defaults to D ** -0.5.  Returns (o, lse [B, T, H])."""
    return _attn_fwd(q, k, v, None, window, scale, o, lse, want_lse, stream)


def gdn2_attn_fwd_varlen(q, k, v, cu_seqlens, *, window=0, scale=None, o=None, lse=None, want_lse=True, stream=None):
    """gdn2_attn_fwd over packed sequences: q [total_T, H, D], cu_seqlens int32 [N + 1] on the device.
    Rows behind the last sequence are left as they were (unset in outputs allocated here)."""
    if cu_seqlens is None:
        raise ValueError("cu_seqlens is required")
    return _attn_fwd(q, k, v, cu_seqlens, window, scale, o, lse, want_lse, stream)


def _attn_bwd(q, k, v, o, lse, d_o, cu_seqlens, window, scale, out, workspace, stream):
    packed = cu_seqlens is not None
    dev, H, Hkv, D = _attn_args(q, k, v, packed)
    _need("o", o, q.dtype, q.shape, dev)
    _need("d_o", d_o, q.dtype, q.shape, dev)
    _need("lse", lse, torch.float32, q.shape[:-1], dev)
    with _on(q, stream):
        if out is None:
            out = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v)}
        else:
            for n, t in (("dq", q), ("dk", k), ("dv", v)):
                _need(n, out[n], q.dtype, t.shape, dev)
        N, T = (1, q.shape[0]) if packed else q.shape[:2]
        workspace = _workspace(workspace, int(raw().gdn2_attn_workspace_size(_dt(q), N, T, H, Hkv, D)), dev)
        tail = (_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(d_o), _ptr(out["dq"]), _ptr(out["dk"]),
                _ptr(out["dv"]), _ptr(workspace), _bytes(workspace), _current())
        if packed:
            _need("cu_seqlens", cu_seqlens, torch.int32, None, dev)
            st = raw().gdn2_attn_bwd_varlen(_dt(q), cu_seqlens.numel() - 1, T, H, Hkv, D, window, _scale(scale, D),
                                            _ptr(cu_seqlens), *tail)
        else:
            st = raw().gdn2_attn_bwd(_dt(q), N, T, H, Hkv, D, window, _scale(scale, D), *tail)
    _check("gdn2_attn_bwd_varlen" if packed else "gdn2_attn_bwd", st)
    return out


def gdn2_attn_bwd(q, k, v, o, lse, d_o, *, window=0, scale=None, out=None, workspace=None, stream=None):
    """The gradients of gdn2_attn_fwd from its inputs and outputs: dict(dq, dk, dv)."""
    return _attn_bwd(q, k, v, o, lse, d_o, None, window, scale, out, workspace, stream)


def gdn2_attn_bwd_varlen(q, k, v, o, lse, d_o, cu_seqlens, *, window=0, scale=None, out=None, workspace=None,
                         stream=None):
    """The gradients of gdn2_attn_fwd_varlen: dict(dq, dk, dv)."""
    if cu_seqlens is None:
        raise ValueError("cu_seqlens is required")
    return _attn_bwd(q, k, v, o, lse, d_o, cu_seqlens, window, scale, out, workspace, stream)


def gdn2_attn_workspace_size(dtype, N: int, T: int, H: int, Hkv: int, D: int) -> int:
    """Bytes of gdn2_attn_bwd's workspace (packed: N = 1, T = total_T)."""
    return int(raw().gdn2_attn_workspace_size(GDN2_F32 if dtype == torch.float32 else GDN2_BF16, N, T, H, Hkv, D))


# ------------------------------------------------------------------ the paged cache
def _cache_args(k_cache, v_cache, cu_seqlens, kv_lens, block_table, k_scale, v_scale):
    dev = k_cache.device
    if k_cache.dim() != 4:
        raise ValueError("k_cache and v_cache are [num_pages, page_size, Hkv, D]")
    if k_cache.dtype == torch.bfloat16:
        kind = CACHE_BF16
    elif k_cache.dtype == torch.float8_e4m3fn:
        kind = CACHE_E4M3
        if k_scale is None or v_scale is None:
            raise ValueError("an e4m3 cache has k_scale and v_scale")
        _need("k_scale", k_scale, torch.float32, k_cache.shape[:3], dev)
        _need("v_scale", v_scale, torch.float32, k_cache.shape[:3], dev)
    else:
        raise TypeError(f"unsupported cache dtype {k_cache.dtype} (bfloat16 or float8_e4m3fn)")
    _need("k_cache", k_cache, k_cache.dtype, None, dev)
    _need("v_cache", v_cache, k_cache.dtype, k_cache.shape, dev)
    N = kv_lens.numel()
    _need("cu_seqlens", cu_seqlens, torch.int32, (N + 1,), dev)
    _need("kv_lens", kv_lens, torch.int32, (N,), dev)
    if block_table.dim() != 2:
        raise ValueError("block_table is [N, max_pages]")
    _need("block_table", block_table, torch.int32, (N, block_table.shape[1]), dev)
    pages, page, Hkv, D = k_cache.shape
    return dev, kind, N, Hkv, D, (block_table.shape[1], pages, page)


def gdn2_cache_write(k, v, k_cache, v_cache, cu_seqlens, kv_lens, block_table, k_scale=None, v_scale=None, *,
                     stream=None):
    """Stores the new tokens' k and v [total_T, Hkv, D] in the paged cache [num_pages, page_size, Hkv, D]
    (bfloat16, or float8_e4m3fn with fp32 scales [num_pages, page_size, Hkv]).  Sequence n's rows are its
    last positions, kv_lens[n] counting them."""
    dev, kind, N, Hkv, D, sizes = _cache_args(k_cache, v_cache, cu_seqlens, kv_lens, block_table, k_scale, v_scale)
    T = k.shape[0]
    _need("k", k, torch.bfloat16, (T, Hkv, D), dev)
    _need("v", v, torch.bfloat16, (T, Hkv, D), dev)
    with _on(k, stream):
        st = raw().gdn2_cache_write(kind, GDN2_BF16, N, T, Hkv, D, _ptr(cu_seqlens), _ptr(kv_lens), _ptr(block_table),
                                    *sizes, _ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale),
                                    _ptr(v_scale), _current())
    _check("gdn2_cache_write", st)


def gdn2_cache_read(k_cache, v_cache, cu_seqlens, kv_lens, block_table, k_scale=None, v_scale=None, *, total_T=None,
                    k=None, v=None, stream=None):
    """Reads the last cu_seqlens[n + 1] - cu_seqlens[n] positions of every sequence back as bfloat16.
    Returns (k, v) [total_T, Hkv, D]; give total_T (cu_seqlens[-1]) or k and v."""
    dev, kind, N, Hkv, D, sizes = _cache_args(k_cache, v_cache, cu_seqlens, kv_lens, block_table, k_scale, v_scale)
    if total_T is None:
        if k is None:
            raise ValueError("give total_T, or k and v")
        total_T = k.shape[0]
    with _on(k_cache, stream):
        k = torch.empty(total_T, Hkv, D, dtype=torch.bfloat16, device=dev) if k is None else k
        v = torch.empty(total_T, Hkv, D, dtype=torch.bfloat16, device=dev) if v is None else v
        _need("k", k, torch.bfloat16, (total_T, Hkv, D), dev)
        _need("v", v, torch.bfloat16, (total_T, Hkv, D), dev)
        st = raw().gdn2_cache_read(kind, GDN2_BF16, N, total_T, Hkv, D, _ptr(cu_seqlens), _ptr(kv_lens),
                                   _ptr(block_table), *sizes, _ptr(k_cache), _ptr(v_cache), _ptr(k_scale),
                                   _ptr(v_scale), _ptr(k), _ptr(v), _current())
    _check("gdn2_cache_read", st)
    return k, v


def gdn2_attn_cached_workspace_size(N: int, total_T: int, H: int, Hkv: int, D: int, window: int, max_pages: int,
                                    page_size: int) -> int:
    return int(raw().gdn2_attn_cached_workspace_size(GDN2_BF16, N, total_T, H, Hkv, D, window, max_pages, page_size))


def gdn2_attn_cached(q, k_cache, v_cache, cu_seqlens, kv_lens, block_table, k_scale=None, v_scale=None, *, window=0,
                     scale=None, o=None, lse=None, want_lse=True, workspace=None, stream=None):
    """Attention of each sequence's newest tokens, q [total_T, H, D], over the paged cache that already
    holds them.  Returns (o [total_T, H, D], lse [total_T, H])."""
    dev, kind, N, Hkv, D, sizes = _cache_args(k_cache, v_cache, cu_seqlens, kv_lens, block_table, k_scale, v_scale)
    if q.dim() != 3:
        raise ValueError("q is [total_T, H, D]")
    T, H = q.shape[:2]
    _need("q", q, torch.bfloat16, (T, H, D), dev)
    with _on(q, stream):
        o = torch.empty_like(q) if o is None else o
        if lse is None and want_lse:
            lse = torch.empty(T, H, dtype=torch.float32, device=dev)
        _need("o", o, torch.bfloat16, q.shape, dev)
        _need("lse", lse, torch.float32, (T, H), dev)
        if workspace is None:
            workspace = _workspace(None, gdn2_attn_cached_workspace_size(N, T, H, Hkv, D, window, sizes[0], sizes[2]),
                                   dev)
        st = raw().gdn2_attn_cached(kind, GDN2_BF16, N, T, H, Hkv, D, window, _scale(scale, D), _ptr(cu_seqlens),
                                    _ptr(kv_lens), _ptr(block_table), *sizes, _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                    _ptr(k_scale), _ptr(v_scale), _ptr(o), _ptr(lse), _ptr(workspace),
                                    _bytes(workspace), _current())
    _check("gdn2_attn_cached", st)
    return o, lse
