"""ctypes binding of the attention layer's operators (argument marshalling only, as ``_lib``).

Every tensor of a call lives on one CUDA device; the call runs on that device, on ``stream`` or the
device's current stream, and allocates its outputs and workspace there.
"""
from __future__ import annotations

import contextlib
import math

import torch

from ._lib import GDN2_BF16, GDN2_F32, _check, _dt, raw

# flags of gdn2_qk_rope (gdn2_rope_flags in include/gdn2.h)
ROPE_RMSNORM, ROPE_INTERLEAVED = 1, 2
# gdn2_cache_type
CACHE_BF16, CACHE_E4M3 = 0, 1


def _ptr(t):
    return None if t is None else t.data_ptr()


def _bytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def _need(name, t, dtype, shape, dev):
    """`t` is a contiguous tensor of this dtype, shape (a tuple; None: any) and device, or None.  One
    expression on the way of every call; what is wrong is found out afterwards."""
    if t is None or (t.dtype is dtype and t.get_device() == dev and (shape is None or t.shape == shape) and t.is_contiguous()):
        return
    if t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor on the call's device, is on {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, has {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _device(t):
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"the tensors must be CUDA tensors, are on {t.device}")
    return dev


@contextlib.contextmanager
def _elsewhere(dev, stream):
    with torch.cuda.device(dev), torch.cuda.stream(stream):
        yield


_HERE = contextlib.nullcontext()


def _on(dev, stream):
    """The device and stream of a call, for its allocations and its launches."""
    if stream is None and dev == torch.cuda.current_device():
        return _HERE
    return _elsewhere(dev, torch.cuda.current_stream(dev) if stream is None else stream)


def _current(dev):
    # the handle alone: torch.cuda.current_stream() builds a Stream object, 3 us of a decode step's call
    return torch._C._cuda_getCurrentRawStream(dev)


def _workspace(ws, nbytes, dev):
    if ws is None and nbytes > 0:
        return torch.empty(nbytes, dtype=torch.uint8, device=dev)
    if ws is not None and ws.get_device() != dev:
        raise ValueError("workspace must be on the call's device")
    return ws


def _scale(scale, D):
    return D ** -0.5 if scale is None else float(scale)


# ------------------------------------------------------------------ norm and rotation
def _rope_args(q, k, q_weight, k_weight, positions, inv_freq):
    dev, dtype, qs, ks = _device(q), q.dtype, q.shape, k.shape
    if len(qs) < 2 or len(ks) != len(qs) or ks[:-2] != qs[:-2] or ks[-1] != qs[-1]:
        raise ValueError("q and k are [.., H, D] and [.., Hkv, D] over the same rows")
    H, D = qs[-2:]
    N = math.prod(qs[:-2])
    _need("q", q, dtype, qs, dev)
    _need("k", k, dtype, ks, dev)
    _need("q_weight", q_weight, torch.float32, (D,), dev)
    _need("k_weight", k_weight, torch.float32, (D,), dev)
    rot = 0
    if inv_freq is not None:
        _need("inv_freq", inv_freq, torch.float32, None, dev)
        rot = 2 * inv_freq.numel()
        if positions is None or positions.numel() != N:
            raise ValueError(f"inv_freq needs positions, one entry for each of the {N} rows")
        _need("positions", positions, torch.int32, None, dev)
    return dev, dtype, qs, ks, N, H, ks[-2], D, rot


def gdn2_qk_rope(q, k, q_weight=None, k_weight=None, positions=None, inv_freq=None, *, flags=ROPE_RMSNORM, eps=1e-6,
                 rot_scale=1.0, q_out=None, k_out=None, stream=None):
    """Per-head RMS norm of q [.., H, D] and k [.., Hkv, D] (with ROPE_RMSNORM) and the rotation of
    their first 2 * len(inv_freq) channels by positions (int32, one per row).  Returns (q_out, k_out);
    q_out may be q and k_out k."""
    dev, dtype, qs, ks, N, H, Hkv, D, rot = _rope_args(q, k, q_weight, k_weight, positions, inv_freq)
    with _on(dev, stream):
        if q_out is None:
            q_out = torch.empty_like(q)
        else:
            _need("q_out", q_out, dtype, qs, dev)
        if k_out is None:
            k_out = torch.empty_like(k)
        else:
            _need("k_out", k_out, dtype, ks, dev)
        st = raw().gdn2_qk_rope(flags, _dt(q), N, H, Hkv, D, rot, _ptr(q), _ptr(k), _ptr(q_weight), _ptr(k_weight),
                                _ptr(positions), _ptr(inv_freq), eps, rot_scale, _ptr(q_out), _ptr(k_out), _current(dev))
    _check("gdn2_qk_rope", st)
    return q_out, k_out


def gdn2_qk_rope_bwd(q, k, q_weight, k_weight, positions, inv_freq, d_q_out, d_k_out, *, flags=ROPE_RMSNORM, eps=1e-6,
                     rot_scale=1.0, out=None, workspace=None, stream=None):
    """The gradients of gdn2_qk_rope: dict(dq, dk, dq_weight, dk_weight).  The weight gradients (fp32
    [D]) are None without ROPE_RMSNORM.  Of a given ``out`` a weight gradient may be None."""
    dev, dtype, qs, ks, N, H, Hkv, D, rot = _rope_args(q, k, q_weight, k_weight, positions, inv_freq)
    _need("d_q_out", d_q_out, dtype, qs, dev)
    _need("d_k_out", d_k_out, dtype, ks, dev)
    norm = bool(flags & ROPE_RMSNORM)
    with _on(dev, stream):
        if out is None:
            w = torch.empty(2, D, dtype=torch.float32, device=dev) if norm else (None, None)
            out = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dq_weight": w[0], "dk_weight": w[1]}
        else:
            _need("dq", out["dq"], q.dtype, q.shape, dev)
            _need("dk", out["dk"], q.dtype, k.shape, dev)
            _need("dq_weight", out["dq_weight"], torch.float32, (D,), dev)
            _need("dk_weight", out["dk_weight"], torch.float32, (D,), dev)
        if norm and (out["dq_weight"] is not None or out["dk_weight"] is not None):
            workspace = _workspace(workspace, raw().gdn2_qk_rope_workspace_size(flags, _dt(q), N, H, Hkv, D), dev)
        st = raw().gdn2_qk_rope_bwd(flags, _dt(q), N, H, Hkv, D, rot, _ptr(q), _ptr(k), _ptr(q_weight), _ptr(k_weight),
                                    _ptr(positions), _ptr(inv_freq), eps, rot_scale, _ptr(d_q_out), _ptr(d_k_out),
                                    _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dq_weight"]), _ptr(out["dk_weight"]),
                                    _ptr(workspace), _bytes(workspace), _current(dev))
    _check("gdn2_qk_rope_bwd", st)
    return out


def gdn2_qk_rope_workspace_size(dtype, N: int, H: int, Hkv: int, D: int, flags: int = ROPE_RMSNORM) -> int:
    """Bytes of gdn2_qk_rope_bwd's workspace for up to N rows (0 without ROPE_RMSNORM: none is needed)."""
    return int(raw().gdn2_qk_rope_workspace_size(flags, GDN2_F32 if dtype == torch.float32 else GDN2_BF16, N, H, Hkv, D))


# ------------------------------------------------------------------ attention over whole sequences
def _attn_args(q, k, v, cu_seqlens):
    dev, dtype, qs, ks = _device(q), q.dtype, q.shape, k.shape
    packed = cu_seqlens is not None
    if len(qs) != (3 if packed else 4) or len(ks) != len(qs):
        raise ValueError("q and k, v are " + ("[total_T, H, D] and [total_T, Hkv, D]" if packed else
                                              "[B, T, H, D] and [B, T, Hkv, D]"))
    *lead, H, D = qs
    _need("q", q, dtype, qs, dev)
    _need("k", k, dtype, (*lead, ks[-2], D), dev)
    _need("v", v, dtype, ks, dev)
    if packed:
        _need("cu_seqlens", cu_seqlens, torch.int32, None, dev)
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens is [N + 1] with N >= 1")
        lead = (cu_seqlens.numel() - 1, *lead)
    return dev, dtype, qs, lead, H, ks[-2], D


def _attn_fwd(q, k, v, cu_seqlens, window, scale, o, lse, want_lse, stream):
    dev, dtype, qs, (n, t), H, Hkv, D = _attn_args(q, k, v, cu_seqlens)
    with _on(dev, stream):
        if o is None:
            o = torch.empty_like(q)
        else:
            _need("o", o, dtype, qs, dev)
        if lse is not None:
            _need("lse", lse, torch.float32, qs[:-1], dev)
        elif want_lse:
            lse = torch.empty(qs[:-1], dtype=torch.float32, device=dev)
        head = (_dt(q), n, t, H, Hkv, D, window, _scale(scale, D))
        tail = (_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _current(dev))
        if cu_seqlens is not None:
            st = raw().gdn2_attn_fwd_varlen(*head, _ptr(cu_seqlens), *tail)
        else:
            st = raw().gdn2_attn_fwd(*head, *tail)
    _check("gdn2_attn_fwd" if cu_seqlens is None else "gdn2_attn_fwd_varlen", st)
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
    dev, dtype, qs, (n, t), H, Hkv, D = _attn_args(q, k, v, cu_seqlens)
    _need("o", o, dtype, qs, dev)
    _need("d_o", d_o, dtype, qs, dev)
    _need("lse", lse, torch.float32, qs[:-1], dev)
    with _on(dev, stream):
        if out is None:
            out = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v)}
        else:
            for name, x in (("dq", q), ("dk", k), ("dv", v)):
                _need(name, out[name], dtype, x.shape, dev)
        rows = t if cu_seqlens is not None else n * t
        workspace = _workspace(workspace, raw().gdn2_attn_workspace_size(_dt(q), 1, rows, H, Hkv, D), dev)
        head = (_dt(q), n, t, H, Hkv, D, window, _scale(scale, D))
        tail = (_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(d_o), _ptr(out["dq"]), _ptr(out["dk"]),
                _ptr(out["dv"]), _ptr(workspace), _bytes(workspace), _current(dev))
        if cu_seqlens is not None:
            st = raw().gdn2_attn_bwd_varlen(*head, _ptr(cu_seqlens), *tail)
        else:
            st = raw().gdn2_attn_bwd(*head, *tail)
    _check("gdn2_attn_bwd" if cu_seqlens is None else "gdn2_attn_bwd_varlen", st)
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
    dev, dtype, shape = _device(k_cache), k_cache.dtype, k_cache.shape
    if len(shape) != 4 or block_table.dim() != 2:
        raise ValueError("k_cache and v_cache are [num_pages, page_size, Hkv, D], block_table is [N, max_pages]")
    if dtype is torch.bfloat16:
        kind = CACHE_BF16
    elif dtype is torch.float8_e4m3fn:
        kind = CACHE_E4M3
        if k_scale is None or v_scale is None:
            raise ValueError("an e4m3 cache has k_scale and v_scale")
        _need("k_scale", k_scale, torch.float32, shape[:3], dev)
        _need("v_scale", v_scale, torch.float32, shape[:3], dev)
    else:
        raise TypeError(f"unsupported cache dtype {dtype} (bfloat16 or float8_e4m3fn)")
    pages, page, Hkv, D = shape
    N, width = block_table.shape
    _need("k_cache", k_cache, dtype, shape, dev)
    _need("v_cache", v_cache, dtype, shape, dev)
    _need("block_table", block_table, torch.int32, (N, width), dev)
    _need("cu_seqlens", cu_seqlens, torch.int32, (N + 1,), dev)
    _need("kv_lens", kv_lens, torch.int32, (N,), dev)
    return dev, kind, N, Hkv, D, (width, pages, page)


def gdn2_cache_write(k, v, k_cache, v_cache, cu_seqlens, kv_lens, block_table, k_scale=None, v_scale=None, *,
                     stream=None):
    """Stores the new tokens' k and v [total_T, Hkv, D] in the paged cache [num_pages, page_size, Hkv, D]
    (bfloat16, or float8_e4m3fn with fp32 scales [num_pages, page_size, Hkv]).  Sequence n's rows are its
    last positions, kv_lens[n] counting them."""
    dev, kind, N, Hkv, D, sizes = _cache_args(k_cache, v_cache, cu_seqlens, kv_lens, block_table, k_scale, v_scale)
    T = k.shape[0]
    _need("k", k, torch.bfloat16, (T, Hkv, D), dev)
    _need("v", v, torch.bfloat16, (T, Hkv, D), dev)
    with _on(dev, stream):
        st = raw().gdn2_cache_write(kind, GDN2_BF16, N, T, Hkv, D, _ptr(cu_seqlens), _ptr(kv_lens), _ptr(block_table),
                                    *sizes, _ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale),
                                    _ptr(v_scale), _current(dev))
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
    with _on(dev, stream):
        if k is None:
            k = torch.empty(total_T, Hkv, D, dtype=torch.bfloat16, device=dev)
        if v is None:
            v = torch.empty_like(k)
        _need("k", k, torch.bfloat16, (total_T, Hkv, D), dev)
        _need("v", v, torch.bfloat16, (total_T, Hkv, D), dev)
        st = raw().gdn2_cache_read(kind, GDN2_BF16, N, total_T, Hkv, D, _ptr(cu_seqlens), _ptr(kv_lens),
                                   _ptr(block_table), *sizes, _ptr(k_cache), _ptr(v_cache), _ptr(k_scale),
                                   _ptr(v_scale), _ptr(k), _ptr(v), _current(dev))
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
    with _on(dev, stream):
        if o is None:
            o = torch.empty_like(q)
        else:
            _need("o", o, torch.bfloat16, (T, H, D), dev)
        if lse is not None:
            _need("lse", lse, torch.float32, (T, H), dev)
        elif want_lse:
            lse = torch.empty(T, H, dtype=torch.float32, device=dev)
        if workspace is None:
            workspace = _workspace(None, raw().gdn2_attn_cached_workspace_size(GDN2_BF16, N, T, H, Hkv, D, window,
                                                                               sizes[0], sizes[2]), dev)
        else:
            _workspace(workspace, 0, dev)
        st = raw().gdn2_attn_cached(kind, GDN2_BF16, N, T, H, Hkv, D, window, _scale(scale, D), _ptr(cu_seqlens),
                                    _ptr(kv_lens), _ptr(block_table), *sizes, _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                    _ptr(k_scale), _ptr(v_scale), _ptr(o), _ptr(lse), _ptr(workspace),
                                    _bytes(workspace), _current(dev))
    _check("gdn2_attn_cached", st)
    return o, lse
