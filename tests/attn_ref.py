"""Plain 64-bit forms of the attention layer's operators, and bounds on how far a result may be off.

The bounds follow from the arithmetic, before any run.  Rounding to bf16 is off by at most half a step,
2^-8 of the value.  The bf16 kernels round, besides their outputs, the softmax weights p (and in the
backward p and ds) once to bf16; everything else is fp32, whose sums over n terms are off by at most
n 2^-24 of the sum of magnitudes.  With u the rounding of the weights (2^-8, or 0 for fp32), r that of
the output and a = (D + T + 64) 2^-23 for the fp32 sums and exponentials (twice the plain bound, for
the two products on the way):

    |d o|  <= (u + a + 2 t_i) sum_j p |v|              + r |o|
    |d dv| <= sum_i (u + a + 2 t_i) p |do|             + r |dv|
    e_ij    = (u + a + 2 t_i) |ds_ij| + p_ij (D_i + a E_ij),   E_ij = sum_c |do v| + sum_c |do o|
    t_i     = a max_j scale sum_c |q k| + small change: how far a score or the row's log-sum may be off.
              p = e^(s - lse), so with both off by t_i a weight is off by 2 t_i of itself.
    D_i     = sum_c |do| |d o|     (the backward is given the rounded o)
    |d dq| <= scale sum_j e_ij |k| + r |dq|,  |d dk| <= scale sum_i e_ij |q| + r |dk|
"""
import math

import torch

STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def lens_to_cu(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32)


def mask_of(first, nq, nk, window):
    i = first + torch.arange(nq)[:, None]
    j = torch.arange(nk)[None, :]
    m = j <= i
    return m & (j > i - window) if window else m


def head(q, k, v, first, window, scale, dt, do=None, weights=True):
    """One head in 64 bits: q [nq, D] at positions first .., k, v [nk, D].  Returns values and bounds."""
    q, k, v = q.double(), k.double(), v.double()
    r = STEP[dt]
    u = r if weights and dt == torch.bfloat16 else 0.0
    a = (q.shape[1] + k.shape[0] + 64) * 2.0 ** -23
    mask = mask_of(first, q.shape[0], k.shape[0], window)
    s = (scale * (q @ k.T)).masked_fill(~mask, -math.inf)
    lse = torch.logsumexp(s, 1)
    p = torch.exp(s - lse[:, None])
    p = torch.where(mask, p, 0.0)
    o = p @ v
    so = p @ v.abs()
    big = (scale * (q.abs() @ k.abs().T)).masked_fill(~mask, 0).amax(1)
    t = a * big + 2.0 ** -19 + 2.0 ** -22 * lse.abs()
    out = {"o": o, "lse": lse, "lse_tol": t, "o_tol": (u + a + 2 * t[:, None]) * so + r * o.abs() + 1e-30}
    if do is not None:
        do = do.double()
        dp = do @ v.T
        delta = (do * o).sum(1, keepdim=True)
        ds = p * (dp - delta)
        e = (u + a + 2 * t[:, None]) * ds.abs() + p * ((do.abs() * out["o_tol"]).sum(1, keepdim=True)
                                      + a * (do.abs() @ v.abs().T + (do * o).abs().sum(1, keepdim=True)))
        out["dv"], out["dv_abs"] = p.T @ do, (p * (u + a + 2 * t[:, None])).T @ do.abs()
        out["dq"], out["dq_abs"] = scale * ds @ k, scale * e @ k.abs()
        out["dk"], out["dk_abs"] = scale * ds.T @ q, scale * e.T @ q.abs()
    return out


def attention(q, k, v, spans, window, scale, do=None):
    """Packed q [rows, H, D], k, v [rows, Hkv, D] over spans [(first row, rows)]: values and bounds in the
    kernels' layouts.  Rows of no span are NaN."""
    H, Hkv, D = q.shape[1], k.shape[1], q.shape[2]
    G, dt = H // Hkv, q.dtype
    r = STEP[dt]
    nan = float("nan")
    out = {n: torch.full(q.shape, nan, dtype=torch.float64) for n in ("o", "o_tol", "dq", "dq_tol")}
    out.update({n: torch.full(q.shape[:2], nan, dtype=torch.float64) for n in ("lse", "lse_tol")})
    out.update({n: torch.full(k.shape, nan, dtype=torch.float64) for n in ("dk", "dk_tol", "dv", "dv_tol")})
    for b, n in spans:
        if n == 0:
            continue
        rows = slice(b, b + n)
        if do is not None:
            for x in ("dk", "dk_tol", "dv", "dv_tol"):
                out[x][rows] = 0
        for h in range(H):
            g = h // G
            x = head(q[rows, h], k[rows, g], v[rows, g], 0, window, scale, dt, None if do is None else do[rows, h])
            for name in ("o", "o_tol", "lse", "lse_tol"):
                out[name][rows, h] = x[name]
            if do is not None:
                out["dq"][rows, h] = x["dq"]
                out["dq_tol"][rows, h] = x["dq_abs"] + r * x["dq"].abs() + 1e-30
                for name in ("dk", "dv"):
                    out[name][rows, g] += x[name]
                    out[name + "_tol"][rows, g] += x[name + "_abs"]
        if do is not None:
            for name in ("dk", "dv"):
                out[name + "_tol"][rows] += r * out[name][rows].abs() + 1e-30
    return out


def check(got, ref, tol, name):
    """Every element within its bound; both sides share NaN rows (rows of no sequence are not compared)."""
    got = got.detach().cpu().double()
    live = ~torch.isnan(ref)
    assert torch.isfinite(got[live]).all(), f"{name}: non-finite values"
    over = ((got - ref).abs() / tol)[live]
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 1.0, f"{name}: {worst:.2f} times its bound"
    return worst


def rope(x, weight, pos, inv, interleaved, eps, rot_scale, norm):
    """y in 64 bits of x [N, H, D]."""
    x = x.double()
    if norm:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        if weight is not None:
            x = x * weight.double()
    if inv is None or inv.numel() == 0:
        return x
    rot = 2 * inv.numel()
    ang = pos.double()[:, None, None] * inv.double()
    c, s = rot_scale * ang.cos(), rot_scale * ang.sin()
    z = x[..., :rot]
    z = z.unflatten(-1, (-1, 2)) if interleaved else z.unflatten(-1, (2, -1)).transpose(-1, -2)
    a, b = z[..., 0], z[..., 1]
    z = torch.stack([a * c - b * s, b * c + a * s], -1)
    z = z.flatten(-2) if interleaved else z.transpose(-1, -2).flatten(-2)
    return torch.cat([z, x[..., rot:]], -1)


def e4m3(x):
    """Nearest e4m3 value (ties to even) of |x| <= 448 in 64 bits."""
    x = x.double()
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def quantise(x):
    """A row's e4m3 values and fp32 scale as the cache defines them, of rows x [.., D]; exact divisions in
    fp32.  Non-finite channels become NaN and do not count for the scale."""
    x = x.float()
    fine = torch.isfinite(x)
    top = torch.where(fine, x.abs(), 0).amax(-1)
    scale = top / 448
    y = torch.where(scale[..., None] > 0, x / torch.where(scale > 0, scale, 1)[..., None], 0.0)
    return torch.where(fine, e4m3(y.clamp(-448, 448)), float("nan")), scale
