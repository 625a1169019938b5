"""Per-head norm with rotation, forward and backward, against the 64-bit form.

Bounds: outputs are rounded once (2^-8 of a bf16 value, 2^-24 of an fp32 one); before that a row goes
through a dozen fp32 operations, each off by 2^-24, on channels no larger than the pair (a, b) they
mix: 2^-20 of the pair's magnitude covers them, and the sum of squares over 128 channels, whose
relative error of 2^-20 at most halves in the root."""
import pytest
import torch

import attn_ref as R

pytestmark = pytest.mark.gpu


def make(N, H, Hkv, D, rot, dt, far=5000, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return {"q": r(N, H, D).to(dt), "k": r(N, Hkv, D).to(dt), "wq": 1 + 0.2 * r(D), "wk": 1 + 0.2 * r(D),
            "pos": torch.randint(0, far, (N,), generator=g, dtype=torch.int32),
            "inv": torch.tensor([10000.0 ** (-2 * i / rot) for i in range(rot // 2)]) if rot else None,
            "dq": r(N, H, D).to(dt), "dk": r(N, Hkv, D).to(dt)}


def size_of(y, rot, interleaved):
    """The magnitude of the pair that each channel of y belongs to (rotation keeps it)."""
    out = y.abs().clone()
    if rot:
        z = y[..., :rot]
        z = z.unflatten(-1, (-1, 2)) if interleaved else z.unflatten(-1, (2, -1)).transpose(-1, -2)
        m = z.norm(dim=-1, keepdim=True).expand_as(z)
        out[..., :rot] = m.flatten(-2) if interleaved else m.transpose(-1, -2).flatten(-2)
    return out


def run(g, x, flags, eps=1e-6, rot_scale=1.0, backward=True, weights=True):
    c = {n: None if t is None else t.cuda() for n, t in x.items()}
    w = (c["wq"], c["wk"]) if weights else (None, None)
    qo, ko = g.gdn2_qk_rope(c["q"], c["k"], *w, c["pos"] if c["inv"] is not None else None, c["inv"], flags=flags, eps=eps, rot_scale=rot_scale)
    grads = g.gdn2_qk_rope_bwd(c["q"], c["k"], *w, c["pos"] if c["inv"] is not None else None, c["inv"], c["dq"], c["dk"], flags=flags, eps=eps,
                               rot_scale=rot_scale) if backward else None
    assert g.gdn2_sync_status() == 0
    return qo, ko, grads


def verify(x, flags, got, eps=1e-6, rot_scale=1.0, weights=True):
    norm, inter = bool(flags & 1), bool(flags & 2)
    rot = 0 if x["inv"] is None else 2 * x["inv"].numel()
    qo, ko, grads = got
    for name, o, w in (("q", qo, "wq"), ("k", ko, "wk")):
        a = x[name].double().requires_grad_()
        wt = x[w].double().requires_grad_() if weights else None
        y = R.rope(a, wt, x["pos"], x["inv"], inter, eps, rot_scale, norm)
        r = R.STEP[x[name].dtype]
        yd = y.detach()
        R.check(o, yd, r * yd.abs() + 2.0 ** -20 * size_of(yd, rot, inter) + 1e-30, name)
        if grads is None:
            continue
        dy = x["d" + name].double()
        inputs = (a, wt) if norm and weights else (a,)
        res = torch.autograd.grad(y, inputs, dy)
        dx = res[0]
        # dx = rr (g w - xh mean(g w xh)): both terms are bounded by rr max|w| |g| over the row
        rr = (torch.rsqrt((a.detach() ** 2).mean(-1, keepdim=True) + eps) if norm else 1.0) * max(1.0, abs(rot_scale))
        big = rr * dy.norm(dim=-1, keepdim=True) * (wt.detach().abs().max() if wt is not None else 1.0)
        R.check(grads["d" + name], dx, r * dx.abs() + 2.0 ** -19 * big.expand_as(dx) + 1e-30, "d" + name)
        if norm and weights:
            # sums over N H rows of terms of a few units, in fp32 in pieces
            terms = x[name].shape[0] * x[name].shape[1]
            xh = a.detach() * torch.rsqrt((a.detach() ** 2).mean(-1, keepdim=True) + eps)
            mag = (size_of(dy, rot, inter) * abs(rot_scale) * xh.abs()).sum((0, 1))
            R.check(grads["d" + name + "_weight"], res[1], (terms + 16) * 2.0 ** -24 * mag + 2.0 ** -19 * mag + 1e-30, "d" + w)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("flags", [0, 1, 2, 3])
def test_flags(cuda_lib, flags, D, dt):
    x = make(37, 5, 2, D, D, dt, seed=flags + D)
    verify(x, flags, run(cuda_lib, x, flags))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rot", [0, 2, 6, 16, 30, 32, 62, 64, 100, 126])
@pytest.mark.parametrize("inter", [0, 2])
def test_part_of_the_head(cuda_lib, rot, inter, dt):
    x = make(9, 3, 3, 128, rot, dt, seed=rot)
    verify(x, 1 | inter, run(cuda_lib, x, 1 | inter))


@pytest.mark.parametrize("N", [1, 7, 2047, 2048, 5003])
def test_rows(cuda_lib, N):
    """Either side of where a block's warps stop sharing a token, and grids that wrap around."""
    x = make(N, 3, 1, 64, 64, torch.bfloat16, seed=N)
    verify(x, 1, run(cuda_lib, x, 1))


@pytest.mark.parametrize("H,Hkv", [(1, 1), (32, 1), (2, 7), (17, 3)])
def test_heads(cuda_lib, H, Hkv):
    x = make(50, H, Hkv, 128, 128, torch.float32, seed=H)
    verify(x, 1, run(cuda_lib, x, 1))


@pytest.mark.parametrize("flags", [1, 3])
def test_far_positions(cuda_lib, flags):
    """Positions up to 2^31 - 1, and negative ones: the angle is reduced in 64 bits."""
    x = make(64, 2, 1, 128, 128, torch.float32, seed=3)
    x["pos"] = torch.tensor([2 ** 31 - 1, -2 ** 31, -1, 0] * 16, dtype=torch.int32)
    verify(x, flags, run(cuda_lib, x, flags))


def test_scaled_rotation_without_weights(cuda_lib):
    x = make(20, 4, 2, 64, 32, torch.float32, seed=6)
    got = run(cuda_lib, x, 1, eps=1e-3, rot_scale=1.375, weights=False)
    verify(x, 1, got, eps=1e-3, rot_scale=1.375, weights=False)


def test_zero_rows_and_extremes(cuda_lib):
    """A row of zeros gives zeros (eps keeps its root finite); large and tiny rows normalise."""
    x = make(8, 2, 1, 64, 64, torch.float32, seed=7)
    x["q"][0] = 0
    x["q"][1] *= 1e15
    x["q"][2] *= 1e-3
    got = run(cuda_lib, x, 1, backward=False)
    assert (got[0][0] == 0).all()
    verify(x, 1, got)


def test_in_place(cuda_lib):
    g = cuda_lib
    x = make(300, 4, 2, 128, 128, torch.bfloat16, seed=8)
    qo, ko, grads = run(g, x, 1)
    c = {n: t.cuda() for n, t in x.items()}
    q, k = c["q"].clone(), c["k"].clone()
    g.gdn2_qk_rope(q, k, c["wq"], c["wk"], c["pos"], c["inv"], q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko)
    out = {"dq": c["dq"].clone(), "dk": c["dk"].clone(), "dq_weight": None, "dk_weight": torch.empty(128, device="cuda")}
    g.gdn2_qk_rope_bwd(c["q"], c["k"], c["wq"], c["wk"], c["pos"], c["inv"], out["dq"], out["dk"], out=out)
    assert torch.equal(out["dq"], grads["dq"]) and torch.equal(out["dk"], grads["dk"])
    assert torch.equal(out["dk_weight"], grads["dk_weight"])


def test_leading_dimensions_and_no_rows(cuda_lib):
    g = cuda_lib
    x = make(24, 4, 2, 64, 64, torch.bfloat16, seed=9)
    qo, ko, _ = run(g, x, 1, backward=False)
    c = {n: t.cuda() for n, t in x.items()}
    q4, k4 = g.gdn2_qk_rope(c["q"].view(2, 12, 4, 64), c["k"].view(2, 12, 2, 64), c["wq"], c["wk"], c["pos"].view(2, 12), c["inv"])
    assert torch.equal(q4.flatten(0, 1), qo) and torch.equal(k4.flatten(0, 1), ko)
    e = g.gdn2_qk_rope_bwd(c["q"][:0], c["k"][:0], c["wq"], c["wk"], c["pos"][:0], c["inv"], c["dq"][:0], c["dk"][:0])
    assert (e["dq_weight"] == 0).all() and (e["dk_weight"] == 0).all()


def test_weight_gradient_is_repeatable_and_graphs(cuda_lib):
    g = cuda_lib
    x = make(3000, 8, 2, 128, 128, torch.bfloat16, seed=10)
    _, _, a = run(g, x, 1)
    c = {n: t.cuda() for n, t in x.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b = g.gdn2_qk_rope_bwd(c["q"], c["k"], c["wq"], c["wk"], c["pos"], c["inv"], c["dq"], c["dk"])
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for n in a:
        assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,Hkv", [(1, 3), (16, 5)])
def test_no_eps(cuda_lib, H, Hkv, dt):
    """eps 0 is allowed: passes that end past the last head add nothing to the weights' gradients."""
    x = make(40, H, Hkv, 128, 128, dt, seed=H)
    verify(x, 1, run(cuda_lib, x, 1, eps=0.0), eps=0.0)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("flags", [1, 3])
def test_far_scales_without_eps(cuda_lib, flags, dt):
    """Rows of 1e15 to 1e-16 with eps 0: 1 / rms goes from 1e-15 to 1e16, whose cubes fp32 does not hold."""
    x = make(9, 2, 1, 64, 64, torch.float32, seed=11)
    for n in ("q", "k"):
        x[n] *= torch.logspace(15, -16, 9)[:, None, None]
    x = {n: t.to(dt) if n in ("q", "k", "dq", "dk") else t for n, t in x.items()}
    verify(x, flags, run(cuda_lib, x, flags, eps=0.0), eps=0.0)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N", [511, 512, 513])
def test_rows_where_warps_stop_sharing(cuda_lib, N, dt):
    """The warps of a block share a token's heads below 512 tokens."""
    x = make(N, 19, 2, 64, 64, dt, seed=N)
    verify(x, 1, run(cuda_lib, x, 1))
