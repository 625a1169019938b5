"""Causal attention over whole sequences, forward and backward, against the 64-bit form."""
import pytest
import torch

import attn_ref as R

pytestmark = pytest.mark.gpu


def make(lens, H, Hkv, D, dt, seed=0, tail=0, sd=1.0):
    g = torch.Generator().manual_seed(seed)
    n = sum(lens) + tail
    x = {m: (sd * torch.randn(n, h, D, generator=g)).to(dt) for m, h in (("q", H), ("k", Hkv), ("v", Hkv), ("do", H))}
    spans, at = [], 0
    for m in lens:
        spans.append((at, m))
        at += m
    return x, spans


def run_packed(g, x, lens, window, scale, backward=True, out=None):
    d = {n: t.cuda() for n, t in x.items()}
    cu = R.lens_to_cu(lens).cuda()
    o, lse = g.gdn2_attn_fwd_varlen(d["q"], d["k"], d["v"], cu, window=window, scale=scale)
    grads = {}
    if backward:
        grads = g.gdn2_attn_bwd_varlen(d["q"], d["k"], d["v"], o, lse, d["do"], cu, window=window, scale=scale, out=out)
    assert g.gdn2_sync_status() == 0
    return {"o": o, "lse": lse, **grads}


def compare(got, x, spans, window, scale):
    ref = R.attention(x["q"], x["k"], x["v"], spans, window, scale, x["do"] if "dq" in got else None)
    for n in ("o", "lse", "dq", "dk", "dv"):
        if n in got:
            R.check(got[n], ref[n], ref[n + "_tol"], n)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[1], [2, 1], [127], [128], [129, 0, 1], [255, 256, 257], [300, 64, 37]])
def test_lengths(cuda_lib, lens, D, dt):
    x, spans = make(lens, 2, 1, D, dt, seed=len(lens) + lens[0])
    compare(run_packed(cuda_lib, x, lens, 0, D ** -0.5), x, spans, 0, D ** -0.5)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (4, 4), (3, 1), (8, 2), (5, 1), (14, 2), (64, 1), (16, 16)])
def test_heads(cuda_lib, H, Hkv, dt):
    lens = [140, 3, 61]
    x, spans = make(lens, H, Hkv, 64, dt, seed=H)
    compare(run_packed(cuda_lib, x, lens, 0, 0.125), x, spans, 0, 0.125)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("window", [1, 2, 63, 64, 128, 129, 200, 100000, 2 ** 31 - 1])
def test_windows(cuda_lib, window, dt):
    lens = [390, 5, 129]
    x, spans = make(lens, 4, 2, 128, dt, seed=window % 97)
    compare(run_packed(cuda_lib, x, lens, window, 0.1), x, spans, window, 0.1)


def test_many_sequences(cuda_lib):
    """More sequences than a warp looks up at a time, empty ones among them."""
    lens = [(7 * i) % 23 for i in range(75)] + [0, 0, 150, 0]
    x, spans = make(lens, 2, 2, 64, torch.bfloat16, seed=5)
    compare(run_packed(cuda_lib, x, lens, 0, 0.125), x, spans, 0, 0.125)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_fixed_length_equals_packed(cuda_lib, dt):
    g = cuda_lib
    B, T = 3, 150
    x, spans = make([T] * B, 4, 2, 64, dt, seed=2)
    got = run_packed(g, x, [T] * B, 33, 0.125)
    d = {n: t.cuda().view(B, T, *t.shape[1:]) for n, t in x.items()}
    o, lse = g.gdn2_attn_fwd(d["q"], d["k"], d["v"], window=33)
    grads = g.gdn2_attn_bwd(d["q"], d["k"], d["v"], o, lse, d["do"], window=33)
    assert g.gdn2_sync_status() == 0
    assert torch.equal(o.flatten(0, 1), got["o"]) and torch.equal(lse.flatten(0, 1), got["lse"])
    for n in ("dq", "dk", "dv"):
        assert torch.equal(grads[n].flatten(0, 1), got[n]), n


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_large_scores(cuda_lib, dt):
    """Scores of a few hundred: the running maximum moves far, and most weights underflow."""
    lens = [300]
    x, spans = make(lens, 2, 1, 128, dt, seed=9, sd=3.0)
    x["k"][::7] *= 4
    compare(run_packed(cuda_lib, x, lens, 0, 0.5, backward=False), x, spans, 0, 0.5)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_rising_scores(cuda_lib, dt):
    """Every later key scores higher than all before it: the reference moves in every tile."""
    n, D = 520, 64
    x, spans = make([n], 1, 1, D, dt, seed=1)
    x["q"][:] = 1
    x["k"][:] = (torch.arange(n) / 16)[:, None, None].to(dt)
    compare(run_packed(cuda_lib, x, [n], 0, 0.125), x, spans, 0, 0.125)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_rows_behind_the_last_sequence(cuda_lib, dt):
    """A padded batch: rows past cu_seqlens[-1] hold NaN and stay as they were in every output."""
    g = cuda_lib
    lens, tail = [70, 131], 90
    x, spans = make(lens, 4, 2, 64, dt, seed=3, tail=tail)
    for t in x.values():
        t[sum(lens):] = float("nan")
    d = {n: t.cuda() for n, t in x.items()}
    cu = R.lens_to_cu(lens).cuda()
    o = torch.full_like(d["q"], 7.0)
    lse = torch.full(o.shape[:2], 7.0, device="cuda")
    g.gdn2_attn_fwd_varlen(d["q"], d["k"], d["v"], cu, scale=0.125, o=o, lse=lse)
    out = {"dq": torch.full_like(d["q"], 7.0), "dk": torch.full_like(d["k"], 7.0), "dv": torch.full_like(d["v"], 7.0)}
    g.gdn2_attn_bwd_varlen(d["q"], d["k"], d["v"], o, lse, d["do"], cu, scale=0.125, out=out)
    assert g.gdn2_sync_status() == 0
    got = {"o": o, "lse": lse, **out}
    for n, t in got.items():
        assert (t[sum(lens):] == 7.0).all(), n
    compare(got, x, spans, 0, 0.125)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_neighbours_do_not_leak(cuda_lib, dt, bad):
    """A sequence of non-finite values leaves its neighbours in the batch untouched."""
    g = cuda_lib
    lens = [130, 77, 150]
    x, _ = make(lens, 4, 2, 128, dt, seed=4)
    clean = run_packed(g, x, lens, 0, 0.1)
    for t in x.values():
        t[130:207] = bad
    dirty = run_packed(g, x, lens, 0, 0.1)
    for n in clean:
        for rows in (slice(0, 130), slice(207, None)):
            assert torch.equal(clean[n][rows], dirty[n][rows]), n


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_repeatable(cuda_lib, dt):
    x, _ = make([700, 300], 8, 2, 128, dt, seed=6)
    a = run_packed(cuda_lib, x, [700, 300], 0, 0.1)
    b = run_packed(cuda_lib, x, [700, 300], 0, 0.1)
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_gradients_against_differences(cuda_lib):
    """fp32 gradients against central differences of the kernel's own forward in random directions.
    h = 2^-6: the difference's truncation is h^2/6 of the third derivative (below 1e-4 of the
    directional derivative's scale here), its rounding about 1e-6 / h."""
    g = cuda_lib
    x, _ = make([37], 2, 1, 64, torch.float32, seed=8, sd=0.5)
    d = {n: t.cuda() for n, t in x.items()}
    cu = R.lens_to_cu([37]).cuda()

    def loss(q, k, v):
        o, _ = g.gdn2_attn_fwd_varlen(q, k, v, cu, window=20)
        return float((o.double() * d["do"].double()).sum())

    o, lse = g.gdn2_attn_fwd_varlen(d["q"], d["k"], d["v"], cu, window=20)
    grads = g.gdn2_attn_bwd_varlen(d["q"], d["k"], d["v"], o, lse, d["do"], cu, window=20)
    h = 2.0 ** -6
    for n in ("q", "k", "v"):
        gen = torch.Generator().manual_seed(11)
        for _ in range(3):
            e = torch.randn(d[n].shape, generator=gen).cuda()
            up = loss(**{m: d[m] + h * e if m == n else d[m] for m in ("q", "k", "v")})
            dn = loss(**{m: d[m] - h * e if m == n else d[m] for m in ("q", "k", "v")})
            num, ana = (up - dn) / (2 * h), float((grads["d" + n].double() * e.double()).sum())
            size = float(grads["d" + n].double().norm())
            assert abs(num - ana) <= 5e-3 * size, (n, num, ana)


def test_invalid_seqlens_are_reported(cuda_lib):
    g = cuda_lib
    x, _ = make([200], 2, 1, 64, torch.bfloat16)
    d = {n: t.cuda() for n, t in x.items()}
    for bad in ([0, 150, 100], [0, 100, 201], [3, 100, 200]):
        o = torch.full_like(d["q"], 7.0)
        lse = torch.full(o.shape[:2], 7.0, device="cuda")
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        g.gdn2_attn_fwd_varlen(d["q"], d["k"], d["v"], cu, o=o, lse=lse)
        assert g.gdn2_sync_status() == -10
    g.gdn2_attn_fwd_varlen(d["q"], d["k"], d["v"], R.lens_to_cu([200]).cuda())
    assert g.gdn2_sync_status() == 0


def test_streams_and_graphs(cuda_lib):
    """On a stream of its own, and captured and replayed on new inputs in the same buffers."""
    g = cuda_lib
    x, spans = make([260, 40], 4, 2, 128, torch.bfloat16, seed=12)
    want = run_packed(g, x, [260, 40], 0, 0.1)
    d = {n: t.cuda() for n, t in x.items()}
    cu = R.lens_to_cu([260, 40]).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, lse = g.gdn2_attn_fwd_varlen(d["q"], d["k"], d["v"], cu, scale=0.1, stream=side)
    grads = g.gdn2_attn_bwd_varlen(d["q"], d["k"], d["v"], o, lse, d["do"], cu, scale=0.1, stream=side)
    side.synchronize()
    for n, t in (("o", o), ("lse", lse), *grads.items()):
        assert torch.equal(t, want[n]), n
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = g.gdn2_attn_fwd_varlen(d["q"], d["k"], d["v"], cu, scale=0.1)
        grads = g.gdn2_attn_bwd_varlen(d["q"], d["k"], d["v"], o, lse, d["do"], cu, scale=0.1)
    y, _ = make([260, 40], 4, 2, 128, torch.bfloat16, seed=13)
    want = run_packed(g, y, [260, 40], 0, 0.1)
    for n in d:
        d[n].copy_(y[n])
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for n, t in (("o", o), ("lse", lse), *grads.items()):
        assert torch.equal(t, want[n]), n


BAD_SEQLENS = [
    # entries, rows, the sequences that are valid by their own two entries
    ([0, 150, 100], [(0, 150)]),
    ([0, 100, 201], [(0, 100)]),
    ([3, 100, 200], [(100, 100)]),
    ([0, -5, 100, 200], [(100, 100)]),
    ([0, 40, 2 ** 31 - 1, 200], [(0, 40)]),
    ([0, -2 ** 31, -2 ** 31], []),
    # more sequences than a warp looks up at a time, an entry in the middle
    ([0] + [5 * i if i != 21 else -1 for i in range(1, 41)], [(5 * i, 5) for i in range(40) if i not in (20, 21)]),
    ([0] + [5 * i if i != 37 else 201 for i in range(1, 41)], [(5 * i, 5) for i in range(40) if i not in (36, 37)]),
]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("window", [0, 30])
@pytest.mark.parametrize("case", range(len(BAD_SEQLENS)))
def test_invalid_sequences_are_skipped(cuda_lib, case, window, dt):
    """Forward and backward leave the rows of a sequence with invalid entries as they were; the valid ones
    are as without it."""
    g = cuda_lib
    entries, spans = BAD_SEQLENS[case]
    x, _ = make([200], 4, 2, 64, dt, seed=case)
    d = {n: t.cuda() for n, t in x.items()}
    cu = torch.tensor(entries, dtype=torch.int32, device="cuda")
    o, lse = torch.full_like(d["q"], 7.0), torch.full(d["q"].shape[:2], 7.0, device="cuda")
    g.gdn2_attn_fwd_varlen(d["q"], d["k"], d["v"], cu, window=window, scale=0.125, o=o, lse=lse)
    assert g.gdn2_sync_status() == -10
    out = {"dq": torch.full_like(d["q"], 7.0), "dk": torch.full_like(d["k"], 7.0), "dv": torch.full_like(d["v"], 7.0)}
    g.gdn2_attn_bwd_varlen(d["q"], d["k"], d["v"], o, lse, d["do"], cu, window=window, scale=0.125, out=out)
    assert g.gdn2_sync_status() == -10
    skipped = torch.ones(200, dtype=torch.bool)
    for b, n in spans:
        skipped[b:b + n] = False
    got = {"o": o, "lse": lse, **out}
    for n, t in got.items():
        assert (t.cpu()[skipped] == 7.0).all(), n
    compare(got, x, spans, window, 0.125)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hkv,window", [(16, 16, 0), (32, 16, 0), (16, 16, 45)])
def test_fp32_batches_that_fill_the_device(cuda_lib, H, Hkv, window, D):
    """fp32 keys by 32 to a block, which batches of at least two blocks to an SM take."""
    lens = [333, 1, 260, 47]
    x, spans = make(lens, H, Hkv, D, torch.float32, seed=D + H)
    compare(run_packed(cuda_lib, x, lens, window, D ** -0.5), x, spans, window, D ** -0.5)
