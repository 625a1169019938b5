"""The attention layer's operators together, as training and serving use them, next to the recurrence."""
import pytest
import torch

import attn_ref as R

pytestmark = pytest.mark.gpu
H, HKV, D, ROT = 8, 2, 64, 32
INV = torch.tensor([10000.0 ** (-2 * i / ROT) for i in range(ROT // 2)])


def weights(seed):
    g = torch.Generator().manual_seed(seed)
    return 1 + 0.1 * torch.randn(D, generator=g), 1 + 0.1 * torch.randn(D, generator=g)


def tokens(n, seed, dt=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(n, h, D, generator=g).to(dt) for h in (H, HKV, HKV, H)]


def positions(lens):
    return torch.cat([torch.arange(n, dtype=torch.int32) for n in lens])


@pytest.mark.parametrize("window", [0, 50])
def test_training_step_fp32(cuda_lib, window):
    """Norm, rotation and attention forward, and the gradients back to q, k, v and the norm's weights,
    against autograd in 64 bits.  fp32 throughout: the bound is the framework's 1e-4 of the largest."""
    g = cuda_lib
    lens = [70, 1, 129]
    q, k, v, do = tokens(sum(lens), 1, torch.float32)
    wq, wk = weights(2)
    pos = positions(lens)
    c = lambda *x: [t.cuda() for t in x]  # noqa: E731
    dq_, dk_, dv_, ddo, dwq_, dwk_, dpos, dinv = c(q, k, v, do, wq, wk, pos, INV)
    cu = R.lens_to_cu(lens).cuda()
    qr, kr = g.gdn2_qk_rope(dq_, dk_, dwq_, dwk_, dpos, dinv)
    o, lse = g.gdn2_attn_fwd_varlen(qr, kr, dv_, cu, window=window)
    ga = g.gdn2_attn_bwd_varlen(qr, kr, dv_, o, lse, ddo, cu, window=window)
    gr = g.gdn2_qk_rope_bwd(dq_, dk_, dwq_, dwk_, dpos, dinv, ga["dq"], ga["dk"])
    assert g.gdn2_sync_status() == 0

    leaves = [t.double().requires_grad_() for t in (q, k, v, wq, wk)]
    a, b, vv, aw, bw = leaves
    qq, kk = R.rope(a, aw, pos, INV, False, 1e-6, 1.0, True), R.rope(b, bw, pos, INV, False, 1e-6, 1.0, True)
    outs, at = [], 0
    for n in lens:
        s = torch.einsum("qhd,khd->hqk", qq[at:at + n], kk[at:at + n].repeat_interleave(H // HKV, 1)) * D ** -0.5
        s = s.masked_fill(~R.mask_of(0, n, n, window), -float("inf"))
        outs.append(torch.einsum("hqk,khd->qhd", torch.softmax(s, -1), vv[at:at + n].repeat_interleave(H // HKV, 1)))
        at += n
    ref = torch.cat(outs)
    grads = torch.autograd.grad(ref, leaves, do.double())
    got = (gr["dq"], gr["dk"], ga["dv"], gr["dq_weight"], gr["dk_weight"])
    for name, x, y in zip(("o", "dq", "dk", "dv", "dwq", "dwk"), (o, *got), (ref.detach(), *grads)):
        err = float((x.cpu().double() - y).abs().max() / y.abs().max())
        assert err <= 1e-4, (name, err)


@pytest.mark.parametrize("e4m3", [False, True])
def test_serving_equals_the_prompt(cuda_lib, e4m3):
    """A prompt written to the cache in chunks and then token by token, each step's attention against the
    64-bit attention over what the cache holds; with a bf16 cache that is the whole-prompt attention."""
    g = cuda_lib
    lens, page = [150, 37], 16
    steps = [[64, 20], [70, 1], [1, 1], [1, 0], [14, 15]]  # new tokens of each sequence, summing to lens
    q, k, v, _ = tokens(sum(lens), 3)
    wq, wk = weights(4)
    pos = positions(lens)
    qr, kr = (t.cpu() for t in g.gdn2_qk_rope(q.cuda(), k.cuda(), wq.cuda(), wk.cuda(), pos.cuda(), INV.cuda()))
    width = -(-max(lens) // page)
    dt = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    kc, vc = (torch.zeros(2 * width, page, HKV, D, dtype=dt, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(2 * width, page, HKV, device="cuda") if e4m3 else None for _ in range(2))
    table = torch.randperm(2 * width, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(2, width).cuda()
    held = lambda x: (lambda y, s: y * s.double()[..., None])(*R.quantise(x)) if e4m3 else x.double()  # noqa: E731
    off, done, o_all, lse_all = [0, lens[0]], [0, 0], torch.empty_like(q), torch.empty(sum(lens), H)
    for step in steps:
        rows = torch.cat([torch.arange(off[i] + done[i], off[i] + done[i] + n) for i, n in enumerate(step)])
        done = [a + b for a, b in zip(done, step)]
        cu, kv = R.lens_to_cu(step).cuda(), torch.tensor(done, dtype=torch.int32).cuda()
        g.gdn2_cache_write(kr[rows].cuda(), v[rows].cuda(), kc, vc, cu, kv, table, ks, vs)
        o, lse = g.gdn2_attn_cached(qr[rows].cuda(), kc, vc, cu, kv, table, ks, vs)
        assert g.gdn2_sync_status() == 0
        o_all[rows], lse_all[rows] = o.cpu(), lse.cpu()
    assert done == lens
    for i, n in enumerate(lens):
        r = slice(off[i], off[i] + n)
        kk, vv = held(kr[r]), held(v[r])
        for h in range(H):
            x = R.head(qr[r, h], kk[:, h // (H // HKV)], vv[:, h // (H // HKV)], 0, 0, D ** -0.5, torch.bfloat16)
            R.check(o_all[r, h], x["o"], x["o_tol"], "o")
            R.check(lse_all[r, h], x["lse"], x["lse_tol"], "lse")
    # the cache read back gives what was written
    kb, vb = g.gdn2_cache_read(kc, vc, R.lens_to_cu(lens).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), table, ks, vs,
                               total_T=sum(lens))
    assert torch.equal(kb.cpu(), held(kr).float().bfloat16()) and torch.equal(vb.cpu(), held(v).float().bfloat16())
    # a chunk of the read-back rows through the whole-sequence call
    o, _ = g.gdn2_attn_fwd_varlen(qr.cuda(), kb, vb, R.lens_to_cu(lens).cuda())
    ref = R.attention(qr, kb.cpu(), vb.cpu(), [(0, lens[0]), (lens[0], lens[1])], 0, D ** -0.5)
    R.check(o, ref["o"], ref["o_tol"], "o over the read-back cache")


def test_next_to_the_recurrence(cuda_lib):
    """A recurrent layer's output as the values of an attention layer, in one captured graph, replayed on
    new inputs: the same as the calls made one by one."""
    from synthetic_inputs import make_inputs
    g = cuda_lib
    B, T = 1, 200

    def inputs(seed):
        x = make_inputs(B, T, HKV, D, D, dtype="bf16", seed=seed)
        q, k, _, _ = tokens(T, seed)
        return {**{n: x[n] for n in ("q", "k", "v", "log_alpha", "b", "w")}, "aq": q[None], "ak": k[None]}

    pos, inv = torch.arange(T, dtype=torch.int32).view(1, T).cuda(), INV.cuda()
    wq, wk = (t.cuda() for t in weights(5))

    def layer(x):
        y, _ = g.gdn2_chunk_fwd(x["q"], x["k"], x["v"], x["log_alpha"], x["b"], x["w"])
        a, b = g.gdn2_qk_rope(x["aq"], x["ak"], wq, wk, pos, inv)
        o, lse = g.gdn2_attn_fwd(a, b, y, window=64)
        gr = g.gdn2_attn_bwd(a, b, y, o, lse, o, window=64)
        return o, gr["dv"], *g.gdn2_qk_rope_bwd(x["aq"], x["ak"], wq, wk, pos, inv, gr["dq"], gr["dk"]).values()

    x = {n: t.cuda() for n, t in inputs(1).items()}
    eager = layer(x)  # an eager step's tensors live on while the graph is captured
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(x)
    new = inputs(2)
    for n in x:
        x[n].copy_(new[n])
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    want = layer({n: t.cuda() for n, t in new.items()})
    assert g.gdn2_sync_status() == 0
    for a, b, e in zip(out, want, eager):
        assert torch.equal(a, b) and not torch.equal(a, e)


def test_calls_on_two_streams_at_once(cuda_lib):
    """Independent calls of every operator on two streams together: the same as one after the other."""
    g = cuda_lib
    lens = [300, 41]
    cu = R.lens_to_cu(lens).cuda()
    pos, inv = positions(lens).cuda(), INV.cuda()
    kv = torch.tensor(lens, dtype=torch.int32).cuda()
    table = torch.arange(2 * 19, dtype=torch.int32).view(2, 19).cuda()

    def run(x, stream):
        q, k, v, do = x
        a, b = g.gdn2_qk_rope(q, k, None, None, pos, inv, stream=stream)
        o, lse = g.gdn2_attn_fwd_varlen(a, b, v, cu, stream=stream)
        gr = g.gdn2_attn_bwd_varlen(a, b, v, o, lse, do, cu, stream=stream)
        rb = g.gdn2_qk_rope_bwd(q, k, None, None, pos, inv, gr["dq"], gr["dk"], stream=stream)
        with torch.cuda.stream(stream):
            kc, vc = (torch.zeros(38, 16, HKV, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        g.gdn2_cache_write(b, v, kc, vc, cu, kv, table, stream=stream)
        oc, _ = g.gdn2_attn_cached(a, kc, vc, cu, kv, table, stream=stream)
        return [o, lse, gr["dv"], *rb.values(), oc, kc]

    xs = [[t.cuda() for t in tokens(sum(lens), s)] for s in (10, 11)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    together = [run(x, s) for x, s in zip(xs, streams) for _ in range(1)]
    torch.cuda.synchronize()
    for x, got in zip(xs, together):
        for a, b in zip(run(x, streams[0]), got):
            streams[0].synchronize()
            assert torch.equal(a, b)
    assert g.gdn2_sync_status() == 0


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("rows", [1, 40])
def test_cache_past_32_bit_offsets(cuda_lib, rows, e4m3):
    """Pages whose elements and bytes lie past 2^32: written, read back, attended to."""
    g = cuda_lib
    hkv, d, page, pages = 8, 128, 64, 66000 if e4m3 else 34000  # 4.3e9 and 2.2e9 elements a tensor
    dt = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    kc, vc = (torch.empty(pages, page, hkv, d, dtype=dt, device="cuda") for _ in range(2))
    ks, vs = (torch.empty(pages, page, hkv, device="cuda") if e4m3 else None for _ in range(2))
    n = 200
    table = torch.tensor([[pages - 1, 0, pages - 2, pages - 3]], dtype=torch.int32).cuda()
    gen = torch.Generator().manual_seed(1)
    k, v = (torch.randn(n, hkv, d, generator=gen).bfloat16() for _ in range(2))
    q = torch.randn(rows, hkv, d, generator=gen).bfloat16()
    kv, cu = torch.tensor([n], dtype=torch.int32).cuda(), R.lens_to_cu([n]).cuda()
    g.gdn2_cache_write(k.cuda(), v.cuda(), kc, vc, cu, kv, table, ks, vs)
    kb, vb = (t.cpu() for t in g.gdn2_cache_read(kc, vc, cu, kv, table, ks, vs, total_T=n))
    o, lse = g.gdn2_attn_cached(q.cuda(), kc, vc, R.lens_to_cu([rows]).cuda(), kv, table, ks, vs)
    assert g.gdn2_sync_status() == 0
    held = [(lambda y, s: y * s.double()[..., None])(*R.quantise(x)) if e4m3 else x.double() for x in (k, v)]
    for got, x in zip((kb, vb), held):
        assert torch.equal(got, x.float().bfloat16())
    for h in range(hkv):
        x = R.head(q[:, h], held[0][:, h], held[1][:, h], n - rows, 0, d ** -0.5, torch.bfloat16)
        R.check(o[:, h], x["o"], x["o_tol"], "o")
        R.check(lse[:, h], x["lse"], x["lse_tol"], "lse")


def test_stale_rows_behind_a_sequence_do_not_matter(cuda_lib):
    """What lies behind a sequence in its last page (here NaN) changes nothing, bit for bit, for one token
    and for a chunk, by box and by copy."""
    g = cuda_lib
    for page in (64, 7):
        for rows in (1, 60):
            n = 75
            gen = torch.Generator().manual_seed(rows)
            k, v, q = (torch.randn(m, HKV, D, generator=gen).bfloat16().cuda() for m in (n, n, rows))
            pages = -(-n // page)
            table = torch.arange(pages, dtype=torch.int32).view(1, -1).cuda()
            outs = []
            for fill in (0.0, float("nan"), float("inf")):
                kc, vc = (torch.full((pages, page, HKV, D), fill, dtype=torch.bfloat16, device="cuda") for _ in range(2))
                kv = torch.tensor([n], dtype=torch.int32).cuda()
                g.gdn2_cache_write(k, v, kc, vc, R.lens_to_cu([n]).cuda(), kv, table)
                outs.append(g.gdn2_attn_cached(q, kc, vc, R.lens_to_cu([rows]).cuda(), kv, table)[0])
            assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2]), (page, rows)


def at_16(t):
    """t's values at an address that 16 divides and 32 does not, which is all that the entry points ask for."""
    n = t.numel() * t.element_size()
    raw = torch.empty(n + 64, dtype=torch.uint8, device="cuda")
    at = (16 - raw.data_ptr()) % 32
    x = raw[at:at + n].view(t.dtype).view(t.shape)
    assert x.data_ptr() % 32 == 16
    return x.copy_(t)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 128])
def test_tensors_aligned_to_16_bytes_only(cuda_lib, D, dt):
    """Rotation and attention, forward and backward, with every tensor and workspace at an odd multiple of
    16 bytes: bit for bit what they give elsewhere."""
    g = cuda_lib
    lens, gen = [150, 37], torch.Generator().manual_seed(7)
    q, k, v, do = (torch.randn(sum(lens), h, D, generator=gen).to(dt).cuda() for h in (H, HKV, HKV, H))
    w, inv, pos, cu = torch.ones(D).cuda(), INV.cuda(), positions(lens).cuda(), R.lens_to_cu(lens).cuda()

    def calls(f, e):
        a, b, c, d, ww, pp, ii, cc = (f(t) for t in (q, k, v, do, w, pos, inv, cu))
        qr, kr = g.gdn2_qk_rope(a, b, ww, ww, pp, ii, q_out=e(a), k_out=e(b))
        lse = e(torch.empty(sum(lens), H, device="cuda"))
        o, _ = g.gdn2_attn_fwd_varlen(qr, kr, c, cc, o=e(a), lse=lse)
        ws = e(torch.empty(g.gdn2_attn_workspace_size(dt, len(lens), max(lens), H, HKV, D), dtype=torch.uint8, device="cuda"))
        ga = g.gdn2_attn_bwd_varlen(qr, kr, c, o, lse, d, cc, out={"dq": e(a), "dk": e(b), "dv": e(c)}, workspace=ws)
        gr = g.gdn2_qk_rope_bwd(a, b, ww, ww, pp, ii, ga["dq"], ga["dk"])
        assert g.gdn2_sync_status() == 0
        return [qr, kr, o, lse, *(ga[n] for n in ("dq", "dk", "dv")), *(gr[n] for n in ("dq", "dk", "dq_weight", "dk_weight"))]

    for x, y in zip(calls(lambda t: t, torch.empty_like), calls(at_16, lambda t: at_16(torch.zeros_like(t)))):
        assert torch.equal(x, y)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,page", [([1, 2], 16), ([150, 37], 16), ([150, 37], 12)])
def test_cache_aligned_to_16_bytes_only(cuda_lib, lens, page, D, e4m3):
    """... and the cache's calls: few and many rows, with and without a split key axis."""
    g = cuda_lib
    gen = torch.Generator().manual_seed(8)
    kv = [n + 600 for n in lens]
    q, k, v = (torch.randn(n, h, D, generator=gen).bfloat16().cuda() for n, h in ((sum(lens), H), (sum(kv), HKV), (sum(kv), HKV)))
    width = -(-max(kv) // page)
    table = torch.arange(2 * width, dtype=torch.int32).view(2, width).cuda()
    dt = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    cus, kvs = [R.lens_to_cu(n).cuda() for n in (lens, kv)], torch.tensor(kv, dtype=torch.int32).cuda()

    def calls(f, e):
        kc, vc = (f(torch.zeros(2 * width * page * HKV * D, dtype=torch.uint8, device="cuda").view(torch.uint8)
                    if e4m3 else torch.zeros(2 * width * page * HKV * D, dtype=torch.bfloat16, device="cuda"))
                  .view(dt).view(2 * width, page, HKV, D) for _ in range(2))
        ks, vs = (f(torch.zeros(2 * width, page, HKV, device="cuda")) if e4m3 else None for _ in range(2))
        a, b, c, t, n, c0, c1 = (f(x) for x in (q, k, v, table, kvs, *cus))
        g.gdn2_cache_write(b, c, kc, vc, c1, n, t, ks, vs)
        kb, vb = g.gdn2_cache_read(kc, vc, c1, n, t, ks, vs, k=e(b), v=e(c))
        out = [kb, vb]
        for window in (0, 40):
            ws = e(torch.empty(max(16, g.gdn2_attn_cached_workspace_size(2, sum(lens), H, HKV, D, window, width, page)),
                               dtype=torch.uint8, device="cuda"))
            out += g.gdn2_attn_cached(a, kc, vc, c0, n, t, ks, vs, window=window, o=e(a),
                                      lse=e(torch.empty(sum(lens), H, device="cuda")), workspace=ws)
        assert g.gdn2_sync_status() == 0
        return out

    for x, y in zip(calls(lambda t: t, torch.empty_like), calls(at_16, lambda t: at_16(torch.zeros_like(t)))):
        assert torch.equal(x, y)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [0, 70])
def test_many_short_sequences(cuda_lib, window, D):
    """A long packed batch, several tiles of keys and of queries to a block, each found by a search that
    takes longer than the tile before it."""
    g = cuda_lib
    gen = torch.Generator().manual_seed(11)
    lens = torch.randint(0, 40, (1500,), generator=gen).tolist()
    lens[700], lens[1400] = 300, 200
    n = sum(lens)
    q, k, v, do = (torch.randn(n, h, D, generator=gen).bfloat16() for h in (4, 2, 2, 4))
    cu = R.lens_to_cu(lens).cuda()
    qd, kd, vd, dod = (t.cuda() for t in (q, k, v, do))
    o, lse = g.gdn2_attn_fwd_varlen(qd, kd, vd, cu, window=window)
    got = {"o": o, "lse": lse, **g.gdn2_attn_bwd_varlen(qd, kd, vd, o, lse, dod, cu, window=window)}
    assert g.gdn2_sync_status() == 0
    spans, at = [], 0
    for m in lens:
        spans.append((at, m))
        at += m
    ref = R.attention(q, k, v, spans, window, D ** -0.5, do)
    for name in ("o", "lse", "dq", "dk", "dv"):
        R.check(got[name], ref[name], ref[name + "_tol"], name)


@pytest.mark.parametrize("D", [64, 128])
def test_nan_is_not_lost(cuda_lib, D):
    """A NaN in one query: every gradient that it has a part in says so, in every channel."""
    g = cuda_lib
    q, k, v, do = (torch.randn(1, 300, 2, D, generator=torch.Generator().manual_seed(i)).bfloat16().cuda() for i in range(4))
    q[0, 200, 1, 5] = float("nan")
    o, lse = g.gdn2_attn_fwd(q, k, v)
    r = g.gdn2_attn_bwd(q, k, v, o, lse, do)
    assert g.gdn2_sync_status() == 0
    bad = {n: ~torch.isfinite(t[0]) for n, t in {"o": o, "lse": lse[..., None], **r}.items()}
    for n in ("o", "lse", "dq"):  # the row alone
        assert bad[n][200, 1].all() and bad[n].sum() == bad[n][200, 1].numel(), n
    for n in ("dk", "dv"):  # the keys that the row sees (other keys of its sequence and head may have it: 0 * NaN)
        assert bad[n][:201, 1].all() and not bad[n][:, 0].any(), n


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("news", [[1, 1, 0], [3, 1, 2], [70, 20, 0]])
def test_padded_batches_and_shared_pages(cuda_lib, news, e4m3):
    """Serving with a batch padded to a fixed number of rows and sequences that share their first pages: the
    cache and the outputs behind the last row stay as they were, and the sharing changes nothing."""
    g = cuda_lib
    page, shared, gen = 16, 5, torch.Generator().manual_seed(12)
    kv = [90 + 3 * n for n in news]
    kv = [max(a, n + shared * page) for a, n in zip(kv, news)]
    n, tail, width = sum(news), 9, 24
    q, k, v = (torch.randn(n + tail, h, D, generator=gen).bfloat16() for h in (H, HKV, HKV))
    for t in (q, k, v):
        t[n:] = float("nan")
    q, k, v = q.cuda(), k.cuda(), v.cuda()
    dt = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    pages = 3 * width
    raw = [torch.randint(0, 120, (pages, page, HKV, D), generator=gen).to(torch.uint8).view(dt) if e4m3 else
           torch.randn(pages, page, HKV, D, generator=gen).bfloat16() for _ in range(2)]
    sc = [0.01 + torch.rand(pages, page, HKV, generator=gen) for _ in range(2)] if e4m3 else [None, None]
    own = torch.arange(pages, dtype=torch.int32).view(3, width)
    both = own.clone()
    both[1:, :shared] = own[0, :shared]  # one prefix for all
    for t in (*raw, *sc):  # ... which the table without sharing holds three times
        if t is not None:
            t = t.view(torch.uint8) if e4m3 and t.dtype == dt else t
            for i in (1, 2):
                t[own[i, :shared].long()] = t[own[0, :shared].long()]
    cu, lens = R.lens_to_cu(news).cuda(), torch.tensor(kv, dtype=torch.int32).cuda()
    got = []
    for table in (own, both):
        kc, vc, ks, vs = (None if t is None else t.cuda() for t in (*raw, *sc))
        before = [t.clone() for t in (kc, vc)]
        tb = table.cuda()
        g.gdn2_cache_write(k, v, kc, vc, cu, lens, tb, ks, vs)
        o, lse = torch.full_like(q, 7.0), torch.full((n + tail, H), 7.0, device="cuda")
        g.gdn2_attn_cached(q, kc, vc, cu, lens, tb, ks, vs, o=o, lse=lse)
        kb, vb = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
        g.gdn2_cache_read(kc, vc, cu, lens, tb, ks, vs, k=kb, v=vb)
        assert g.gdn2_sync_status() == 0
        for t in (o, lse, kb, vb):
            assert (t[n:] == 7).all() and torch.isfinite(t.float()).all()
        written = torch.zeros(pages, page, dtype=torch.bool)
        for i, m in enumerate(news):
            for p in range(kv[i] - m, kv[i]):
                written[table[i, p // page], p % page] = True
        for x, y in zip((kc, vc), before):
            same = (x.view(torch.uint8) == y.view(torch.uint8)).flatten(2).all(2).cpu()
            assert same[~written].all() and not same[written].any()
        got.append((o[:n], lse[:n], kb[:n], vb[:n]))
    for x, y in zip(*got):
        assert torch.equal(x, y)
