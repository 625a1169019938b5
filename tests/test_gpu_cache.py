"""The paged cache and the attention that reads it, against the 64-bit forms."""
import random

import pytest
import torch

import attn_ref as R

pytestmark = pytest.mark.gpu


class Batch:
    """Sequences over a paged cache whose unused rows and scales hold NaN."""

    def __init__(self, q_lens, kv_lens, page, Hkv, D, e4m3, seed=0, tail=0, slack=2):
        g = torch.Generator().manual_seed(seed)
        order = random.Random(seed)
        self.q_lens, self.kv, self.page, self.Hkv, self.D, self.e4m3 = q_lens, kv_lens, page, Hkv, D, e4m3
        need = [-(-n // page) for n in kv_lens]
        pages = sum(need) + slack
        ids = list(range(pages))
        order.shuffle(ids)
        width = max(need + [1]) + 1
        self.table = torch.full((len(kv_lens), width), -5, dtype=torch.int32)
        at = 0
        for i, n in enumerate(need):
            self.table[i, :n] = torch.tensor(ids[at:at + n], dtype=torch.int32)
            at += n
        self.total = sum(q_lens) + tail
        self.k_all = [torch.randn(n, Hkv, D, generator=g).bfloat16() for n in kv_lens]
        self.v_all = [torch.randn(n, Hkv, D, generator=g).bfloat16() for n in kv_lens]
        shape = (pages, page, Hkv, D)
        self.kc, self.vc = torch.full(shape, float("nan")).bfloat16(), torch.full(shape, float("nan")).bfloat16()
        self.ks = self.vs = None
        if e4m3:
            self.kc, self.vc = self.kc.to(torch.float8_e4m3fn), self.vc.to(torch.float8_e4m3fn)
            self.ks, self.vs = torch.full(shape[:3], float("nan")), torch.full(shape[:3], float("nan"))
        self.cu = R.lens_to_cu(q_lens)
        self.dev = {n: getattr(self, n).cuda() for n in ("table", "kc", "vc", "cu")}
        self.dev["kv"] = torch.tensor(kv_lens, dtype=torch.int32).cuda()
        self.dev["ks"], self.dev["vs"] = (None, None) if not e4m3 else (self.ks.cuda(), self.vs.cuda())

    def args(self):
        d = self.dev
        return (d["cu"], d["kv"], d["table"], d["ks"], d["vs"])

    def fill(self, g):
        """Everything into the cache: the past in one call, then the new tokens in another."""
        for part in ("past", "new"):
            lens = [n - m if part == "past" else m for n, m in zip(self.kv, self.q_lens)]
            ends = [n - m if part == "past" else n for n, m in zip(self.kv, self.q_lens)]
            if sum(lens) == 0:
                continue
            pick = lambda xs: torch.cat([x[e - n:e] for x, n, e in zip(xs, lens, ends)]).cuda()  # noqa: E731
            d = self.dev
            g.gdn2_cache_write(pick(self.k_all), pick(self.v_all), d["kc"], d["vc"], R.lens_to_cu(lens).cuda(),
                               torch.tensor(ends, dtype=torch.int32).cuda(), d["table"], d["ks"], d["vs"])
        return self

    def held(self, i):
        """Sequence i's keys and values as the cache holds them, in 64 bits."""
        if not self.e4m3:
            return self.k_all[i].double(), self.v_all[i].double()
        return tuple(y * s.double()[..., None] for y, s in (R.quantise(x[i]) for x in (self.k_all, self.v_all)))


KINDS = [False, True]


@pytest.mark.parametrize("e4m3", KINDS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page,Hkv", [(1, 1), (16, 3), (48, 2), (64, 8), (7, 5)])
def test_write_and_read(cuda_lib, page, Hkv, D, e4m3):
    g = cuda_lib
    b = Batch([1, 0, 40, 17, 3], [1, 9, 100, 17, 60], page, Hkv, D, e4m3, seed=page).fill(g)
    d = b.dev
    # everything of every sequence
    cu = R.lens_to_cu(b.kv).cuda()
    k, v = g.gdn2_cache_read(d["kc"], d["vc"], cu, d["kv"], d["table"], d["ks"], d["vs"], total_T=sum(b.kv))
    assert g.gdn2_sync_status() == 0
    want = [torch.cat(x) for x in zip(*[b.held(i) for i in range(len(b.kv))])]
    for got, ref in zip((k, v), want):
        if e4m3:
            # the scale and the division are rounded in fp32, which moves a value to the neighbouring
            # e4m3 step only next to a border; then bf16's half step of the product, on both sides
            exact = ref.to(torch.float32).to(torch.bfloat16)
            assert torch.equal(got.cpu(), exact)
        else:
            assert torch.equal(got.cpu().double(), ref)


def test_e4m3_edges(cuda_lib):
    """Zero rows, the largest values, subnormal quotients, ties, infinities and NaN."""
    g = cuda_lib
    rows = torch.zeros(8, 1, 64)
    rows[1, 0, 0] = 448
    rows[1, 0, 1:9] = torch.tensor([17.0, 19.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, -1.0625, -1.1875, 232.0])
    rows[2] = 1e30
    rows[3, 0, :3] = torch.tensor([float("inf"), 2.0, float("nan")])
    rows[4] = float("nan")
    rows[5, 0, 0] = 1e-38
    rows[6] = 3.3e38
    rows[7, 0, 5] = -5
    rows = rows.bfloat16()
    b = Batch([8], [8], 4, 1, 64, True)
    b.k_all, b.v_all = [rows], [rows.flip(0)]
    b.fill(g)
    d = b.dev
    k, v = g.gdn2_cache_read(d["kc"], d["vc"], *b.args(), total_T=8)
    assert g.gdn2_sync_status() == 0
    for got, x in ((k, rows), (v, rows.flip(0))):
        y, s = R.quantise(x)
        ref = (y * s.double()[..., None]).float().bfloat16()
        assert torch.equal(torch.isnan(got.cpu()), torch.isnan(ref))
        assert torch.equal(torch.nan_to_num(got.cpu()), torch.nan_to_num(ref))


def attend(g, b, H, window=0, scale=0.11, seed=0, workspace=None):
    gen = torch.Generator().manual_seed(seed)
    q = torch.randn(b.total, H, b.D, generator=gen).bfloat16()
    d = b.dev
    o = torch.full(q.shape, 7.0).bfloat16().cuda()
    lse = torch.full(q.shape[:2], 7.0).cuda()
    g.gdn2_attn_cached(q.cuda(), d["kc"], d["vc"], *b.args(), window=window, scale=scale, o=o, lse=lse, workspace=workspace)
    assert g.gdn2_sync_status() == 0
    return q, o, lse


def verify(b, q, o, lse, H, window, scale):
    G, at = H // b.Hkv, 0
    for i, (n, kv) in enumerate(zip(b.q_lens, b.kv)):
        k, v = b.held(i)
        for h in range(H):
            if n == 0:
                continue
            x = R.head(q[at:at + n, h], k[:, h // G], v[:, h // G], kv - n, window, scale, torch.bfloat16)
            R.check(o[at:at + n, h], x["o"], x["o_tol"], f"o of sequence {i} head {h}")
            R.check(lse[at:at + n, h], x["lse"], x["lse_tol"], f"lse of sequence {i} head {h}")
        at += n
    assert (o[at:] == 7.0).all() and (lse[at:] == 7.0).all()


@pytest.mark.parametrize("e4m3", KINDS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q_lens,kv_lens", [
    ([1], [1]), ([1, 1, 1], [5, 64, 700]), ([1, 0, 2, 3], [333, 0, 2, 40]), ([5, 1], [5, 600]),
])
def test_decode(cuda_lib, q_lens, kv_lens, D, e4m3):
    b = Batch(q_lens, kv_lens, 16, 2, D, e4m3, seed=sum(kv_lens), tail=2).fill(cuda_lib)
    verify(b, *attend(cuda_lib, b, 8), 8, 0, 0.11)


@pytest.mark.parametrize("e4m3", KINDS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q_lens,kv_lens,page", [
    ([70], [70], 64), ([130, 1], [130, 900], 16), ([64, 300], [500, 301], 48), ([200, 0, 90], [1000, 3, 129], 256),
])
def test_chunks(cuda_lib, q_lens, kv_lens, page, D, e4m3):
    b = Batch(q_lens, kv_lens, page, 2, D, e4m3, seed=sum(kv_lens) + 1, tail=3).fill(cuda_lib)
    verify(b, *attend(cuda_lib, b, 8), 8, 0, 0.11)


@pytest.mark.parametrize("e4m3", KINDS)
@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 1), (40, 2), (64, 1), (14, 2)])
@pytest.mark.parametrize("rows", [1, 45])
def test_heads(cuda_lib, rows, H, Hkv, e4m3):
    b = Batch([rows, 1], [rows + 150, 77], 32, Hkv, 64, e4m3, seed=H).fill(cuda_lib)
    verify(b, *attend(cuda_lib, b, H), H, 0, 0.11)


@pytest.mark.parametrize("e4m3", KINDS)
@pytest.mark.parametrize("window", [1, 16, 100, 2 ** 31 - 1])
@pytest.mark.parametrize("rows", [1, 3, 150])
def test_windows(cuda_lib, rows, window, e4m3):
    b = Batch([rows, 1], [rows + 700, 1000], 16, 2, 128, e4m3, seed=window % 89).fill(cuda_lib)
    verify(b, *attend(cuda_lib, b, 4, window=window), 4, window, 0.11)


@pytest.mark.parametrize("e4m3", KINDS)
@pytest.mark.parametrize("rows", [1, 40])
def test_long_axis_in_parts(cuda_lib, rows, e4m3):
    """One sequence, few rows: the key axis is cut into parts that a second kernel joins."""
    g = cuda_lib
    b = Batch([rows], [6001], 16, 1, 128, e4m3, seed=5).fill(g)
    assert g.gdn2_attn_cached_workspace_size(1, rows, 4, 1, 128, 0, b.table.shape[1], 16) > 0
    verify(b, *attend(g, b, 4), 4, 0, 0.11)


def test_page_sizes(cuda_lib):
    for page in (1, 3, 8, 128, 1000):
        for rows in (1, 80):
            b = Batch([rows], [rows + 300], page, 1, 64, False, seed=page).fill(cuda_lib)
            verify(b, *attend(cuda_lib, b, 2), 2, 0, 0.11)


@pytest.mark.parametrize("rows", [1, 100])
def test_bad_pages_and_lengths_are_reported(cuda_lib, rows):
    """A page outside the cache or a length outside the table sets the status; nothing else is touched."""
    g = cuda_lib
    for which in ("page", "negative", "long", "short"):
        b = Batch([rows, rows], [rows + 40, rows + 90], 16, 2, 64, False, seed=1).fill(g)
        assert g.gdn2_sync_status() == 0
        q = torch.randn(b.total, 4, 64).bfloat16().cuda()
        d = b.dev
        good, _ = g.gdn2_attn_cached(q, d["kc"], d["vc"], *b.args())
        if which == "page":
            d["table"][1, 0] = b.kc.shape[0]
        elif which == "negative":
            d["table"][1, 2] = -1
        elif which == "long":
            d["kv"][1] = b.table.shape[1] * 16 + 1
        else:
            d["kv"][1] = rows - 1
        o = torch.full_like(q, 7.0)
        g.gdn2_attn_cached(q, d["kc"], d["vc"], *b.args(), o=o)
        assert g.gdn2_sync_status() == -11, which
        assert torch.equal(o[:rows], good[:rows]), which
        if which in ("long", "short"):
            assert (o[rows:] == 7.0).all()
        before = d["kc"].clone()
        k = torch.randn(b.total, 2, 64).bfloat16().cuda()
        g.gdn2_cache_write(k, k, d["kc"], d["vc"], d["cu"], d["kv"], d["table"])
        st = g.gdn2_sync_status()
        if which in ("long", "short"):
            assert st == -11
            # only sequence 0's new rows changed
            changed = (before.view(torch.int16) != d["kc"].view(torch.int16)).any(-1).any(-1).sum()
            assert int(changed) == rows


@pytest.mark.parametrize("e4m3", KINDS)
def test_repeatable_and_graphs(cuda_lib, e4m3):
    """Captured and replayed over lengths and pages that changed in place."""
    g = cuda_lib
    b = Batch([1, 1, 1], [40, 900, 2500], 16, 2, 128, e4m3, seed=2).fill(g)
    d = b.dev
    q = torch.randn(3, 8, 128).bfloat16().cuda()
    a = g.gdn2_attn_cached(q, d["kc"], d["vc"], *b.args())
    c = g.gdn2_attn_cached(q, d["kc"], d["vc"], *b.args())
    assert all(torch.equal(x, y) for x, y in zip(a, c))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = g.gdn2_attn_cached(q, d["kc"], d["vc"], *b.args())
    d["kv"].copy_(torch.tensor([17, 640, 2100], dtype=torch.int32))
    want = g.gdn2_attn_cached(q, d["kc"], d["vc"], *b.args())
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("e4m3", KINDS)
@pytest.mark.parametrize("rows,capacity", [(1, 160), (1, 4096), (70, 160), (70, 4096)])
def test_lengths_far_below_zero(cuda_lib, rows, capacity, e4m3):
    """A length whose difference to the new tokens wraps in 32 bits skips the sequence as any other below
    them does, in one part (no workspace) and in several, few rows and many."""
    g = cuda_lib
    for bad in (-2 ** 31, -2 ** 31 + rows - 1, -2 ** 31 + rows, -1, rows - 1):
        b = Batch([rows, rows], [rows + 40, rows + 50], 16, 2, 64, e4m3, seed=3).fill(g)
        d = b.dev
        wide = torch.full((2, capacity // 16), -5, dtype=torch.int32)
        wide[:, :b.table.shape[1]] = b.table[:, :capacity // 16]
        d["table"] = wide.cuda()
        q = torch.randn(b.total, 4, 64).bfloat16().cuda()
        good, good_lse = g.gdn2_attn_cached(q, d["kc"], d["vc"], *b.args())
        assert g.gdn2_sync_status() == 0
        d["kv"][1] = bad
        o, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
        g.gdn2_attn_cached(q, d["kc"], d["vc"], *b.args(), o=o, lse=lse)
        assert g.gdn2_sync_status() == -11, bad
        assert torch.equal(o[:rows], good[:rows]) and torch.equal(lse[:rows], good_lse[:rows])
        assert (o[rows:] == 7.0).all() and (lse[rows:] == 7.0).all()
        k, v = (torch.full((b.total, 2, 64), 7.0).bfloat16().cuda() for _ in range(2))
        g.gdn2_cache_read(d["kc"], d["vc"], *b.args(), k=k, v=v)
        assert g.gdn2_sync_status() == -11, bad
        assert (k[rows:] == 7.0).all() and (v[rows:] == 7.0).all() and (k[:rows] != 7.0).any()
        before = d["kc"].view(torch.uint8).clone()
        g.gdn2_cache_write(k, k, d["kc"], d["vc"], *b.args())
        assert g.gdn2_sync_status() == -11, bad
        changed = (before != d["kc"].view(torch.uint8)).flatten(2).any(-1).flatten()
        first = b.kv[0] - rows
        own = {int(b.table[0, p // 16]) * 16 + p % 16 for p in range(first, b.kv[0])}
        assert set(changed.nonzero().flatten().tolist()) <= own


@pytest.mark.parametrize("e4m3", KINDS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page,rows,window", [(1, 1, 40), (16, 1, 40), (1, 150, 40), (7, 150, 100), (8, 150, 100), (16, 300, 1),
                                              (64, 150, 20), (256, 150, 20)])
def test_pages_behind_the_window(cuda_lib, page, rows, window, D, e4m3):
    """Pages that no query sees any more (a server frees them) are not looked up: their entries may be no
    page, or one that has become another sequence's, NaN among its values."""
    g = cuda_lib
    b = Batch([rows, rows], [rows + 700, rows + 515], page, 2, D, e4m3, seed=page + rows).fill(g)
    d = b.dev
    q = torch.randn(b.total, 4, D, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    want = g.gdn2_attn_cached(q, d["kc"], d["vc"], *b.args(), window=window)
    assert g.gdn2_sync_status() == 0
    poison = min(set(range(b.kc.shape[0])) - set(b.table.flatten().tolist()))  # of no sequence: still all NaN
    for entry in (-1, b.kc.shape[0], poison):
        table = b.table.clone()
        for i, kv in enumerate(b.kv):
            gone = max(0, kv - rows - window + 1) // page
            assert gone > 0 or page == 256
            table[i, :gone] = entry
        d["table"] = table.cuda()
        got = g.gdn2_attn_cached(q, d["kc"], d["vc"], *b.args(), window=window)
        assert g.gdn2_sync_status() == 0, entry
        for x, y in zip(got, want):
            assert torch.equal(x, y), entry


@pytest.mark.parametrize("e4m3", KINDS)
def test_one_workspace_for_smaller_calls(cuda_lib, e4m3):
    """A server's workspace, sized once for its largest call: chunks and single tokens of fewer sequences
    over shorter tables give the same with it as with one of their own."""
    g = cuda_lib
    H, Hkv, page = 16, 4, 16
    size = g.gdn2_attn_cached_workspace_size(4, 2048, H, Hkv, 64, 0, 512, page)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    for q_lens, width in (([512] * 4, 512), ([1] * 4, 512), ([1], 512), ([60], 512), ([30, 1], 200), ([1] * 3, 40)):
        b = Batch(q_lens, [n + 230 + 50 * i for i, n in enumerate(q_lens)], page, Hkv, 64, e4m3, seed=width).fill(g)
        d = b.dev
        d["table"] = torch.nn.functional.pad(b.table, (0, width - b.table.shape[1]), value=-5).cuda()
        q = torch.randn(b.total, H, 64, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
        ws.fill_(255)  # NaN
        want = g.gdn2_attn_cached(q, d["kc"], d["vc"], *b.args())
        got = g.gdn2_attn_cached(q, d["kc"], d["vc"], *b.args(), workspace=ws)
        assert g.gdn2_sync_status() == 0
        assert all(torch.equal(x, y) for x, y in zip(got, want)), (q_lens, width)


@pytest.mark.parametrize("D,Hkv", [(128, 8), (64, 5), (128, 3)])
def test_write_e4m3_prompts(cuda_lib, D, Hkv):
    """Enough rows (more than 4096 warp passes) that a warp takes several passes of a token's heads."""
    g = cuda_lib
    b = Batch([700, 0, 811, 3], [700, 5, 900, 3], 16, Hkv, D, True, seed=D + Hkv).fill(g)
    d = b.dev
    k, v = g.gdn2_cache_read(d["kc"], d["vc"], R.lens_to_cu(b.kv).cuda(), d["kv"], d["table"], d["ks"], d["vs"], total_T=sum(b.kv))
    assert g.gdn2_sync_status() == 0
    for got, ref in zip((k, v), [torch.cat(x) for x in zip(*[b.held(i) for i in range(4)])]):
        assert torch.equal(got.cpu(), ref.float().bfloat16())


@pytest.mark.parametrize("e4m3", KINDS)
@pytest.mark.parametrize("window", [0, 33])
@pytest.mark.parametrize("most", [1, 3, 90])
def test_many_sequences(cuda_lib, most, window, e4m3):
    """More sequences than a warp looks up at a time, empty ones among them: single tokens, some with more
    (further tiles of the rows kernel), and mostly chunks (tiles of the tensor core), in one part and in several."""
    order = random.Random(most)
    q_lens = [order.choice([0, 1, 1, most]) for _ in range(75)]
    q_lens[40], q_lens[70] = max(most, 13), 1
    kv = [n + order.choice([0, 5, 130, 400]) for n in q_lens]
    kv[70] = 3000
    b = Batch(q_lens, kv, 16, 1, 64, e4m3, seed=most, tail=2).fill(cuda_lib)
    verify(b, *attend(cuda_lib, b, 4, window=window), 4, window, 0.11)


@pytest.mark.parametrize("e4m3", KINDS)
@pytest.mark.parametrize("page", [16, 7])
@pytest.mark.parametrize("rows", [1, 100])
def test_rows_of_bad_pages(cuda_lib, rows, page, e4m3):
    """A page outside the cache: its rows are skipped by write and read, and attention reads zeros for
    them (a score of 0 and nothing of its value); the rows of other pages are as always."""
    g = cuda_lib
    for bad in (-1, 10 ** 9, -2 ** 31):
        b = Batch([rows, rows], [rows + 40, rows + 90], page, 2, 64, e4m3, seed=page + rows).fill(g)
        d = b.dev
        lost = [(1, 2), (1, (rows + 89) // page)]  # a page of the past, and the last, which holds new rows
        if rows > 1:
            lost.append((0, (40 + rows // 2) // page))
        gone = [torch.zeros(n, dtype=torch.bool) for n in b.kv]
        table = b.table.clone()
        for i, pg in lost:
            table[i, pg] = bad
            gone[i][pg * page:(pg + 1) * page] = True
        d["table"] = table.cuda()
        # attention, against the cache with zeros there
        q, o, lse = torch.randn(b.total, 4, 64).bfloat16(), None, None
        o, lse = g.gdn2_attn_cached(q.cuda(), d["kc"], d["vc"], *b.args(), scale=0.11)
        assert g.gdn2_sync_status() == -11
        for i in range(2):
            at = slice(i * rows, (i + 1) * rows)
            k, v = (t.clone() for t in b.held(i))
            k[gone[i]], v[gone[i]] = 0, 0
            for h in range(4):
                x = R.head(q[at, h], k[:, h // 2], v[:, h // 2], b.kv[i] - rows, 0, 0.11, torch.bfloat16)
                R.check(o[at, h], x["o"], x["o_tol"], "o")
                R.check(lse[at, h], x["lse"], x["lse_tol"], "lse")
        # reading the new rows
        kb, vb = (torch.full((b.total, 2, 64), 7.0).bfloat16().cuda() for _ in range(2))
        g.gdn2_cache_read(d["kc"], d["vc"], *b.args(), k=kb, v=vb)
        assert g.gdn2_sync_status() == -11
        new_gone = torch.cat([gone[i][b.kv[i] - rows:] for i in range(2)])
        assert new_gone.any()
        for got, which in ((kb.cpu(), 0), (vb.cpu(), 1)):
            ref = torch.cat([b.held(i)[which][b.kv[i] - rows:] for i in range(2)]).float().bfloat16()
            assert (got[new_gone] == 7.0).all() and torch.equal(got[~new_gone], ref[~new_gone])
        # writing others in their place
        before = [d[n].view(torch.uint8).cpu().flatten(2) for n in ("kc", "vc")]
        fresh = torch.randn(b.total, 2, 64).bfloat16().cuda()
        g.gdn2_cache_write(fresh, -fresh, d["kc"], d["vc"], *b.args())
        assert g.gdn2_sync_status() == -11
        written = torch.zeros(b.kc.shape[:2], dtype=torch.bool)
        for i in range(2):
            for p in range(b.kv[i] - rows, b.kv[i]):
                if not gone[i][p]:
                    written[b.table[i, p // page], p % page] = True
        for was, n in zip(before, ("kc", "vc")):
            same = (was == d[n].view(torch.uint8).cpu().flatten(2)).all(-1)
            assert same[~written].all() and not same[written].any()


@pytest.mark.parametrize("e4m3", KINDS)
@pytest.mark.parametrize("most", [1, 90])
def test_invalid_sequences_are_skipped(cuda_lib, most, e4m3):
    """Invalid cu_seqlens entries in a batch of many sequences: the two around one are skipped by every
    call of the cache, the others are as without it, in one part and in several."""
    g = cuda_lib
    H = 4
    for entry in (-1, 2 ** 31 - 1):
        q_lens = [1 + (i % 3) * (most // 3) for i in range(45)]
        kv = [n + 20 * (i % 4) + (2500 if i == 7 else 0) for i, n in enumerate(q_lens)]
        b = Batch(q_lens, kv, 16, 2, 64, e4m3, seed=most).fill(g)
        cu = R.lens_to_cu(q_lens)
        skipped = torch.zeros(b.total, dtype=torch.bool)
        skipped[cu[35]:cu[37]] = True
        cu[36] = entry
        q = torch.randn(b.total, H, 64, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
        d = b.dev
        want = g.gdn2_attn_cached(q, d["kc"], d["vc"], *b.args())
        want_kv = g.gdn2_cache_read(d["kc"], d["vc"], *b.args(), total_T=b.total)
        assert g.gdn2_sync_status() == 0
        d["cu"] = cu.cuda()
        o, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
        g.gdn2_attn_cached(q, d["kc"], d["vc"], *b.args(), o=o, lse=lse)
        assert g.gdn2_sync_status() == -10
        kb, vb = (torch.full((b.total, 2, 64), 7.0).bfloat16().cuda() for _ in range(2))
        g.gdn2_cache_read(d["kc"], d["vc"], *b.args(), k=kb, v=vb)
        assert g.gdn2_sync_status() == -10
        for got, ref in zip((o, lse, kb, vb), (*want, *want_kv)):
            got, ref = got.cpu(), ref.cpu()
            assert (got[skipped] == 7.0).all() and torch.equal(got[~skipped], ref[~skipped])


@pytest.mark.parametrize("e4m3", KINDS)
@pytest.mark.parametrize("window", [0, 200])
@pytest.mark.parametrize("n,rows", [(3, 1), (70, 1), (2, 90)])
def test_tables_far_wider_than_the_sequences(cuda_lib, n, rows, window, e4m3):
    """A table for 131072 positions, as a server or a captured graph has it: most parts of the key axis are
    empty, and few or many rows are joined over them."""
    g = cuda_lib
    kv = [rows + (997 * i) % 1500 for i in range(n)]
    b = Batch([rows] * n, kv, 16, 2, 64, e4m3, seed=n).fill(g)
    b.dev["table"] = torch.nn.functional.pad(b.table, (0, 8192 - b.table.shape[1]), value=-5).cuda()
    assert g.gdn2_attn_cached_workspace_size(n, n * rows, 16, 2, 64, 0, 8192, 16) > 0
    verify(b, *attend(g, b, 16, window=window), 16, window, 0.11)


@pytest.mark.parametrize("e4m3", KINDS)
@pytest.mark.parametrize("rows", [1, 70])
@pytest.mark.parametrize("big_q,big_k,big_v", [(1e-20, 1e20, 1.0), (1e20, 1e-20, 1e30), (1.0, 1.0, 1e-30), (30.0, 1.0, 1.0)])
def test_far_scales(cuda_lib, big_q, big_k, big_v, rows, e4m3):
    """Queries, keys and values far from 1 whose scores are not, values whose rows differ by 1e6 in scale, and
    scores of hundreds."""
    g = cuda_lib
    b = Batch([rows, rows], [rows + 300, rows + 4000], 16, 2, 64, e4m3, seed=9)
    gen = torch.Generator().manual_seed(7)
    b.k_all = [(big_k * x.float()).bfloat16() for x in b.k_all]
    b.v_all = [(big_v * x.float() * 10.0 ** torch.randint(-3, 4, (len(x), 1, 1), generator=gen)).bfloat16() for x in b.v_all]
    b.fill(g)
    d = b.dev
    q = (big_q * torch.randn(b.total, 8, 64, generator=gen)).bfloat16()
    o, lse = g.gdn2_attn_cached(q.cuda(), d["kc"], d["vc"], *b.args(), scale=0.11)
    assert g.gdn2_sync_status() == 0
    verify(b, q, o, lse, 8, 0, 0.11)
