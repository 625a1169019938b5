"""The attention layer's entry points refuse invalid arguments with the documented status before
touching the GPU, and their binding refuses tensors it cannot pass on (CPU only)."""
import ctypes

import pytest
import torch

import attn_ref as R
import gated_delta_rule_78_b200 as g

F32, BF16 = 0, 1
P = ctypes.c_void_p(0x7F0000000000)    # aligned stand-in address, never dereferenced
MIS = ctypes.c_void_p(0x7F0000000004)  # 4-byte aligned only
NUL = ctypes.c_void_p(0)
OK, NULL, SHAPE, DTYPE, ALIGN, WS, UNSUP = 0, -1, -2, -3, -4, -5, -8


@pytest.fixture(scope="module")
def lib():
    return g.load()


def rope(lib, flags=1, dt=BF16, N=4, H=2, Hkv=1, D=128, rot=128, q=P, k=P, wq=P, wk=P, pos=P, inv=P, eps=1e-6, rs=1.0, qo=P, ko=P):
    return lib.gdn2_qk_rope(flags, dt, N, H, Hkv, D, rot, q, k, wq, wk, pos, inv, eps, rs, qo, ko, NUL)


def rope_bwd(lib, flags=1, dt=BF16, N=4, D=128, rot=128, q=P, dqo=P, dq=P, dwq=P, dwk=P, ws=P, nb=1 << 30):
    return lib.gdn2_qk_rope_bwd(flags, dt, N, 2, 1, D, rot, q, P, P, P, P, P, 1e-6, 1.0, dqo, P, dq, P, dwq, dwk, ws, nb, NUL)


def fwd(lib, dt=BF16, B=1, T=8, H=2, Hkv=1, D=128, window=0, scale=1.0, q=P, o=P, lse=NUL):
    return lib.gdn2_attn_fwd(dt, B, T, H, Hkv, D, window, scale, q, P, P, o, lse, NUL)


def fwd_varlen(lib, dt=BF16, N=1, T=8, H=2, Hkv=1, D=128, window=0, scale=1.0, cu=P, q=P, lse=NUL):
    return lib.gdn2_attn_fwd_varlen(dt, N, T, H, Hkv, D, window, scale, cu, q, P, P, P, lse, NUL)


def bwd(lib, dt=BF16, B=1, T=8, H=2, Hkv=1, D=128, lse=P, do=P, dq=P, ws=P, nb=1 << 30):
    return lib.gdn2_attn_bwd(dt, B, T, H, Hkv, D, 0, 1.0, P, P, P, P, lse, do, dq, P, P, ws, nb, NUL)


def cache(lib, fn="gdn2_cache_write", kind=0, dt=BF16, N=1, T=8, Hkv=1, D=128, cu=P, kv=P, table=P, width=4, pages=4, page=16, k=P,
          kc=P, ks=NUL, vs=NUL):
    tail = (k, P, kc, P, ks, vs) if fn == "gdn2_cache_write" else (kc, P, ks, vs, k, P)
    return getattr(lib, fn)(kind, dt, N, T, Hkv, D, cu, kv, table, width, pages, page, *tail, NUL)


def cached(lib, kind=0, dt=BF16, N=1, T=1, H=2, Hkv=1, D=128, window=0, scale=1.0, width=4, pages=4, page=16, q=P, ks=NUL, vs=NUL, o=P,
           lse=NUL, ws=P, nb=1 << 30, table=P):
    return lib.gdn2_attn_cached(kind, dt, N, T, H, Hkv, D, window, scale, P, P, table, width, pages, page, q, P, P, ks, vs, o, lse, ws,
                                nb, NUL)


def test_rope_refusals(lib):
    assert rope(lib, flags=4) == UNSUP
    assert rope(lib, dt=2) == DTYPE
    assert rope(lib, N=-1) == SHAPE and rope(lib, H=0) == SHAPE and rope(lib, Hkv=0) == SHAPE
    assert rope(lib, D=96) == UNSUP and rope(lib, D=256) == UNSUP
    assert rope(lib, rot=3) == SHAPE and rope(lib, rot=130) == SHAPE and rope(lib, rot=-2) == SHAPE
    assert rope(lib, eps=-1.0) == SHAPE and rope(lib, eps=float("nan")) == SHAPE
    assert rope(lib, rs=float("inf")) == SHAPE
    for name in ("q", "k", "qo", "ko", "pos", "inv"):
        assert rope(lib, **{name: NUL}) == NULL, name
        assert rope(lib, **{name: MIS}) == ALIGN, name
    assert rope(lib, wq=MIS) == ALIGN and rope(lib, wk=MIS) == ALIGN
    assert rope(lib, N=1 << 30, H=2) == UNSUP  # (row, head) pairs past 32 bits
    assert rope(lib, N=0, q=NUL) == OK


def test_rope_bwd_refusals(lib):
    need = lib.gdn2_qk_rope_workspace_size(1, BF16, 4, 2, 1, 128)
    assert need > 0 and lib.gdn2_qk_rope_workspace_size(0, BF16, 4, 2, 1, 128) == 0
    assert lib.gdn2_qk_rope_workspace_size(1, BF16, 4, 2, 1, 96) == 0
    assert rope_bwd(lib, ws=NUL) == WS and rope_bwd(lib, nb=need - 1) == WS and rope_bwd(lib, ws=MIS) == ALIGN
    assert rope_bwd(lib, dwq=MIS) == ALIGN and rope_bwd(lib, dqo=NUL) == NULL and rope_bwd(lib, dq=MIS) == ALIGN
    assert rope_bwd(lib, q=NUL) == NULL
    assert rope_bwd(lib, rot=7) == SHAPE


def test_rope_workspace_serves_smaller_batches(lib):
    """A workspace sized for N rows is enough for fewer: the need of a call, found where it starts to be
    refused, never exceeds the size of a larger one.  (An unaligned address is refused after the size.)"""
    def need(n):
        lo, hi = 0, 1 << 30  # the least size that is not refused
        while lo < hi:
            mid = (lo + hi) // 2
            lo, hi = (lo, mid) if rope_bwd(lib, N=n, ws=MIS, nb=mid) == ALIGN else (mid + 1, hi)
        return lo

    last = 0
    for n in (1, 63, 64, 65, 296, 297, 400, 511, 512, 513, 2047, 2048, 4096, 100000, 1 << 29):
        size = lib.gdn2_qk_rope_workspace_size(1, BF16, n, 2, 1, 128)
        assert last <= size and need(n) <= size, n
        assert size == g.gdn2_qk_rope_workspace_size(torch.bfloat16, n, 2, 1, 128)
        last = size
    assert need(511) > need(512)  # what makes it worth a test


def test_attention_refusals(lib):
    for f in (fwd, fwd_varlen):
        assert f(lib, dt=7) == DTYPE
        assert f(lib, T=-1) == SHAPE and f(lib, H=0) == SHAPE and f(lib, Hkv=0) == SHAPE
        assert f(lib, H=3, Hkv=2) == SHAPE  # heads not a multiple of the key heads
        assert f(lib, D=32) == UNSUP and f(lib, H=65, Hkv=1) == UNSUP
        assert f(lib, window=-1) == SHAPE
        for bad in (0.0, -1.0, float("nan"), float("inf")):
            assert f(lib, scale=bad) == SHAPE
        assert f(lib, q=NUL) == NULL and f(lib, q=MIS) == ALIGN and f(lib, lse=MIS) == ALIGN
        assert f(lib, T=0, q=NUL) == OK
        assert f(lib, T=1 << 30, H=64, Hkv=64) == UNSUP
    assert fwd(lib, B=0) == SHAPE and fwd(lib, o=NUL) == NULL
    assert fwd_varlen(lib, N=0) == SHAPE and fwd_varlen(lib, cu=NUL) == NULL and fwd_varlen(lib, cu=MIS) == ALIGN
    need = lib.gdn2_attn_workspace_size(BF16, 1, 8, 2, 1, 128)
    assert need == 8 * 2 * 4
    assert lib.gdn2_attn_workspace_size(BF16, 1, 8, 3, 2, 128) == 0
    assert bwd(lib, ws=NUL) == WS and bwd(lib, nb=need - 1) == WS and bwd(lib, ws=MIS) == ALIGN
    assert bwd(lib, lse=NUL) == NULL and bwd(lib, do=MIS) == ALIGN and bwd(lib, dq=NUL) == NULL
    assert bwd(lib, T=0, ws=NUL, lse=NUL) == OK


def test_cache_refusals(lib):
    for fn in ("gdn2_cache_write", "gdn2_cache_read"):
        assert cache(lib, fn, kind=2) == DTYPE and cache(lib, fn, dt=5) == DTYPE
        assert cache(lib, fn, dt=F32) == UNSUP
        assert cache(lib, fn, N=0) == SHAPE and cache(lib, fn, width=0) == SHAPE and cache(lib, fn, pages=0) == SHAPE
        assert cache(lib, fn, page=0) == SHAPE and cache(lib, fn, D=80) == UNSUP
        assert cache(lib, fn, width=1 << 20, page=1 << 12) == UNSUP and cache(lib, fn, pages=1 << 20, page=1 << 12, width=1) == UNSUP
        for name in ("cu", "kv", "table", "k", "kc"):
            assert cache(lib, fn, **{name: NUL}) == NULL, name
            assert cache(lib, fn, **{name: MIS}) == ALIGN, name
        assert cache(lib, fn, kind=1) == NULL and cache(lib, fn, kind=1, ks=P, vs=MIS) == ALIGN
        assert cache(lib, fn, T=0, cu=NUL) == OK


def test_cached_attention_refusals(lib):
    assert cached(lib, kind=9) == DTYPE and cached(lib, dt=F32) == UNSUP
    assert cached(lib, H=3, Hkv=2) == SHAPE and cached(lib, scale=0.0) == SHAPE and cached(lib, window=-5) == SHAPE
    assert cached(lib, q=NUL) == NULL and cached(lib, o=MIS) == ALIGN and cached(lib, table=MIS) == ALIGN
    assert cached(lib, kind=1, ks=P) == NULL
    assert cached(lib, T=0, q=NUL) == OK
    need = lib.gdn2_attn_cached_workspace_size(BF16, 1, 1, 2, 1, 128, 0, 4096, 16)
    assert need > 0
    assert cached(lib, width=4096, ws=NUL) == WS and cached(lib, width=4096, nb=need - 1) == WS
    assert cached(lib, width=4096, ws=MIS) == ALIGN
    assert lib.gdn2_attn_cached_workspace_size(F32, 1, 1, 2, 1, 128, 0, 4096, 16) == 0
    # a window bounds the keys, and with them the parts
    assert lib.gdn2_attn_cached_workspace_size(BF16, 1, 1, 2, 1, 128, 64, 4096, 16) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="a call that needs no workspace would launch on the stand-in addresses")
@pytest.mark.parametrize("H,Hkv", [(16, 4), (8, 8), (64, 1), (6, 2)])
@pytest.mark.parametrize("window", [0, 2048])
def test_cached_workspace_serves_smaller_calls(lib, window, H, Hkv):
    """A workspace sized for a call is enough for every call of fewer sequences, tokens and pages, over
    either type of cache.  (A misaligned address is refused after the size; without a device, a call that
    needs none ends at the status word.)"""
    def need(kind, n, t, width):
        lo, hi = 0, 1 << 40
        if cached(lib, kind, N=n, T=t, H=H, Hkv=Hkv, window=window, width=width, ks=P, vs=P, ws=NUL, nb=0) != WS:
            return 0
        while lo < hi:
            mid = (lo + hi) // 2
            ok = cached(lib, kind, N=n, T=t, H=H, Hkv=Hkv, window=window, width=width, ks=P, vs=P, ws=MIS, nb=mid) == ALIGN
            lo, hi = (lo, mid) if ok else (mid + 1, hi)
        return lo

    ns, ts, widths = [1, 2, 3, 5, 37, 75, 256], [1, 2, 4, 7, 16, 17, 64, 65, 130, 256, 300, 513, 2048], [4, 150, 1024, 8192]
    size = {(n, t, w): lib.gdn2_attn_cached_workspace_size(BF16, n, t, H, Hkv, 128, window, w, 16) for n in ns for t in ts for w in widths}
    needs = {(n, t, w): max(need(kind, n, t, w) for kind in (0, 1)) for n in ns for t in ts for w in widths}
    some = 0
    for (n, t, w), have in size.items():
        most = max(v for (a, b, c), v in needs.items() if a <= n and b <= t and c <= w)
        assert most <= have, (n, t, w)
        some += needs[n, t, w] < most
    assert some > 0  # calls that need less than a smaller one are what makes it worth a test


def test_status_names(lib):
    assert g.STATUS_NAMES[-11] == "GDN2_ERR_PAGES" and b"paged" in lib.gdn2_strerror(-11)


def test_binding_refuses_host_tensors_and_wrong_shapes():
    q, k = torch.zeros(4, 2, 64), torch.zeros(4, 1, 64)
    with pytest.raises(ValueError, match="CUDA"):
        g.gdn2_qk_rope(q, k)
    with pytest.raises(ValueError):
        g.gdn2_attn_fwd(q, k, k)
    with pytest.raises(ValueError, match="cu_seqlens"):
        g.gdn2_attn_fwd_varlen(q, k, k, None)
    with pytest.raises(ValueError):
        g.gdn2_cache_write(k, k, k, k, k, k, k)


# ---------------------------------------------------------------- the 64-bit forms themselves
def test_reference_gradients_match_autograd():
    gen = torch.Generator().manual_seed(0)
    q, k, v, do = (torch.randn(9, 5, generator=gen, dtype=torch.float64, requires_grad=i < 3) for i in range(4))
    x = R.head(q, k, v, 0, 4, 0.3, torch.float32, do)
    s = 0.3 * q @ k.T
    s = s.masked_fill(~R.mask_of(0, 9, 9, 4), -float("inf"))
    o = torch.softmax(s, 1) @ v
    for a, b in zip((x["dq"], x["dk"], x["dv"]), torch.autograd.grad(o, (q, k, v), do)):
        assert torch.allclose(a, b, rtol=0, atol=1e-12)
    assert torch.allclose(x["o"], o.detach(), rtol=0, atol=1e-13)


def test_bounds_reject_planted_mistakes():
    """A key too many, a missing scale, another window or a head's neighbour is far outside the bounds."""
    gen = torch.Generator().manual_seed(1)
    q, k, v, do = (torch.randn(40, h, 64, generator=gen).bfloat16() for h in (4, 2, 2, 4))
    spans = [(0, 25), (25, 15)]
    ref = R.attention(q, k, v, spans, 8, 0.125, do)
    for wrong in (R.attention(q, k, v, spans, 9, 0.125, do), R.attention(q, k, v, spans, 8, 0.13, do),
                  R.attention(q, k, v, [(0, 40)], 8, 0.125, do), R.attention(q, k.flip(1), v, spans, 8, 0.125, do)):
        for n in ("o", "dq", "dk", "dv"):
            if torch.equal(wrong[n], ref[n]):
                continue
            with pytest.raises(AssertionError):
                R.check(wrong[n], ref[n], ref[n + "_tol"], n)
    for n in ("o", "dq", "dk", "dv"):  # and its own rounding to bf16 is inside
        R.check(ref[n].bfloat16(), ref[n], ref[n + "_tol"], n)


def test_reference_e4m3_matches_the_cast():
    x = torch.cat([torch.linspace(-448, 448, 4001), torch.logspace(-12, 2.6, 2000), torch.tensor([0.0, 2 ** -10, 3 * 2.0 ** -10])])
    assert torch.equal(R.e4m3(x).float(), x.to(torch.float8_e4m3fn).float())


def test_reference_rotation_is_a_rotation():
    gen = torch.Generator().manual_seed(2)
    x = torch.randn(6, 3, 16, generator=gen)
    pos = torch.arange(6, dtype=torch.int32) * 1000
    inv = torch.tensor([1.0, 0.1, 0.01, 0.001])
    for inter in (False, True):
        y = R.rope(x, None, pos, inv, inter, 0.0, 1.0, False)
        assert torch.allclose(y.norm(dim=-1), x.double().norm(dim=-1), atol=1e-12)
        assert torch.equal(y[..., 8:], x.double()[..., 8:]) and torch.equal(y[0], x.double()[0])
        back = R.rope(y, None, -pos, inv, inter, 0.0, 1.0, False)
        assert torch.allclose(back, x.double(), atol=1e-12)
