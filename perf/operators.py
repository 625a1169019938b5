"""The attention layer of a hybrid stack, next to the recurrence: what is measured of its operators.

A hybrid stack interleaves the library's recurrent layers with sliding-window or full softmax
attention layers.  Four operators make such a layer, in training and in serving:

  rope    per-head RMS norm of q and k with the rotation by position, and its backward pass
  attn    causal attention over whole sequences (fixed length or packed, grouped heads, an
          optional window), and its backward pass
  cache   new keys and values written into a paged cache (bf16, or e4m3 with one scale per token
          and head) and read back from it
  cached  attention of each sequence's newest tokens (one, or a chunk) over the paged cache

`own` false computes the plain forms with elementary torch operations; `own` true makes the calls
of gated_delta_rule_78_b200 a user makes.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def _lens(n, lo, hi):
    """n lengths spread evenly over the logarithm between lo and hi, in an order of their own."""
    r = random.Random(n * 1000003 + lo * 1009 + hi)
    return [max(lo, min(hi, round(math.exp(r.uniform(math.log(lo), math.log(hi)))))) for _ in range(n)]


def _ints(text):
    return [int(x) for x in text.split(",")]


def listed():
    return [
        # one decode step of 256 sequences: their new token's queries and keys, far positions
        {"name": "rope_decode_256", "op": "rope", "dt": "bf16", "n": 256, "h": 16, "hkv": 4, "d": 128, "rot": 128,
         "interleaved": False, "grad": False, "far": 131072},
        # a training step's pass over 8 x 4096 tokens, forward and backward
        {"name": "rope_step_8x4k", "op": "rope", "dt": "bf16", "n": 32768, "h": 16, "hkv": 16, "d": 128, "rot": 128,
         "interleaved": False, "grad": True, "far": 4096},
        # fp32, interleaved pairs, half of a small head rotated, an odd number of tokens
        {"name": "rope_step_f32_part", "op": "rope", "dt": "f32", "n": 4099, "h": 16, "hkv": 4, "d": 64, "rot": 32,
         "interleaved": True, "grad": True, "far": 32768},
        # prompts of very different lengths packed into one prefill, full causal, grouped heads
        {"name": "attn_prompt_packed", "op": "attn", "dt": "bf16", "lens": "5003,1,2048,129,777,64,170", "packed": True,
         "h": 16, "hkv": 4, "d": 128, "window": 0, "grad": False},
        # a training step of the layer at 4K tokens with the hybrid stack's 2K window
        {"name": "attn_step_4x4k_w2k", "op": "attn", "dt": "bf16", "lens": "4096,4096,4096,4096", "packed": False,
         "h": 16, "hkv": 16, "d": 128, "window": 2048, "grad": True},
        # a packed training step with the small head size, grouped heads, odd lengths, no window
        {"name": "attn_step_d64_packed", "op": "attn", "dt": "bf16", "lens": "1900,1025,37,1137", "packed": True,
         "h": 32, "hkv": 8, "d": 64, "window": 0, "grad": True},
        # a small fp32 step, as a numerics check of a model runs it
        {"name": "attn_step_f32", "op": "attn", "dt": "f32", "lens": "500,500", "packed": False, "h": 4, "hkv": 2,
         "d": 64, "window": 0, "grad": True},
        # one decode step's keys and values of 256 sequences, quantised as they are written, read back
        {"name": "cache_step_256_e4m3", "op": "cache", "type": "e4m3", "nseq": 256, "qlo": 1, "qhi": 1, "lo": 64,
         "hi": 1024, "page": 64, "hkv": 4, "d": 128},
        # the prompts' keys and values written into a bf16 cache of small pages
        {"name": "cache_prompt_bf16", "op": "cache", "type": "bf16", "nseq": 12, "qlo": 300, "qhi": 4096, "lo": 4096,
         "hi": 6000, "page": 16, "hkv": 8, "d": 128},
        # one decode step of 256 sequences over an e4m3 cache, lengths from short to 8K
        {"name": "cached_step_256_e4m3", "op": "cached", "type": "e4m3", "nseq": 256, "qlo": 1, "qhi": 1, "lo": 256,
         "hi": 8192, "page": 64, "h": 16, "hkv": 4, "d": 128, "window": 0},
        # one sequence's decode step over a long bf16 cache: few rows, one long axis
        {"name": "cached_step_1x32k", "op": "cached", "type": "bf16", "nseq": 1, "qlo": 1, "qhi": 1, "lo": 32768,
         "hi": 32768, "page": 16, "h": 16, "hkv": 4, "d": 128, "window": 0},
        # chunks of new tokens (a prefill in pieces) over 8K to 16K cached ones
        {"name": "cached_chunk_4x512", "op": "cached", "type": "bf16", "nseq": 4, "qlo": 512, "qhi": 512, "lo": 8192,
         "hi": 16384, "page": 64, "h": 16, "hkv": 4, "d": 128, "window": 0},
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    """One more case, no dearer than the largest of listed()."""
    most = [max(work(c)[k] for c in listed()) for k in ("bytes", "flops")]
    while True:
        c = _draw(rng)
        w = work(c)
        if w["bytes"] <= most[0] and w["flops"] <= most[1]:
            return c


def _draw(rng):
    op = rng.choice(["rope", "attn", "attn", "cache", "cached", "cached"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    h = hkv * rng.choice([1, 2, 3, 4, 8]) if hkv < 8 else hkv * rng.choice([1, 2])
    if op == "rope":
        return {"op": op, "dt": rng.choice(["bf16", "bf16", "f32"]), "n": _logint(rng, 1, 20000), "h": h, "hkv": hkv,
                "d": d, "rot": rng.choice([d, d, d // 2, 2 * rng.randint(1, d // 2)]),
                "interleaved": rng.random() < 0.5, "grad": rng.random() < 0.6, "far": _logint(rng, 64, 500000)}
    if op == "attn":
        dt = rng.choice(["bf16", "bf16", "bf16", "f32"])
        total = _logint(rng, 16, 6000) if dt == "bf16" else _logint(rng, 16, 700)
        packed = rng.random() < 0.6
        n = rng.randint(1, 6)
        if packed:
            lens = [max(1, x * total // 4000) for x in _lens(n, rng.randint(1, 50), 4000)]
        else:
            lens = [max(1, total // n)] * n
        # a query that sees itself alone has no gradient but rounding: such rows come beside others
        lens[0] = max(2, lens[0]) if packed else lens[0]
        grad = rng.random() < 0.6 and max(lens) > 1
        return {"op": op, "dt": dt, "lens": ",".join(map(str, lens)), "packed": packed, "h": h, "hkv": hkv, "d": d,
                "window": rng.choice([0, 0, _logint(rng, 2, 2048)]), "grad": grad}
    chunk = rng.random() < 0.4
    nseq = _logint(rng, 1, 8) if chunk else _logint(rng, 1, 128)
    lo = _logint(rng, 1, 2000)
    c = {"op": op, "type": rng.choice(["bf16", "e4m3"]), "nseq": nseq, "qlo": 1, "qhi": _logint(rng, 2, 700) if chunk else 1,
         "lo": lo, "hi": _logint(rng, lo, 8192), "page": rng.choice([8, 16, 32, 48, 64, 128, 256]), "hkv": hkv, "d": d}
    if op == "cached":
        c.update(h=h, window=rng.choice([0, 0, _logint(rng, 1, 2048)]))
    return c


# ---------------------------------------------------------------- sizes that follow from a case
def _spans(c):
    """Of a cache case: each sequence's new tokens and its length with them."""
    q = _lens(c["nseq"], c["qlo"], c["qhi"])
    old = _lens(c["nseq"], c["lo"], c["hi"])
    return q, [max(a, b) for a, b in zip(q, old)]


def _pairs(qlen, kvlen, window):
    """Visible (query, key) pairs of a sequence whose qlen queries are its last positions."""
    first = kvlen - qlen
    if not window:
        return qlen * first + qlen * (qlen + 1) // 2
    return sum(min(window, p + 1) for p in range(first, kvlen))


def _touched(qlen, kvlen, window):
    """Keys that at least one of those queries sees."""
    return kvlen if not window else min(kvlen, qlen + window - 1)


def work(c):
    if c["op"] == "rope":
        es = 2 if c["dt"] == "bf16" else 4
        n = c["n"] * (c["h"] + c["hkv"]) * c["d"]
        small = 2 * c["d"] * 4 + c["n"] * 4 + c["rot"] * 2
        # forward: read, write; backward: x and the gradient read, the gradient written
        return {"bytes": n * es * (5 if c["grad"] else 2) + small * (3 if c["grad"] else 1), "flops": n * (25 if c["grad"] else 8)}
    if c["op"] == "attn":
        es = 2 if c["dt"] == "bf16" else 4
        lens = _ints(c["lens"])
        t = sum(lens)
        pairs = sum(_pairs(x, x, c["window"]) for x in lens)
        qo, kv = t * c["h"] * c["d"] * es, t * c["hkv"] * c["d"] * es
        b = 2 * qo + 2 * kv + t * c["h"] * 4
        f = 4 * pairs * c["h"] * c["d"]
        if c["grad"]:  # q, k, v, o, do, lse read; dq, dk, dv written; five products
            b += 4 * qo + 4 * kv + t * c["h"] * 4
            f += 10 * pairs * c["h"] * c["d"]
        return {"bytes": b, "flops": f}
    q, kv = _spans(c)
    row = c["hkv"] * c["d"] * (2 if c["type"] == "bf16" else 1) + (4 * c["hkv"] if c["type"] == "e4m3" else 0)
    if c["op"] == "cache":
        new = sum(q) * c["hkv"] * c["d"] * 2
        if c["type"] == "bf16":  # k and v read, written to the pages
            return {"bytes": 2 * new + 2 * sum(q) * row, "flops": 0}
        return {"bytes": 4 * new + 4 * sum(q) * row, "flops": 8 * sum(q) * c["hkv"] * c["d"]}
    pairs = sum(_pairs(a, b, c["window"]) for a, b in zip(q, kv))
    keys = sum(_touched(a, b, c["window"]) for a, b in zip(q, kv))
    return {"bytes": 2 * keys * row + sum(q) * c["h"] * (4 * c["d"] + 4), "flops": 4 * pairs * c["h"] * c["d"]}


# ---------------------------------------------------------------- inputs
def _cu(lens, dev):
    out = [0]
    for x in lens:
        out.append(out[-1] + x)
    return torch.tensor(out, dtype=torch.int32, device=dev)


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    host = random.Random(seed)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device=dev).to(dtype)

    d, hkv = c["d"], c["hkv"]
    if c["op"] == "rope":
        dt, n, h = DT[c["dt"]], c["n"], c["h"]
        s = {"c": c, "q": normal(n, h, d, dtype=dt), "k": normal(n, hkv, d, dtype=dt),
             "wq": 1 + 0.1 * normal(d, dtype=torch.float32), "wk": 1 + 0.1 * normal(d, dtype=torch.float32),
             "pos": torch.randint(0, c["far"], (n,), generator=g, device=dev, dtype=torch.int32),
             "inv": torch.tensor([10000.0 ** (-2 * i / c["rot"]) for i in range(c["rot"] // 2)], device=dev)}
        if c["grad"]:
            s.update(dqo=normal(n, h, d, dtype=dt), dko=normal(n, hkv, d, dtype=dt))
        return s
    if c["op"] == "attn":
        dt, h, lens = DT[c["dt"]], c["h"], _ints(c["lens"])
        lead = (sum(lens),) if c["packed"] else (len(lens), lens[0])
        s = {"c": c, "q": normal(*lead, h, d, dtype=dt), "k": normal(*lead, hkv, d, dtype=dt),
             "v": normal(*lead, hkv, d, dtype=dt), "cu": _cu(lens, dev) if c["packed"] else None}
        if c["grad"]:
            s["do"] = normal(*lead, h, d, dtype=dt)
        return s
    q, kv = _spans(c)
    page = c["page"]
    need = [-(-x // page) for x in kv]
    width, pages = max(need), sum(need) + 3
    order = list(range(pages))
    host.shuffle(order)
    table, at = [], 0
    for x in need:
        table.append(order[at:at + x] + [0] * (width - x))
        at += x
    s = {"c": c, "cu": _cu(q, dev), "kv_lens": torch.tensor(kv, dtype=torch.int32, device=dev),
         "table": torch.tensor(table, dtype=torch.int32, device=dev), "total": sum(q), "ks": None, "vs": None}
    kc, vc = (normal(pages, page, hkv, d) for _ in range(2))
    if c["type"] == "e4m3":
        s["kc"], s["ks"] = _quantise(kc)
        s["vc"], s["vs"] = _quantise(vc)
    else:
        s["kc"], s["vc"] = kc, vc
    if c["op"] == "cache":
        s.update(k=normal(s["total"], hkv, d), v=normal(s["total"], hkv, d))
    else:
        s["q"] = normal(s["total"], c["h"], d)
    return s


# ---------------------------------------------------------------- the plain forms
def _quantise(x):
    """e4m3 values and the fp32 scale of each row: its largest magnitude over 448."""
    x = x.float()
    scale = x.abs().amax(-1) / 448
    return (x / torch.where(scale > 0, scale, 1)[..., None]).to(torch.float8_e4m3fn), scale


def _angles(s):
    a = s["pos"].double()[:, None, None] * s["inv"].double()
    return a.cos().float(), a.sin().float()


def _rotate(x, cos, sin, rot, interleaved):
    y = x.clone()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def _plain_rope_one(s, x, w, grad):
    c = s["c"]
    cos, sin = _angles(s)
    f = x.float()
    r = torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS)
    out = _rotate(f * r * w, cos, sin, c["rot"], c["interleaved"]).to(x.dtype)
    if grad is None:
        return out, None, None
    u = _rotate(grad.float(), cos, -sin, c["rot"], c["interleaved"])
    dw = (u * f * r).sum((0, 1), dtype=torch.float64).float()
    uw = u * w
    dx = r * (uw - f * (r * r) * (uw * f).mean(-1, keepdim=True))
    return out, dx.to(x.dtype), dw


def _plain_rope(s):
    qo, dq, dwq = _plain_rope_one(s, s["q"], s["wq"], s.get("dqo"))
    ko, dk, dwk = _plain_rope_one(s, s["k"], s["wk"], s.get("dko"))
    return [qo, ko] if dq is None else [qo, ko, dq, dk, dwq, dwk]


def _scores(q, k, mask):
    """Softmax weights and their log-sum of q [.., Tq, Hkv, G, D] over k [.., Tk, Hkv, D], mask [.., Tq, Tk]."""
    sc = torch.einsum("...qhgd,...khd->...hgqk", q, k) * q.shape[-1] ** -0.5
    sc = sc.masked_fill(~mask[..., None, None, :, :], -math.inf)
    top = sc.amax(-1, keepdim=True)
    e = torch.exp(sc - top)
    total = e.sum(-1, keepdim=True)
    return e / total, (top + torch.log(total))[..., 0]


def _plain_attn(s):
    c = s["c"]
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    t = q.shape[-3]
    i = torch.arange(t, device=q.device)
    mask = i[None, :] <= i[:, None]
    if c["window"]:
        mask &= i[None, :] > i[:, None] - c["window"]
    if c["packed"]:
        seq = torch.searchsorted(s["cu"], i, right=True)
        mask &= seq[:, None] == seq[None, :]
    qg = q.unflatten(-2, (c["hkv"], c["h"] // c["hkv"]))
    p, lse = _scores(qg, k, mask)
    o = torch.einsum("...hgqk,...khd->...qhgd", p, v)
    out = [o.flatten(-3, -2).to(s["q"].dtype), lse.flatten(-3, -2).transpose(-1, -2).contiguous()]
    if c["grad"]:
        do = s["do"].float().unflatten(-2, (c["hkv"], c["h"] // c["hkv"]))
        dv = torch.einsum("...hgqk,...qhgd->...khd", p, do)
        ds = torch.einsum("...qhgd,...khd->...hgqk", do, v)
        ds -= torch.einsum("...qhgd,...qhgd->...hgq", do, o)[..., None]
        ds *= p
        ds *= c["d"] ** -0.5
        dq = torch.einsum("...hgqk,...khd->...qhgd", ds, k).flatten(-3, -2)
        dk = torch.einsum("...hgqk,...qhgd->...khd", ds, qg)
        out += [x.to(s["q"].dtype) for x in (dq, dk, dv)]
    return out


def _new_rows(s):
    """Sequence and position of every new token, and its page and row there."""
    c = s["c"]
    tok = torch.arange(s["total"], device=s["cu"].device)
    seq = torch.searchsorted(s["cu"][1:], tok, right=True)
    pos = s["kv_lens"][seq] - s["cu"][seq + 1] + tok
    return seq, pos, s["table"][seq, pos // c["page"]].long(), pos % c["page"]


def _plain_cache(s):
    _, _, page, row = _new_rows(s)
    if s["c"]["type"] == "bf16":
        s["kc"][page, row] = s["k"]
        s["vc"][page, row] = s["v"]
        return [s["kc"], s["vc"]]
    back = []
    for x, cache, scale in ((s["k"], s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])):
        y, scale[page, row] = _quantise(x)
        cache.view(torch.uint8)[page, row] = y.view(torch.uint8)
        back.append((cache.view(torch.uint8)[page, row].view(torch.float8_e4m3fn).float() * scale[page, row][..., None]).to(x.dtype))
    return back + [s["ks"], s["vs"]]


def _plain_cached(s):
    c = s["c"]
    dev = s["q"].device
    most, page = int(s["table"].shape[1]) * c["page"], c["page"]
    at = torch.arange(most, device=dev)
    pages = s["table"][:, at // page].long()
    k, v = (x.view(torch.uint8)[pages, at % page].view(torch.float8_e4m3fn).float() * y[pages, at % page][..., None]
            if y is not None else x[pages, at % page].float() for x, y in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
    seq, pos, _, _ = _new_rows(s)
    slot = torch.arange(s["total"], device=dev) - s["cu"][seq]
    lens = s["cu"][1:] - s["cu"][:-1]
    rows = max(_lens(c["nseq"], c["qlo"], c["qhi"]))
    q = torch.zeros(c["nseq"], rows, c["hkv"], c["h"] // c["hkv"], c["d"], device=dev)
    q[seq, slot] = s["q"].float().unflatten(1, (c["hkv"], -1))
    where = (s["kv_lens"] - lens)[:, None] + torch.arange(rows, device=dev)
    mask = at <= where[..., None]
    if c["window"]:
        mask &= at > where[..., None] - c["window"]
    live = (at < s["kv_lens"][:, None])[..., None, None]
    p, lse = _scores(q, torch.where(live, k, 0), mask)
    o = torch.einsum("...hgqk,...khd->...qhgd", p, torch.where(live, v, 0))
    lse = lse.flatten(1, 2).transpose(1, 2)
    return [o[seq, slot].flatten(1, 2).to(s["q"].dtype), lse[seq, slot].contiguous()]


# ---------------------------------------------------------------- the framework's calls
def _own_rope(s):
    import gated_delta_rule_78_b200 as gdn2
    c = s["c"]
    flags = gdn2.ROPE_RMSNORM | (gdn2.ROPE_INTERLEAVED if c["interleaved"] else 0)
    qo, ko = gdn2.gdn2_qk_rope(s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["inv"], flags=flags, eps=EPS)
    if not c["grad"]:
        return [qo, ko]
    g = gdn2.gdn2_qk_rope_bwd(s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["inv"], s["dqo"], s["dko"], flags=flags,
                              eps=EPS)
    return [qo, ko, g["dq"], g["dk"], g["dq_weight"], g["dk_weight"]]


def _own_attn(s):
    import gated_delta_rule_78_b200 as gdn2
    c = s["c"]
    q, k, v, w = s["q"], s["k"], s["v"], c["window"]
    if c["packed"]:
        o, lse = gdn2.gdn2_attn_fwd_varlen(q, k, v, s["cu"], window=w)
    else:
        o, lse = gdn2.gdn2_attn_fwd(q, k, v, window=w)
    if not c["grad"]:
        return [o, lse]
    if c["packed"]:
        g = gdn2.gdn2_attn_bwd_varlen(q, k, v, o, lse, s["do"], s["cu"], window=w)
    else:
        g = gdn2.gdn2_attn_bwd(q, k, v, o, lse, s["do"], window=w)
    return [o, lse, g["dq"], g["dk"], g["dv"]]


def _own_cache(s):
    import gated_delta_rule_78_b200 as gdn2
    gdn2.gdn2_cache_write(s["k"], s["v"], s["kc"], s["vc"], s["cu"], s["kv_lens"], s["table"], s["ks"], s["vs"])
    if s["c"]["type"] == "bf16":
        return [s["kc"], s["vc"]]
    k, v = gdn2.gdn2_cache_read(s["kc"], s["vc"], s["cu"], s["kv_lens"], s["table"], s["ks"], s["vs"], total_T=s["total"])
    return [k, v, s["ks"], s["vs"]]


def _own_cached(s):
    import gated_delta_rule_78_b200 as gdn2
    o, lse = gdn2.gdn2_attn_cached(s["q"], s["kc"], s["vc"], s["cu"], s["kv_lens"], s["table"], s["ks"], s["vs"],
                                   window=s["c"]["window"])
    return [o, lse]


_PLAIN = {"rope": _plain_rope, "attn": _plain_attn, "cache": _plain_cache, "cached": _plain_cached}
_OWN = {"rope": _own_rope, "attn": _own_attn, "cache": _own_cache, "cached": _own_cached}


def run(s):
    return (_OWN if own else _PLAIN)[s["c"]["op"]](s)


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_rope(s):
    c = s["c"]
    half = c["rot"] // 2
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=s["q"].device),
                       s["pos"].double()[:, None] * s["inv"].double()[None, :])[:, None, :]

    def f(x, w):
        y = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / c["d"] + EPS) * w
        z, rest = y[..., :c["rot"]], y[..., c["rot"]:]
        z = z.unflatten(-1, (half, 2)) if c["interleaved"] else z.unflatten(-1, (2, half)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
        z = z if c["interleaved"] else z.transpose(-1, -2)
        return torch.cat([z.flatten(-2), rest], -1)

    outs, dxs, dws = [], [], []
    for x, w, g in ((s["q"], s["wq"], s.get("dqo")), (s["k"], s["wk"], s.get("dko"))):
        x, w = x.double().requires_grad_(), w.double().requires_grad_()
        y = f(x, w)
        outs.append(y.detach())
        if g is not None:
            dx, dw = torch.autograd.grad(y, (x, w), g.double())
            dxs.append(dx)
            dws.append(dw)
    return outs + dxs + dws


def _softmax64(q, k, v, first, window):
    """One head: queries at positions first, first + 1, ..; keys at 0, 1, ..  Returns o and the log-sum."""
    i = first + torch.arange(q.shape[0], device=q.device)[:, None]
    j = torch.arange(k.shape[0], device=q.device)[None, :]
    hidden = j > i
    if window:
        hidden = hidden | (i - j >= window)
    z = (q @ k.T / math.sqrt(q.shape[1])).masked_fill(hidden, -math.inf)
    lse = torch.logsumexp(z, 1)
    return torch.exp(z - lse[:, None]) @ v, lse


def _exact_attn(s):
    c = s["c"]
    names = ["q", "k", "v"] + (["do"] if c["grad"] else [])
    flat = {n: s[n].double().flatten(0, -3) for n in names}
    t, group = flat["q"].shape[0], c["h"] // c["hkv"]
    o, lse = torch.empty_like(flat["q"]), torch.empty(t, c["h"], dtype=torch.float64, device=s["q"].device)
    grads = [torch.zeros_like(flat[n]) for n in ("q", "k", "v")]
    at = 0
    for n in _ints(c["lens"]):
        rows = slice(at, at + n)
        for head in range(c["h"]):
            x = [flat["q"][rows, head], flat["k"][rows, head // group], flat["v"][rows, head // group]]
            x = [y.clone().requires_grad_(c["grad"]) for y in x]
            oo, ll = _softmax64(*x, 0, c["window"])
            o[rows, head], lse[rows, head] = oo.detach(), ll.detach()
            if c["grad"]:
                for y, dy, hh in zip(grads, torch.autograd.grad(oo, x, flat["do"][rows, head]), (head, head // group, head // group)):
                    y[rows, hh] += dy
        at += n
    out = [o.view(s["q"].shape), lse.view(s["q"].shape[:-1])]
    return out + [g.view(s[n].shape) for g, n in zip(grads, ("q", "k", "v"))] if c["grad"] else out


def _e4m3_64(x):
    """x rounded to e4m3 in 64 bits (ties to even), |x| at most 448."""
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def _exact_cache(s):
    c = s["c"]
    q, kv = _spans(c)
    table, tok, where = s["table"].tolist(), 0, []
    for n, (a, b) in enumerate(zip(q, kv)):
        where += [table[n][p // c["page"]] * c["page"] + p % c["page"] for p in range(b - a, b)]
    where = torch.tensor(where, device=s["k"].device)
    outs, scales = [], []
    for x, cache, scale in ((s["k"], s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])):
        x = x.double()
        if c["type"] == "bf16":
            y = cache.double().flatten(0, 1)
            y[where] = x
            outs.append(y.view(cache.shape))
            continue
        top = x.abs().amax(-1) / 448
        outs.append(_e4m3_64(x / top[..., None]) * top[..., None])
        y = scale.double().flatten(0, 1)
        y[where] = top
        scales.append(y.view(scale.shape))
    return outs + scales


def _exact_cached(s):
    c = s["c"]
    q, kv = _spans(c)
    table = s["table"].tolist()
    group = c["h"] // c["hkv"]
    o = torch.empty(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device=s["q"].device)
    at = 0
    for n, (a, b) in enumerate(zip(q, kv)):
        use = torch.tensor(table[n][:-(-b // c["page"])], device=s["q"].device)
        k, v = (x[use].double().flatten(0, 1)[:b] for x in (s["kc"], s["vc"]))
        if c["type"] == "e4m3":
            k, v = (x * y[use].double().flatten(0, 1)[:b, :, None] for x, y in ((k, s["ks"]), (v, s["vs"])))
        for head in range(c["h"]):
            kh, vh = k[:, head // group], v[:, head // group]
            o[at:at + a, head], lse[at:at + a, head] = _softmax64(s["q"][at:at + a, head].double(), kh, vh, b - a, c["window"])
        at += a
    return [o, lse]


def exact(c, seed):
    return {"rope": _exact_rope, "attn": _exact_attn, "cache": _exact_cache, "cached": _exact_cached}[c["op"]](prepare(c, seed))
