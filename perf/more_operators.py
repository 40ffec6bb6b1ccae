"""Cases of the operators that hold a paged cache to a budget of rows, with
their plain forms.

A conversation's private rows lie in pages of a pool behind one shared
cartridge.  Cartridge row j has place j, private row r place p + r; a query at
place x sees the places up to x, with a window W those above x - W, and always
those below `sinks`.  A token's rotary position is apart from its place, since
rows that were evicted leave no gap.

* ``append``  a prompt's keys (rotated) and values written to page rows;
* ``weigh``   the attention weight that each key gets from a conversation's
              last queries, by their log-sum-exps, set or added up;
* ``evict``   in every layer and kv head the rows of little weight dropped and
              the others moved together, pages given back;
* ``decode``  one new token per conversation: its row appended, attention over
              everything it sees, and the weights that it gives added up.

``run`` computes them in elementary torch operations, or with ``own`` by the
package's entry points.  The tables and weights that ``evict`` changes in place
are copied within the pass, so that a pass can be repeated on one state.
"""
import math

import numpy as np
import torch

own = False

THETA = 1.0e6


# ------------------------------------------------------------------ cases ----
def listed():
    return [
        # one conversation behind the 512-row cartridge of the equivalence
        # gate: latency counts
        dict(name="decode_one_chat", op="decode", B=1, Hq=32, Hkv=8, d=128, p=512, max_len=201,
             page_rows=16, window=0, sinks=0, gone=0),
        # a serving batch whose caches have been evicted before, ragged
        dict(name="decode_budgeted", op="decode", B=96, Hq=32, Hkv=8, d=128, p=2048, max_len=1500,
             page_rows=64, window=0, sinks=0, gone=7001),
        # few long histories, the long-context head layout
        dict(name="decode_long_history", op="decode", B=4, Hq=64, Hkv=8, d=128, p=8192,
             max_len=49159, page_rows=128, window=0, sinks=0, gone=0),
        # a layer of local attention that keeps the cartridge's first rows in
        # sight, groups of seven query heads
        dict(name="decode_window", op="decode", B=200, Hq=28, Hkv=4, d=128, p=1024, max_len=4000,
             page_rows=32, window=1000, sinks=130, gone=0),
        # the last queries of one short conversation
        dict(name="weigh_one_chat", op="weigh", B=1, queries=32, Hq=32, Hkv=8, d=128, p=512,
             max_len=201, page_rows=16, window=0, sinks=0, accumulate=False),
        # the last 32 queries of a serving batch's prompts
        dict(name="weigh_observed", op="weigh", B=64, queries=32, Hq=32, Hkv=8, d=128, p=4096,
             max_len=1031, page_rows=64, window=0, sinks=0, accumulate=False),
        # whole prompts, one chunk after others
        dict(name="weigh_prompt", op="weigh", B=4, queries=1024, Hq=32, Hkv=8, d=128, p=2048,
             max_len=1200, page_rows=64, window=0, sinks=0, accumulate=True),
        # a few tokens of three conversations
        dict(name="append_few", op="append", B=3, n=9, Hkv=8, d=128, p=512, max_len=300,
             page_rows=16, packed=False),
        # ragged prompts of a batch, back to back on one token axis
        dict(name="append_prompts", op="append", B=48, n=2000, Hkv=8, d=128, p=4096, max_len=700,
             page_rows=64, packed=True),
        # a small cache
        dict(name="evict_few", op="evict", B=3, layers=2, Hkv=2, d=64, page_rows=16, max_len=200,
             keep=100, first=4, recent=16, share=1),
        # a serving batch brought back to 512 rows in every layer
        dict(name="evict_serving", op="evict", B=64, layers=16, Hkv=8, d=128, page_rows=64,
             max_len=1100, keep=512, first=4, recent=64, share=1),
        # long histories in pairs of branches that share their pages
        dict(name="evict_long_shared", op="evict", B=6, layers=4, Hkv=8, d=128, page_rows=128,
             max_len=20000, keep=4001, first=16, recent=512, share=2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    heads = [(4, 2, 64), (8, 2, 128), (16, 16, 64), (28, 4, 128), (32, 8, 128), (64, 8, 128),
             (8, 1, 128), (12, 2, 64), (40, 8, 128)]
    op = rng.choice(["decode"] * 3 + ["weigh"] * 2 + ["append", "evict"])
    P = rng.choice([16, 32, 64, 128])
    while True:
        Hq, Hkv, d = rng.choice(heads)
        if op == "evict":
            keep = _log(rng, 16, 4000)
            c = dict(op=op, B=_log(rng, 1, 64), layers=_log(rng, 1, 16), Hkv=Hkv, d=d, page_rows=P,
                     max_len=int(keep * rng.uniform(1.05, 5)) + 8, keep=keep,
                     first=rng.randint(0, 16), recent=int(keep * rng.uniform(0, 0.6)),
                     share=rng.choice([1, 1, 2, 3]))
            if c["B"] * c["layers"] * c["max_len"] * Hkv * d <= 1 << 30:
                return c
            continue
        c = dict(op=op, B=_log(rng, 1, 200), Hkv=Hkv, d=d,
                 p=rng.choice([0, _log(rng, 1, 8192)]) if rng.random() < 0.2 else _log(rng, 64, 8192),
                 max_len=_log(rng, 1, 40000), page_rows=P)
        if op == "append":
            c.update(n=_log(rng, 1, 4000), packed=rng.random() < 0.5)
            if c["B"] * c["n"] * Hkv * d <= 48 << 20 and \
                    c["B"] * (c["n"] + c["max_len"]) * Hkv * d <= 1 << 28:
                return c
            continue
        windowed = rng.random() < 0.3
        c.update(Hq=Hq, window=_log(rng, 64, 4096) if windowed else 0,
                 sinks=rng.choice([0, _log(rng, 1, 300)]) if windowed else 0)
        if op == "decode":
            c.update(gone=rng.choice([0, _log(rng, 1, 100000)]))
            if c["B"] * c["max_len"] * Hkv * d <= 1 << 27:
                return c
            continue
        c.update(queries=_log(rng, 1, 1024), accumulate=rng.random() < 0.5)
        if c["B"] * c["queries"] * Hq * (c["p"] + c["max_len"]) <= 6 << 26 and \
                c["B"] * c["max_len"] * Hkv * d <= 1 << 27:
            return c


# ----------------------------------------------------------------- inputs ----
def _lengths(B, max_len):
    """0 < L <= max_len spread evenly, the longest max_len."""
    return np.array([max(1, max_len * (b + 1) // B) for b in range(B)])


def _normal(g, shape, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16).mul_(std)


def _heavy(g, shape):
    """Accumulated weights: a few keys hold most, some were never looked at."""
    w = torch.randn(shape, generator=g, device="cuda").mul_(2.0).exp_().mul_(1e-2)
    return w.masked_fill_(torch.rand(shape, generator=g, device="cuda") < 0.1, 0.0)


def _ints(x):
    return torch.tensor(np.ascontiguousarray(x), dtype=torch.int32, device="cuda")


def _tables(rng, hold, M, P, share=1, spare=3):
    """A table for conversations that hold hold[b] rows, in groups of `share`
    that share the pages of the group's first as far as both go."""
    n = -(-hold // P)
    first = np.arange(len(hold)) // share * share
    shared = np.where(np.arange(len(hold)) == first, 0, np.minimum(n, n[first]))
    N = int((n - shared).sum()) + spare
    ids, table, at = rng.permutation(N), np.full((len(hold), M), -1, np.int64), 0
    for b in range(len(hold)):
        table[b, :shared[b]] = table[first[b], :shared[b]]
        table[b, shared[b]:n[b]] = ids[at:at + n[b] - shared[b]]
        at += n[b] - shared[b]
    return table, N


def prepare(case, seed):
    s = dict(case)
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, P, Hkv, d = s["B"], s["page_rows"], s["Hkv"], s["d"]
    lens = rng.permutation(_lengths(B, s["max_len"]))
    if s["op"] == "evict":
        M = -(-s["max_len"] // P)
        lens = np.maximum(lens, s["max_len"] // 3)
        keep = np.where(rng.random(B) < 0.05, -1, s["keep"])
        keep[0] = s["keep"]
        table, N = _tables(rng, lens, M, P, s["share"], B * (-(-s["keep"] // P)) + 3)
        refs = np.bincount(table[table >= 0], minlength=N)
        pool = (s["layers"], N, P, Hkv, d)
        s.update(meta=_ints(np.concatenate([table.ravel(), refs, lens])), pages=N, max_pages=M,
                 keeps=_ints(keep), weights=_heavy(g, (s["layers"], B, Hkv, M * P)),
                 k_pages=_normal(g, pool), v_pages=_normal(g, pool))
        return s
    p = s["p"]
    more = {"decode": 1, "weigh": 0}.get(s["op"], s.get("n", 0))
    M = -(-(s["max_len"] + more) // P)
    table, N = _tables(rng, lens + more, M, P)
    s.update(table=_ints(table), lens=_ints(lens), k_pages=_normal(g, (N, P, Hkv, d)))
    if s["op"] == "append":
        s["v_pages"] = _normal(g, (N, P, Hkv, d))
        if s["packed"]:
            cu = np.concatenate([[0], np.cumsum(rng.integers(1, s["n"] + 1, size=B))])
            new = (int(cu[-1]), Hkv, d)
            s.update(cu=_ints(cu))
        else:
            new = (B, s["n"], Hkv, d)
        s.update(k=_normal(g, new), v=_normal(g, new))
        return s
    s.update(kc=_normal(g, (p, Hkv, d)), weights=_heavy(g, (B, Hkv, M * P)))
    if s["op"] == "decode":
        s.update(q=_normal(g, (B, s["Hq"], d), 2.0), k_new=_normal(g, (B, Hkv, d)),
                 v_new=_normal(g, (B, Hkv, d)), vc=_normal(g, (p, Hkv, d)),
                 v_pages=_normal(g, (N, P, Hkv, d)),
                 pos=_ints(p + lens + rng.integers(0, s["gone"] + 1, size=B)))
        return s
    # the log-sum-exps that the attention of these queries came with
    s["q"] = _normal(g, (B, s["queries"], s["Hq"], d), 2.0)
    x, seen = _logits(s)
    s["lse"] = x.masked_fill_(~seen, -math.inf).logsumexp(-1).reshape(B, s["Hq"], -1)
    return s


# ------------------------------------------------------------- plain forms ----
def _rope(x, pos):
    """Rotate-half rotation of x [..., H, d] at positions pos [...]."""
    half = x.shape[-1] // 2
    j = torch.arange(half, dtype=torch.float64, device=x.device)
    ang = pos.double()[..., None, None] * THETA ** (-j / half)
    c, sn = ang.cos().to(x.dtype), ang.sin().to(x.dtype)
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * c - b * sn, b * c + a * sn], -1)


def _rows_of(s, name):
    """A pool's rows by conversation [B, M * P, Hkv, d], and which are there."""
    pages, table = s[name], s["table"].long()
    N, P, Hkv, d = pages.shape
    held = (table >= 0) & (table < N)
    rows = pages[table.clamp(0, N - 1)].view(table.shape[0], -1, Hkv, d)
    return rows, held.repeat_interleave(P, 1)


def _seen(s, place, keys):
    """Whether queries at `place` [B, T] see the keys at places `keys` [n]."""
    x, k = place[:, :, None], keys[None, None]
    m = (k <= x) & (x >= s["p"])
    if s["window"]:
        m &= (k > x - s["window"]) | (k < s["sinks"])
    return m


def _logits(s):
    """Of a weigh case: logits [B, Hkv, G, T, p + rows] and what is seen."""
    q, L, p = s["q"], s["lens"].long(), s["p"]
    B, T, Hq, d = q.shape
    place = p + L[:, None] - T + torch.arange(T, device=q.device)
    qr = _rope(q.float(), place).view(B, T, s["Hkv"], -1, d)
    rows, held = _rows_of(s, "k_pages")
    x = torch.cat([torch.einsum("bthgd,chd->bhgtc", qr, s["kc"].float()),
                   torch.einsum("bthgd,brhd->bhgtr", qr, rows.float())], -1)
    keys = torch.arange(x.shape[-1], device=q.device)
    there = torch.cat([held.new_ones(B, p), held], 1)
    return x.mul_(1.0 / math.sqrt(d)), (_seen(s, place, keys) & there[:, None])[:, None, None]


def _weigh_plain(s):
    x, seen = _logits(s)
    w = x.sub_(s["lse"].view(*x.shape[:-1], 1)).exp_().masked_fill_(~seen, 0.0).sum((2, 3))
    p, old, L = s["p"], s["weights"], s["lens"].long()[:, None]
    r = torch.arange(old.shape[-1], device=old.device)
    add = (r < L - s["q"].shape[1]) if s["accumulate"] else torch.zeros_like(r < L)
    mine = torch.where(add[:, None], old, 0.0) + w[..., p:]
    cart = w[..., :p]
    if s["accumulate"]:
        cart = cart + 0.25
    return [old.copy_(torch.where((r < L)[:, None], mine, old)), cart]


def _decode_plain(s):
    q, table, P, p = s["q"], s["table"], s["page_rows"], s["p"]
    (B, Hq, d), N = q.shape, s["k_pages"].shape[0]
    L, pos, Hkv = s["lens"].long(), s["pos"].long(), s["Hkv"]
    b = torch.arange(B, device=q.device)
    page = table.long()[b, L // P]
    kr = _rope(s["k_new"].float(), pos).to(q.dtype)     # as the cache holds it
    s["k_pages"][page, L % P] = kr
    s["v_pages"][page, L % P] = s["v_new"]
    qr = _rope(q.float(), pos).view(B, Hkv, -1, d)
    (k, held), (v, _) = _rows_of(s, "k_pages"), _rows_of(s, "v_pages")
    x = torch.cat([torch.einsum("bhgd,chd->bhgc", qr, s["kc"].float()),
                   torch.einsum("bhgd,brhd->bhgr", qr, k.float())], -1).mul_(1.0 / math.sqrt(d))
    keys = torch.arange(x.shape[-1], device=q.device)
    seen = _seen(s, p + L[:, None], keys)[:, 0]
    seen[:, p:] &= held
    x = x.masked_fill_(~seen[:, None, None], -math.inf)
    x = x.sub_(x.amax(-1, keepdim=True)).exp_()
    x = x.div_(x.sum(-1, keepdim=True))
    o = torch.einsum("bhgc,chd->bhgd", x[..., :p], s["vc"].float())
    o += torch.einsum("bhgr,brhd->bhgd", x[..., p:], v.float())
    w, r = s["weights"], keys[:k.shape[1]]
    old = torch.where((r < L[:, None])[:, None], w, 0.0)
    w.copy_(torch.where((r <= L[:, None])[:, None], old + x[..., p:].sum(2), w))
    return [o.reshape(B, Hq, d).to(q.dtype), w, s["k_pages"], s["v_pages"]]


def _append_plain(s):
    table, L, P, k, v = s["table"].long(), s["lens"].long(), s["page_rows"], s["k"], s["v"]
    if s["packed"]:
        t = torch.arange(k.shape[0], device=k.device)
        b = torch.searchsorted(s["cu"].long(), t, right=True) - 1
        i = t - s["cu"].long()[b]
    else:
        t = torch.arange(k.shape[0] * k.shape[1], device=k.device)
        b, i = t // k.shape[1], t % k.shape[1]
        k, v = k.flatten(0, 1), v.flatten(0, 1)
    row = L[b] + i
    at = table[b, row // P], row % P
    s["k_pages"][at] = _rope(k.float(), s["p"] + row).to(k.dtype)
    s["v_pages"][at] = v
    return [s["k_pages"], s["v_pages"]]


def _fresh(s):
    """Fresh copies of the tables and weights that an eviction changes."""
    B, M, N = s["B"], s["max_pages"], s["pages"]
    m = s["meta"].clone()
    return m[:B * M].view(B, M), m[B * M:B * M + N], m[B * M + N:], s["weights"].clone()


def _evict_plain(s):
    (table, refs, lens, w), P = _fresh(s), s["page_rows"]
    keep, (B, M), K = s["keeps"].long(), table.shape, s["keep"]
    L = lens.long()
    evict = (keep >= 0) & (L > keep)
    n_first = keep.clamp(max=s["first"])[:, None]
    n_last = torch.minimum(keep[:, None] - n_first, torch.full_like(n_first, s["recent"]))
    r = torch.arange(M * P, device=w.device)
    held = r < L[:, None]
    always = held & ((r < n_first) | (r >= L[:, None] - n_last))
    middle = held & ~always
    order = torch.argsort(torch.where(middle[:, None], w, -1.0), dim=-1, descending=True, stable=True)
    rank = torch.empty_like(order).scatter_(-1, order, r.expand_as(order))
    stays = always[:, None] | (middle[:, None] & (rank < (keep[:, None] - n_first - n_last)[:, None]))
    src = torch.argsort((~stays).to(torch.int8), dim=-1, stable=True)[..., :K]    # [layers, B, Hkv, K]
    # shared pages that rows move into are replaced by free ones, those
    # behind the rows that stay are given back
    k, old = torch.arange(M, device=w.device), table.long()
    end = ((keep + P - 1) // P)[:, None]
    into = evict[:, None] & (k >= n_first // P) & (k < end) & (n_first < keep[:, None])
    swap = into & (refs[old.clamp(min=0)] > 1)
    free = torch.argsort((refs > 0).int(), stable=True)
    nth = (swap.flatten().cumsum(0) - 1).clamp(min=0).view(B, M)
    new = torch.where(swap, free[nth], old)
    back = evict[:, None] & (k >= end) & (old >= 0)
    gone = back | swap
    refs.index_add_(0, old[gone], torch.full_like(old[gone], -1, dtype=refs.dtype))
    refs[new[swap]] = 1
    new = torch.where(back, -1, new)
    i = r[:K]
    moves = evict[:, None] & (i < keep[:, None]) & (i >= n_first // P * P)
    b, dst = moves.nonzero(as_tuple=True)
    to_page, to_row = new[b, dst // P], dst % P
    layer = torch.arange(s["layers"], device=w.device)[None, :, None]
    head = torch.arange(s["Hkv"], device=w.device)[None, None, :]
    frm = src[:, b, :, dst]                                                   # [moves, layers, Hkv]
    from_page = old[b[:, None, None], frm // P]
    for pool in (s["k_pages"], s["v_pages"]):
        pool[layer, to_page[:, None, None], to_row[:, None, None], head] = \
            pool[layer, from_page, frm % P, head]
    w[layer, b[:, None, None], head, dst[:, None, None]] = w[layer, b[:, None, None], head, frm]
    lens = torch.where(evict, keep, L).int()
    return [new.int(), refs, lens, torch.ones_like(lens), w, s["k_pages"], s["v_pages"]]


# --------------------------------------------------------- the package's calls
def _run_own(s):
    from trained_kv_prefix_gb300 import cartattn as ca
    if s["op"] == "decode":
        o = ca.cart_attn_decode_paged(s["q"], s["k_new"], s["v_new"], s["kc"], s["vc"], s["k_pages"],
                                      s["v_pages"], s["table"], s["lens"], pos=s["pos"],
                                      weights=s["weights"], window=s["window"], sinks=s["sinks"],
                                      theta=THETA)
        return [o, s["weights"], s["k_pages"], s["v_pages"]]
    if s["op"] == "weigh":
        cart = torch.full((s["B"], s["Hkv"], s["p"]), 0.25, device="cuda") if s["accumulate"] else None
        return list(ca.cart_attn_weights(s["q"], s["lse"], s["kc"], s["k_pages"], s["table"],
                                         s["lens"], s["weights"], cart, accumulate=s["accumulate"],
                                         window=s["window"], sinks=s["sinks"], theta=THETA))
    if s["op"] == "append":
        return list(ca.cart_pages_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"],
                                         s["lens"], p=s["p"], cu_seqlens=s.get("cu"), theta=THETA))
    table, refs, lens, w = _fresh(s)
    done = ca.cart_pages_evict(s["k_pages"], s["v_pages"], table, lens, refs, w, s["keeps"],
                               first=s["first"], recent=s["recent"])
    return [table, refs, lens, done, w, s["k_pages"], s["v_pages"]]


def run(state):
    if own:
        return _run_own(state)
    return {"decode": _decode_plain, "weigh": _weigh_plain, "append": _append_plain,
            "evict": _evict_plain}[state["op"]](state)


# ------------------------------------------------------------------- work ----
def work(case):
    c = dict(case)
    B, row = c["B"], c["Hkv"] * c["d"] * 2             # bytes of one K (or V) row
    lens = _lengths(B, c["max_len"])
    if c["op"] == "append":
        T = B * (c["n"] + 1) / 2 if c["packed"] else B * c["n"]
        return {"bytes": float(4 * T * row), "flops": 0.0}
    if c["op"] == "evict":
        lens = np.maximum(lens, c["max_len"] // 3)
        out = lens > c["keep"]
        # (few rows before the first that goes)
        moved = (c["keep"] - min(c["first"], c["keep"])) * out.sum()
        return {"bytes": float(c["layers"] * (4 * moved * row + 4 * c["Hkv"] * (lens[out].sum() + moved))),
                "flops": 0.0}
    p, W, S = c["p"], c["window"], c["sinks"]
    T = c.get("queries", 1)
    x = p + lens[:, None] - (T if c["op"] == "weigh" else 0) + np.arange(T)    # places of queries
    low = np.maximum(x - W + 1, 0) if W else np.zeros_like(x)
    see = np.where(x >= p, x + 1 - low + np.minimum(S, low), 0)
    low = np.where(x >= p, low, 1 << 30).min(1)
    own = lens + (1 if c["op"] == "decode" else 0) - np.maximum(low - p, 0)
    cart = min(p, p - min(p, int(low.min())) + min(S, p))
    qo = B * T * c["Hq"] * c["d"] * 2
    if c["op"] == "decode":
        return {"bytes": float(2 * row * (cart + own.sum()) + 8 * c["Hkv"] * own.sum() + 2 * qo + 4 * B * row),
                "flops": float(4 * c["d"] * c["Hq"] * see.sum())}
    return {"bytes": float(row * (cart + own.sum()) + qo + 4 * B * c["Hq"] * T + 4 * c["Hkv"] * (B * p + lens.sum())),
            "flops": float(2 * c["d"] * c["Hq"] * see.sum())}


# ------------------------------------------------------------------ exact ----
def _turn64(x, pos):
    """Rotation by complex numbers of x [n, H, d] at positions pos [n]."""
    half = x.shape[-1] // 2
    f = torch.tensor([THETA ** (-2.0 * j / (2 * half)) for j in range(half)], dtype=torch.float64,
                     device=x.device)
    a = torch.tensor(pos, dtype=torch.float64, device=x.device)[:, None] * f
    z = torch.complex(x[..., :half].double().contiguous(), x[..., half:].double().contiguous())
    z = z * torch.polar(torch.ones_like(a), a)[:, None, :]
    return torch.cat([z.real, z.imag], -1)


def _sight(s, places, n):
    """Truth [len(places), n] of what the queries at those places see."""
    at = torch.arange(n, device="cuda")[None]
    x = torch.tensor(places, device="cuda")[:, None]
    ok = at <= x
    if s["window"]:
        ok &= (x - at < s["window"]) | (at < s["sinks"])
    return ok


def exact(case, seed):
    if case["op"] == "evict":
        return None                     # values are moved, none is computed
    s = prepare(case, seed)
    P, table, lens = s["page_rows"], s["table"].tolist(), s["lens"].tolist()
    kp = s["k_pages"].double()
    vp = s["v_pages"].double() if "v_pages" in s else None

    def rows(pool, b, n):
        ids = torch.tensor(table[b][:-(-n // P)], dtype=torch.int64, device="cuda")
        return pool[ids].flatten(0, 1)[:n]

    if s["op"] == "append":
        cu = s["cu"].tolist() if s["packed"] else [b * s["n"] for b in range(s["B"] + 1)]
        k, v = s["k"].reshape(-1, s["Hkv"], s["d"]), s["v"].reshape(-1, s["Hkv"], s["d"])
        for b in range(s["B"]):
            at = list(range(lens[b], lens[b] + cu[b + 1] - cu[b]))
            turned = _turn64(k[cu[b]:cu[b + 1]], [s["p"] + r for r in at])
            pages = torch.tensor([table[b][r // P] for r in at], device="cuda")
            at = torch.tensor([r % P for r in at], device="cuda")
            kp[pages, at], vp[pages, at] = turned, v[cu[b]:cu[b + 1]].double()
        return [kp, vp]
    p, d, Hkv, G = s["p"], s["d"], s["Hkv"], s["Hq"] // s["Hkv"]
    kc, w = s["kc"].double(), s["weights"].double()
    if s["op"] == "decode":
        o, vc, pos = torch.zeros_like(s["q"], dtype=torch.float64), s["vc"].double(), s["pos"].tolist()
        for b, n in enumerate(lens):
            put = table[b][n // P], n % P
            kp[put] = _turn64(s["k_new"][b:b + 1], pos[b:b + 1])[0].to(torch.bfloat16).double()
            vp[put] = s["v_new"][b].double()
            q = _turn64(s["q"][b:b + 1], pos[b:b + 1])[0].view(Hkv, G, d)
            k, v = torch.cat([kc, rows(kp, b, n + 1)]), torch.cat([vc, rows(vp, b, n + 1)])
            x = torch.matmul(q, k.permute(1, 2, 0)) / math.sqrt(d)
            e = torch.softmax(x.masked_fill(~_sight(s, [p + n], p + n + 1), -math.inf), -1)
            o[b] = torch.matmul(e, v.transpose(0, 1)).reshape(-1, d)
            w[b, :, n] = 0
            w[b, :, :n + 1] += e[..., p:].sum(1)
        return [o, w, kp, vp]
    T, carts = s["queries"], []
    for b, n in enumerate(lens):
        some = list(range(max(0, T - n), T))            # queries that the conversation has
        places = [p + n - T + i for i in some]
        q = _turn64(s["q"][b, some], places)
        k = torch.cat([kc, rows(kp, b, n)])
        got = torch.zeros(Hkv, p + n, dtype=torch.float64, device="cuda")
        for h in range(s["Hq"]):
            x = torch.matmul(q[:, h], k[:, h // G].T) / math.sqrt(d)
            x -= s["lse"][b, h, some].double()[:, None]
            got[h // G] += torch.where(_sight(s, places, p + n), x.exp(), 0.0).sum(0)
        w[b, :, (max(0, n - T) if s["accumulate"] else 0):n] = 0
        w[b, :, :n] += got[:, p:]
        carts.append(got[:, :p] + (0.25 if s["accumulate"] else 0.0))
    return [w, torch.stack(carts)]
