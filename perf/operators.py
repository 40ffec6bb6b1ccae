"""Cases of the paged serving operators, with their plain forms.

The operators keep the private rows of many conversations behind one shared
cartridge in pages of a pool and attend over them:

* ``tree``     attention of a tree of drafted tokens per conversation over the
               cartridge, the conversation's paged rows and the token's own
               ancestors, with the new rows appended (one token, or a chain of
               them, is the plain decode step);
* ``fork``     conversations that share another's pages;
* ``reserve``  room for the rows to come: pages taken from and given back to
               the pool, shared ones copied before they are written;
* ``accept``   the accepted path of a tree moved to follow the cached rows;
* ``compact``  the pool's live pages moved to its front.

``run`` computes them in elementary torch operations, or with ``own`` by the
package's entry points.  The tables that an operator changes in place are
copied within the pass, so that a pass can be repeated on one state.
"""
import math

import numpy as np
import torch

own = False

THETA = 1.0e6


# ------------------------------------------------------------------ cases ----
def listed():
    return [
        # one conversation checks a short draft behind the 512-row cartridge of
        # the equivalence gate: latency counts
        dict(name="tree_one_chat", op="tree", B=1, nodes=8, Hq=32, Hkv=8, d=128, p=512,
             max_len=201, page_rows=16, window=0, chain=False),
        # the benchmark's serving step, its private rows in pages: one token
        # each for 64 conversations behind a 4096-row cartridge
        dict(name="tree_single_tokens", op="tree", B=64, nodes=1, Hq=32, Hkv=8, d=128, p=4096,
             max_len=1024, page_rows=64, window=0, chain=True),
        # long private histories, an odd tree, the long-context head layout
        dict(name="tree_long_history", op="tree", B=4, nodes=25, Hq=64, Hkv=8, d=128, p=8192,
             max_len=49159, page_rows=128, window=0, chain=False),
        # the serving step with the largest tree for every conversation
        dict(name="tree_widest", op="tree", B=64, nodes=64, Hq=32, Hkv=8, d=128, p=4096,
             max_len=1024, page_rows=64, window=0, chain=False),
        # one conversation splits into a few continuations
        dict(name="fork_few", op="fork", B=16, forks=7, max_pages=24, page_rows=16),
        # a search that restarts most of its branches from long parents
        dict(name="fork_many", op="fork", B=1024, forks=700, max_pages=512, page_rows=64),
        # a handful of conversations get room for their next draft
        dict(name="reserve_few", op="reserve", B=6, layers=2, Hkv=2, d=64, page_rows=16,
             max_pages=20, share=2, room=9),
        # 256 branches, four to a parent, are about to write into pages they
        # share, in every layer
        dict(name="reserve_branches", op="reserve", B=256, layers=16, Hkv=8, d=128, page_rows=64,
             max_pages=17, share=4, room=64),
        # drafts of the serving batch accepted in every layer
        dict(name="accept_few", op="accept", B=3, nodes=9, layers=2, Hkv=2, d=64, page_rows=16,
             max_pages=12),
        dict(name="accept_layers", op="accept", B=64, nodes=64, layers=32, Hkv=8, d=128,
             page_rows=64, max_pages=8),
        # a small pool with a few holes, then one that a burst left half empty
        dict(name="compact_few", op="compact", B=5, layers=2, Hkv=2, d=64, page_rows=16, pages=40,
             max_pages=9, live=0.9),
        dict(name="compact_pool", op="compact", B=96, layers=16, Hkv=8, d=128, page_rows=64,
             pages=1200, max_pages=16, live=0.55),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    heads = [(4, 2, 64), (8, 2, 128), (16, 16, 64), (32, 8, 128), (64, 8, 128), (8, 1, 128)]
    op = rng.choice(["tree"] * 4 + ["fork", "reserve", "accept", "compact"])
    P = rng.choice([16, 32, 64, 128])
    Hq, Hkv, d = rng.choice(heads)
    while op == "tree":
        c = dict(op=op, B=_log(rng, 1, 64), nodes=_log(rng, 1, 64), Hq=Hq, Hkv=Hkv, d=d,
                 p=rng.choice([0, _log(rng, 1, 8192)]) if rng.random() < 0.2 else _log(rng, 64, 8192),
                 max_len=_log(rng, 1, 40000), page_rows=P,
                 window=_log(rng, 64, 4096) if rng.random() < 0.2 else 0,
                 chain=rng.random() < 0.25)
        if work(c)["flops"] <= 2.3e11 and c["B"] * c["max_len"] * Hkv * d <= 1 << 28 and \
                c["B"] * c["nodes"] * Hq * (c["p"] + c["max_len"]) <= 7 << 27:
            return c
    if op == "fork":
        B = _log(rng, 4, 1024)
        return dict(op=op, B=B, forks=max(1, int(B * rng.uniform(0.1, 0.7))),
                    max_pages=_log(rng, 4, 512), page_rows=P)
    layers = _log(rng, 1, 24)
    while True:
        B, M = _log(rng, 2, 256), _log(rng, 3, 32)
        if B * M * P * Hkv * d * layers <= 1 << 30:
            break
        layers = max(1, layers // 2)
    if op == "reserve":
        return dict(op=op, B=B, layers=layers, Hkv=Hkv, d=d, page_rows=P, max_pages=M,
                    share=rng.randint(1, 8), room=_log(rng, 1, 96))
    if op == "accept":
        nodes = rng.randint(1, min(64, M * P))
        return dict(op=op, B=B, nodes=nodes, layers=layers, Hkv=Hkv, d=d, page_rows=P, max_pages=M)
    return dict(op=op, B=B, layers=layers, Hkv=Hkv, d=d, page_rows=P, pages=max(4, B * M // 2),
                max_pages=M, live=rng.uniform(0.3, 0.95))


# ----------------------------------------------------------------- inputs ----
def _lengths(B, max_len):
    """0 < L <= max_len spread evenly, the longest max_len."""
    return np.array([max_len * (b + 1) // B for b in range(B)])


def _parents(rng, B, nodes, chain):
    """Trees in which every node follows its parent.  All but the first
    conversation may have fewer nodes than the widest: the rest is unused."""
    t = np.arange(nodes)
    if chain:
        return np.tile(t - 1, (B, 1))
    parents = np.floor(rng.random((B, nodes)) * t).astype(np.int64)
    parents[:, 0] = -1
    used = rng.integers(nodes // 2 + 1, nodes + 1, size=B)
    used[0] = nodes
    return np.where(t < used[:, None], parents, -2)


def _pool(g, shape):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)).mul_(0.5)


def _ints(x):
    return torch.tensor(np.ascontiguousarray(x), dtype=torch.int32, device="cuda")


def _shared_tables(rng, B, M, P, share, hold, N):
    """Conversations in groups of `share` that hold `hold[b]` rows each: the
    group's others share the pages of its first.  The pool has N pages."""
    n = -(-np.asarray(hold) // P)
    first = np.arange(B) - np.arange(B) % share
    shared = np.where(np.arange(B) == first, 0, np.minimum(n, n[first]))
    ids, table, used = rng.permutation(N), np.full((B, M), -1, np.int64), 0
    for b in range(B):
        table[b, :shared[b]] = table[first[b], :shared[b]]
        table[b, shared[b]:n[b]] = ids[used:used + n[b] - shared[b]]
        used += n[b] - shared[b]
    refs = np.bincount(table[table >= 0], minlength=N)
    return table, refs


def prepare(case, seed):
    c = dict(case)
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(c)
    if c["op"] == "tree":
        B, T, P, Hq, Hkv, d, p = (c[k] for k in ("B", "nodes", "page_rows", "Hq", "Hkv", "d", "p"))
        lens = rng.permutation(_lengths(B, c["max_len"]))
        M = -(-(c["max_len"] + T) // P)
        own_pages = -(-(lens + T) // P)
        N = int(own_pages.sum()) + 3
        ids, table, at = rng.permutation(N), np.full((B, M), -1, np.int64), 0
        for b in range(B):
            table[b, :own_pages[b]] = ids[at:at + own_pages[b]]
            at += own_pages[b]
        s.update(q=_pool(g, (B, T, Hq, d)), k_new=_pool(g, (B, T, Hkv, d)),
                 v_new=_pool(g, (B, T, Hkv, d)), kc=_pool(g, (p, Hkv, d)), vc=_pool(g, (p, Hkv, d)),
                 k_pages=_pool(g, (N, P, Hkv, d)), v_pages=_pool(g, (N, P, Hkv, d)),
                 table=_ints(table), lens=_ints(lens),
                 parents=_ints(_parents(rng, B, T, c["chain"])))
        return s
    B, M, P = c["B"], c["max_pages"], c["page_rows"]
    if c["op"] == "fork":
        hold = rng.integers(1, M * P + 1, size=B)
        table, refs = _shared_tables(rng, B, M, P, 1, hold, B * M + 8)
        order = rng.permutation(B)
        dst, free = order[:c["forks"]], order[c["forks"]:]
        src = free[rng.integers(0, len(free), size=len(dst))]
        rows = np.maximum(1, (hold[src] * rng.uniform(0.5, 1.2, size=len(dst)))).astype(np.int64)
        s.update(meta=_ints(np.concatenate([table.ravel(), refs, hold])), pages=len(refs),
                 src=_ints(src), dst=_ints(dst), rows=_ints(rows))
        return s
    pool = (c["layers"], 0, P, c["Hkv"], c["d"])
    if c["op"] == "reserve":
        hold = rng.integers(1, M * P + 1, size=B)
        # branches of the group's first, at its rows or earlier ones
        lens = np.minimum(hold, hold[np.arange(B) - np.arange(B) % c["share"]])
        table, refs = _shared_tables(rng, B, M, P, c["share"], lens,
                                     -(-B // c["share"]) * M + B * (-(-c["room"] // P) + 1))
        rows = np.minimum(lens + c["room"], M * P)
        ends = rng.random(B)
        rows = np.where(ends < 0.06, 0, np.where(ends < 0.1, -1, rows))
        s.update(meta=_ints(np.concatenate([table.ravel(), refs, lens])), pages=len(refs),
                 rows=_ints(rows))
    elif c["op"] == "accept":
        T = c["nodes"]
        lens = rng.integers(0, M * P - T + 1, size=B)
        table, refs = _shared_tables(rng, B, M, P, 1, lens + T, B * M + 2)
        parents = _parents(rng, B, T, False)
        s.update(table=_ints(table), lens=_ints(lens), parents=_ints(parents),
                 node=_ints([_accepted(rng, q) for q in parents]), pages=len(refs))
    else:
        N = c["pages"]
        live = max(1, int(N * c["live"]))
        ids = rng.permutation(N)[:live]
        table = np.full(B * M, -1, np.int64)
        cells = rng.permutation(B * M)
        table[cells[:min(live, B * M)]] = ids[:min(live, B * M)]
        again = cells[live:live + B * M // 8]          # pages of two conversations
        table[again] = ids[rng.integers(0, live, size=len(again))]
        refs = np.bincount(table[table >= 0], minlength=N)
        s.update(meta=_ints(np.concatenate([table, refs])))
        s["pages"] = N
    s["k_pages"] = _pool(g, (pool[0], s["pages"]) + pool[2:])
    s["v_pages"] = _pool(g, (pool[0], s["pages"]) + pool[2:])
    return s


def _accepted(rng, parents):
    """The last accepted node of one tree: a random one whose path's rows are
    not written by the path itself before the pass that repeats them."""
    for t in rng.permutation(len(parents)):
        path, n = [], int(t)
        while n >= 0:
            path.append(n)
            n = int(parents[n])
        path.reverse()
        if n == -1 and all(x == i or x >= len(path) for i, x in enumerate(path)):
            return int(t)
    return -1


def _tables(s):
    """Views of a fresh copy of the tables that the operator changes."""
    B, M, N = s["B"], s["max_pages"], s["pages"]
    m = s["meta"].clone()
    return m[:B * M].view(B, M), m[B * M:B * M + N], m[B * M + N:]


# ------------------------------------------------------------- plain forms ----
def _rope(x, pos):
    """Rotate-half rotation of x [..., H, d] at positions pos [...]."""
    half = x.shape[-1] // 2
    j = torch.arange(half, dtype=torch.float64, device=x.device)
    ang = pos.double()[..., None, None] * THETA ** (-j / half)
    c, sn = ang.cos().to(x.dtype), ang.sin().to(x.dtype)
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * c - b * sn, b * c + a * sn], -1)


def _pages_of(table, N, P, rows):
    """(page id, held?) of the rows [B, R] of every conversation."""
    M = table.shape[1]
    page = table.long().gather(1, (rows // P).clamp(0, M - 1))
    return page, (page >= 0) & (page < N) & (rows >= 0) & (rows < M * P)


def _ancestors(parents, stored):
    """[B, T, T] truth of "j is t or an ancestor of t" over the used nodes: a
    used node's row is stored, and its parents lead to the root through used
    nodes, each before its child."""
    B, T = parents.shape
    t = torch.arange(T, device=parents.device)
    step = (parents[:, :, None] == t) & (t < t[:, None])
    eye = torch.eye(T, dtype=torch.float64, device=parents.device)
    reach = torch.linalg.matrix_power(step.double() + eye, T) > 0
    to_root = (reach & (parents == -1)[:, None, :]).any(-1)
    used = to_root & ~(reach & ~stored[:, None, :]).any(-1)
    return reach & used[:, :, None], used


def _tree_plain(s):
    q, table, P, W, p = s["q"], s["table"], s["page_rows"], s["window"], s["p"]
    (B, T, Hq, d), (N, _, Hkv, _), M = q.shape, s["k_pages"].shape, table.shape[1]
    L = s["lens"].long()
    new_rows = L[:, None] + torch.arange(T, device=q.device)
    page, stored = _pages_of(table, N, P, new_rows)
    anc, used = _ancestors(s["parents"], stored)
    pos = p + L[:, None] + anc.sum(-1) - 1
    qr = _rope(q.float(), pos).view(B, T, Hkv, Hq // Hkv, d)
    kr = _rope(s["k_new"].float(), pos)
    rows = torch.arange(M * P, device=q.device).expand(B, -1)
    held = _pages_of(table, N, P, rows)[1] & (rows < L[:, None])
    at = table.long().clamp(0, N - 1)
    kp, vp = (x[at].view(B, M * P, Hkv, d).float() * held[:, :, None, None]
              for x in (s["k_pages"], s["v_pages"]))
    first = pos - W if W else torch.full_like(pos, -1)      # the last position out of the window
    parts = [(torch.einsum("bthgd,chd->bhgtc", qr, s["kc"].float()),
              torch.arange(p, device=q.device) > first[:, :, None]),
             (torch.einsum("bthgd,brhd->bhgtr", qr, kp),
              held[:, None, :] & (p + rows[:, None, :] > first[:, :, None])),
             (torch.einsum("bthgd,bnhd->bhgtn", qr, kr),
              anc & (pos[:, None, :] > first[:, :, None]))]
    x = torch.cat([a for a, _ in parts], -1).mul_(1.0 / math.sqrt(d))
    seen = torch.cat([m for _, m in parts], -1) & used[:, :, None]
    x = x.masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = x.sum(-1).permute(0, 3, 1, 2)[..., None]
    e = x.split([p, M * P, T], -1)
    o = torch.einsum("bhgtc,chd->bthgd", e[0], s["vc"].float())
    o += torch.einsum("bhgtr,brhd->bthgd", e[1], vp)
    o += torch.einsum("bhgtn,bnhd->bthgd", e[2], s["v_new"].float())
    o = torch.where(total > 0, o / total, 0.0).view(B, T, Hq, d)
    put = (page[used], (new_rows % P)[used])
    s["k_pages"][put] = kr.to(q.dtype)[used]
    s["v_pages"][put] = s["v_new"][used]
    return [o.to(q.dtype), s["k_pages"], s["v_pages"]]


def _fork_plain(s):
    table, refs, lens = _tables(s)
    src, dst, P, (B, M) = s["src"].long(), s["dst"].long(), s["page_rows"], table.shape
    same = dst[:, None] == dst
    done = (same.sum(1) == 1) & ~(dst[:, None] == src).any(1)
    n = torch.minimum(s["rows"], lens[src]).clamp(0, M * P)
    k = torch.arange(M, device=src.device)
    new = torch.where(k < ((n + P - 1) // P)[:, None], table[src], -1)
    old = table[dst]
    for pages, by in ((old, -1), (new, 1)):
        held = (pages >= 0) & done[:, None]
        refs.index_add_(0, torch.where(held, pages, 0).flatten(),
                        (held.flatten() * by).to(refs.dtype))
    table[dst] = torch.where(done[:, None], new, old)
    lens[dst] = torch.where(done, n, lens[dst])
    return [table, refs, lens, done.int()]


def _reserve_plain(s):
    table, refs, lens = _tables(s)
    rows, P, (B, M), N = s["rows"], s["page_rows"], table.shape, len(refs)
    k = torch.arange(M, device=rows.device)
    asks = (rows >= 0) & (rows <= M * P)
    end = (rows + P - 1) // P
    held = table >= 0
    back = asks[:, None] & (k >= end[:, None]) & held
    refs.index_add_(0, torch.where(back, table, 0).flatten(), -back.flatten().to(refs.dtype))
    table.masked_fill_(back, -1)
    lens.copy_(torch.where(asks, torch.minimum(lens.clamp(min=0), rows), lens))
    write = asks[:, None] & (k >= (lens // P)[:, None]) & (k < end[:, None])
    held = table >= 0
    shared = held & (refs[table.clamp(min=0).long()] > 1)
    need = write & (~held | shared)
    free = refs <= 0
    running = need.sum(1).cumsum(0)
    done = asks & ((running <= free.sum()) | ~need.any(1))
    need &= done[:, None]
    order = torch.argsort((~free).int(), stable=True)
    nth = (need.flatten().cumsum(0) - 1).clamp(min=0).view(B, M)
    new = torch.where(need, order[nth.clamp(max=N - 1)].int(), table)
    left = need & shared
    refs.index_add_(0, torch.where(left, table, 0).flatten(), -left.flatten().to(refs.dtype))
    refs[new[need].long()] = 1
    copy = left & (k == (lens // P)[:, None]) & (lens % P > 0)[:, None]
    a, b = table[copy].long(), new[copy].long()
    part = (torch.arange(P, device=rows.device) < (lens % P)[copy.any(1)][:, None])[None, :, :, None, None]
    for pool in (s["k_pages"], s["v_pages"]):
        pool[:, b] = torch.where(part, pool[:, a], pool[:, b])
    return [new, refs, lens, done.int(), s["k_pages"], s["v_pages"]]


def _accept_plain(s):
    table, parents, P, N, L = s["table"], s["parents"], s["page_rows"], s["pages"], s["lens"].long()
    B, T = parents.shape
    rows = L[:, None] + torch.arange(T, device=table.device)
    page, stored = _pages_of(table, N, P, rows)
    anc, used = _ancestors(parents, stored)
    node = s["node"].long()
    path = anc[torch.arange(B, device=table.device), node.clamp(0, T - 1)] & (node >= 0)[:, None]
    to = L[:, None] + path.cumsum(1) - 1
    to_page = _pages_of(table, N, P, to)[0][path]
    at, to = (page[path], (rows % P)[path]), (to_page, (to % P)[path])
    for pool in (s["k_pages"], s["v_pages"]):
        pool[:, to[0], to[1]] = pool[:, at[0], at[1]]
    return [(L + path.sum(1)).int(), s["k_pages"], s["v_pages"]]


def _compact_plain(s):
    table, refs, _ = _tables(s)
    N = len(refs)
    ids = torch.arange(N, device=refs.device)
    live = refs > 0
    n = live.sum()
    a, b = ids[live & (ids >= n)], ids[~live & (ids < n)]
    for pool in (s["k_pages"], s["v_pages"]):
        pool[:, b] = pool[:, a]
    moved = torch.where(live, ids, -1)
    moved[a] = b
    out = torch.where(ids < n, refs, 0)
    out[b] = refs[a]
    table = torch.where(table >= 0, moved[table.clamp(min=0).long()], -1).int()
    return [table, out, moved.int(), n.int().view(1), s["k_pages"], s["v_pages"]]


# --------------------------------------------------------- the package's calls
def _run_own(s):
    from trained_kv_prefix_gb300 import cartattn as ca
    if s["op"] == "tree":
        o = ca.cart_attn_decode_tree(s["q"], s["k_new"], s["v_new"], s["kc"], s["vc"],
                                     s["k_pages"], s["v_pages"], s["table"], s["lens"],
                                     None if s["chain"] else s["parents"], window=s["window"],
                                     theta=THETA)
        return [o, s["k_pages"], s["v_pages"]]
    if s["op"] == "accept":
        lens = ca.cart_pages_accept(s["k_pages"], s["v_pages"], s["table"], s["lens"], s["parents"],
                                    s["node"])
        return [lens, s["k_pages"], s["v_pages"]]
    table, refs, lens = _tables(s)
    if s["op"] == "fork":
        done = ca.cart_pages_fork(table, lens, refs, s["src"], s["dst"], s["rows"],
                                  page_rows=s["page_rows"])
        return [table, refs, lens, done]
    if s["op"] == "reserve":
        done = ca.cart_pages_reserve(s["k_pages"], s["v_pages"], table, lens, refs, s["rows"])
        return [table, refs, lens, done, s["k_pages"], s["v_pages"]]
    moved, live = ca.cart_pages_compact(s["k_pages"], s["v_pages"], table, refs)
    return [table, refs, moved, live, s["k_pages"], s["v_pages"]]


def run(state):
    if own:
        return _run_own(state)
    return {"tree": _tree_plain, "fork": _fork_plain, "reserve": _reserve_plain,
            "accept": _accept_plain, "compact": _compact_plain}[state["op"]](state)


# ------------------------------------------------------------------- work ----
def work(case):
    c = dict(case)
    B, P = c["B"], c["page_rows"]
    if c["op"] == "tree":
        T, p, W, row = c["nodes"], c["p"], c["window"], c["Hkv"] * c["d"] * 2
        lens = _lengths(B, c["max_len"])
        see = p + lens + (T + 1) / 2 if c["chain"] else p + lens + min(T, 3)
        priv, cart = lens, p
        if W:
            see, priv = np.minimum(see, W), np.minimum(lens, W)
            cart = max(0, min(p, W - int(lens.min())))
        used = T if c["chain"] else 0.75 * T
        rows = 2 * row * (cart + priv.sum()) + 2 * 2 * row * used * B
        return {"bytes": float(rows + 4 * B * T * c["Hq"] * c["d"] + 4 * (priv // P).sum()),
                "flops": float(4 * c["d"] * c["Hq"] * used * see.sum())}
    if c["op"] == "fork":
        return {"bytes": 4.0 * c["forks"] * c["max_pages"] * 2.5, "flops": 0.0}
    row = 2 * c["layers"] * c["Hkv"] * c["d"] * 2       # K and V of one row in every layer
    if c["op"] == "reserve":
        copies = 0.9 * B if c["share"] > 1 else 0.0
        return {"bytes": float(copies * P / 2 * row * 2 + 4 * B * c["max_pages"] * 2), "flops": 0.0}
    if c["op"] == "accept":
        return {"bytes": float(B * min(3, c["nodes"]) * row * 2 + 4 * B * c["nodes"]), "flops": 0.0}
    N, live = c["pages"], min(c["live"], B * c["max_pages"] / c["pages"])
    return {"bytes": float(N * live * (1 - live) * P * row * 2 + 8 * B * c["max_pages"] + 12 * N),
            "flops": 0.0}


# ------------------------------------------------------------------ exact ----
def _walk(parents, ok):
    """Paths from the root of the used nodes of one tree, by following each
    node's parents; None for the others."""
    paths = []
    for t, q in enumerate(parents):
        up = None
        if ok[t]:
            up = [] if q == -1 else (paths[q] if 0 <= q < t else None)
        paths.append(None if up is None else up + [t])
    return paths


def _turn64(x, pos):
    """Rotation by complex numbers of x [n, H, d] at positions pos [n]."""
    half = x.shape[-1] // 2
    f = torch.tensor([THETA ** (-2.0 * j / (2 * half)) for j in range(half)], dtype=torch.float64,
                     device=x.device)
    a = torch.tensor(pos, dtype=torch.float64, device=x.device)[:, None] * f
    z = torch.complex(x[..., :half].contiguous(), x[..., half:].contiguous())
    z = z * torch.polar(torch.ones_like(a), a)[:, None, :]
    return torch.cat([z.real, z.imag], -1)


def _exact_tree(s):
    T, P, W, p, d = s["nodes"], s["page_rows"], s["window"], s["p"], s["d"]
    G, dev = s["Hq"] // s["Hkv"], s["q"].device
    table, lens, parents = s["table"].tolist(), s["lens"].tolist(), s["parents"].tolist()
    N = s["k_pages"].shape[0]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    kp, vp = s["k_pages"].double(), s["v_pages"].double()
    for b in range(s["B"]):
        L = lens[b]
        where = [(table[b][r // P], r % P) for r in range(L, L + T)]
        paths = _walk(parents[b], [0 <= pg < N for pg, _ in where])
        nodes = [t for t in range(T) if paths[t] is not None]
        pos = [p + L + len(paths[t]) - 1 for t in nodes]
        q = _turn64(s["q"][b, nodes].double(), pos)
        kn = _turn64(s["k_new"][b, nodes].double(), pos)
        vn = s["v_new"][b, nodes].double()
        ids = torch.tensor(table[b][:-(-L // P)], dtype=torch.int64, device=dev)
        k = torch.cat([s["kc"].double(), kp[ids].flatten(0, 1)[:L], kn])
        v = torch.cat([s["vc"].double(), vp[ids].flatten(0, 1)[:L], vn])
        at = torch.tensor(list(range(p + L)) + pos, device=dev)
        mine = torch.tensor([[u in paths[t] for u in nodes] for t in nodes], device=dev)
        seen = torch.cat([torch.ones(len(nodes), p + L, dtype=torch.bool, device=dev), mine], 1)
        if W:
            seen &= at[None] > torch.tensor(pos, device=dev)[:, None] - W
        for h in range(s["Hkv"]):
            x = torch.matmul(q[:, h * G:(h + 1) * G].transpose(0, 1), k[:, h].T) / math.sqrt(d)
            w = torch.softmax(x.masked_fill(~seen, -math.inf), -1)
            o[b, nodes, h * G:(h + 1) * G] = torch.matmul(w, v[:, h]).transpose(0, 1)
        for i, t in enumerate(nodes):
            kp[where[t]], vp[where[t]] = kn[i], vn[i]
    return [o, kp, vp]


def _exact_pages(s):
    """The page operators one conversation and page at a time."""
    K, V, P = s.get("k_pages"), s.get("v_pages"), s["page_rows"]
    if s["op"] == "accept":
        lens, out = s["lens"].tolist(), []
        table, K2, V2 = s["table"].tolist(), K.clone(), V.clone()
        for b, (q, n) in enumerate(zip(s["parents"].tolist(), s["node"].tolist())):
            path = _walk(q, [True] * len(q))[n] if n >= 0 else []
            for i, t in enumerate(path):
                a, z = lens[b] + t, lens[b] + i
                K2[:, table[b][z // P], z % P] = K[:, table[b][a // P], a % P]
                V2[:, table[b][z // P], z % P] = V[:, table[b][a // P], a % P]
            out.append(lens[b] + len(path))
        return [_ints(out), K2, V2]
    table, refs, lens = (x.tolist() for x in _tables(s))
    if s["op"] == "reserve":
        rows, copies, todo = s["rows"].tolist(), [], []
        for b, n in enumerate(rows):
            if n >= 0:
                for k in range(-(-n // P), len(table[b])):
                    if table[b][k] >= 0:
                        refs[table[b][k]] -= 1
                        table[b][k] = -1
                lens[b] = min(lens[b], n)
                todo.append(b)
        free = [i for i, r in enumerate(refs) if r <= 0]
        before, left, done = list(refs), len(free), [0] * len(rows)
        for b in todo:
            take = [k for k in range(lens[b] // P, -(-rows[b] // P))
                    if table[b][k] < 0 or before[table[b][k]] > 1]
            left -= len(take)
            if take and left < 0:
                continue
            done[b] = 1
            for k in take:
                new, old = free.pop(0), table[b][k]
                if old >= 0:
                    refs[old] -= 1
                    if k == lens[b] // P and lens[b] % P:
                        copies.append((old, new, lens[b] % P))
                table[b][k], refs[new] = new, 1
        K2, V2 = K.clone(), V.clone()
        for a, z, n in copies:
            K2[:, z, :n], V2[:, z, :n] = K[:, a, :n], V[:, a, :n]
        return [_ints(table), _ints(refs), _ints(lens), _ints(done), K2, V2]
    live = [i for i, r in enumerate(refs) if r > 0]
    holes = [i for i in range(len(live)) if refs[i] <= 0]
    moved, out = [i if r > 0 else -1 for i, r in enumerate(refs)], [r if r > 0 else 0 for r in refs]
    K2, V2 = K.clone(), V.clone()
    for z, a in zip(holes, [i for i in live if i >= len(live)]):
        K2[:, z], V2[:, z] = K[:, a], V[:, a]
        moved[a], out[z], out[a] = z, refs[a], 0
    table = [[moved[x] if x >= 0 else -1 for x in r] for r in table]
    return [_ints(table), _ints(out), _ints(moved), _ints([len(live)]), K2, V2]


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "fork":
        return None                     # whole numbers alone
    return _exact_tree(s) if s["op"] == "tree" else _exact_pages(s)
