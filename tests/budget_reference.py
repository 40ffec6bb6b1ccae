"""Plain 64-bit forms of the operators that hold a paged cache to a budget of
rows, one conversation, head and row at a time, with bounds on an
implementation's error, for the tests."""
import math

import numpy as np

from tests.paged_reference import HALF_BF16, page_at, rope
from trained_kv_prefix_gb300 import synth

# Relative error of a logit's terms: the query in two bf16 terms (2^-8 of 2^-8
# of it), f32 products and sums of 128 terms and angles good to 1e-6.
TERMS = HALF_BF16 ** 2 + 1e-5
F32 = 1e-5      # of an exponential and of a sum of them


def sees(x, y, window, sinks):
    """Whether the query at place x sees the key at place y."""
    return y <= x and (window == 0 or y > x - window or y < sinks)


def append(k, v, table, lens, pos, p, N, P, cu=None, theta=synth.ROPE_THETA):
    """{(page, row): (key, value, key's input)} of the rows written, and whether
    a row found no page."""
    out, lost = {}, False
    for b in range(len(lens)):
        rows = (k[cu[b]:cu[b + 1]], v[cu[b]:cu[b + 1]]) if cu is not None else (k[b], v[b])
        for i, (kr, vr) in enumerate(zip(*rows)):
            if lens[b] < 0:
                continue
            at = page_at(table[b], int(lens[b]) + i, N, P)
            lost |= at is None
            if at:
                first = p + lens[b] if pos is None else pos[b]
                out[at] = rope(kr, int(np.clip(first + i, 0, (1 << 24) - 1)), theta), vr, kr
    return out, lost


def weigh(q, lse, kc, k_pages, table, lens, pos=None, window=0, sinks=0, scale=None,
          theta=synth.ROPE_THETA):
    """(weights [B, Hkv, p + rows], their bound, rows held [B])."""
    B, T, Hq, d = q.shape
    N, P, Hkv = k_pages.shape[:3]
    p, M, G = kc.shape[0], table.shape[1], Hq // Hkv
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    w, bound = np.zeros((B, Hkv, p + M * P)), np.zeros((B, Hkv, p + M * P))
    held = np.clip(lens, 0, M * P)
    for b in range(B):
        n = int(held[b])
        at = [(p + r, page_at(table[b], r, N, P)) for r in range(n)]
        at = [(y, x) for y, x in at if x]
        places = np.array(list(range(p)) + [y for y, _ in at], int)
        for i in range(T):
            x = p + n - T + i
            if x < p:
                continue
            see = np.array([sees(x, y, window, sinks) for y in places], bool)
            rot = np.clip(x if pos is None else pos[b] + i, 0, (1 << 24) - 1)
            for g in range(Hkv):
                k = np.concatenate([kc[:, g]] + [k_pages[a][None, g] for _, a in at])[see]
                for h in range(g * G, (g + 1) * G):
                    qr = rope(q[b, i, h], int(rot), theta)
                    e = np.exp(scale * (k @ qr) - lse[b, h, i])
                    off = scale * (np.abs(k) @ np.abs(qr)) * TERMS
                    w[b, g, places[see]] += e
                    bound[b, g, places[see]] += e * (np.expm1(off) + F32)
    return w, bound, held


def decode(q, k_new, v_new, kc, vc, k_pages, v_pages, table, lens, pos=None, window=0, sinks=0,
           scale=None, theta=synth.ROPE_THETA):
    """(o, its bound, weights given [B, Hkv, rows], their bound, {(page, row):
    (key, value)} written, whether a row found no page)."""
    B, Hq, d = q.shape
    N, P, Hkv = k_pages.shape[:3]
    p, M, G = kc.shape[0], table.shape[1], Hq // Hkv
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o, ob = np.zeros(q.shape), np.zeros(q.shape)
    w, wb = np.zeros((B, Hkv, M * P)), np.zeros((B, Hkv, M * P))
    wrote, lost = {}, False
    for b in range(B):
        n = min(int(lens[b]), M * P)
        new = page_at(table[b], n, N, P) if n >= 0 else None
        lost |= n >= 0 and new is None
        if new is None:
            continue
        rot = int(np.clip(p + n if pos is None else pos[b], 0, (1 << 24) - 1))
        kn = rope(k_new[b], rot, theta)
        wrote[new] = kn, v_new[b]
        at = [(r, page_at(table[b], r, N, P)) for r in range(n)]
        at = [(r, x) for r, x in at if x and sees(p + n, p + r, window, sinks)]
        cart = [j for j in range(p) if sees(p + n, j, window, sinks)]
        rows = [r for r, _ in at] + [n]
        for g in range(Hkv):
            k = np.concatenate([kc[cart, g]] + [k_pages[x][None, g] for _, x in at] + [kn[None, g]])
            v = np.concatenate([vc[cart, g]] + [v_pages[x][None, g] for _, x in at] +
                               [v_new[b, g][None]])
            for h in range(g * G, (g + 1) * G):
                qr = rope(q[b, h], rot, theta)
                s = scale * (k @ qr)
                e = np.exp(s - s.max())
                e /= e.sum()
                off = scale * (np.abs(k) @ np.abs(qr)) * TERMS
                off[-1] += scale * (np.abs(k[-1]) @ np.abs(qr)) * HALF_BF16   # the key's rounding
                low = max(0.5, 1 - (e * np.expm1(off)).sum())                 # of the sum
                rel = np.exp(off) / low - 1 + F32
                o[b, h] = e @ v
                ob[b, h] = (e * (rel + HALF_BF16)) @ np.abs(v) * (1 + HALF_BF16) + \
                    HALF_BF16 * np.abs(o[b, h])
                w[b, g, rows] += e[len(cart):]
                wb[b, g, rows] += (e * rel)[len(cart):]
    return o, ob, w, wb, wrote, lost


def evict(table, lens, refs, weights, keep, first, recent, layers, Hkv, P):
    """(table, lens, refs, done, weights, moves, rows): moves [(layer, head,
    (page, row) from, (page, row) to)], rows[b][layer][head] the old rows that
    stay (None: left as it is)."""
    table, lens, refs = table.copy(), lens.copy(), refs.copy()
    weights = None if weights is None else weights.copy()
    (B, M), N = table.shape, len(refs)
    free, shared = [i for i in range(N) if refs[i] <= 0], refs > 1
    room, moves, stay, done = len(free), [], [None] * B, np.ones(B, np.int32)
    old, was = table.copy(), None if weights is None else weights.copy()
    for b in range(B):
        n, k = min(int(lens[b]), M * P), int(keep[b])
        if k < 0 or n <= k:
            continue
        if any(page_at(old[b], r, N, P) is None for r in range(n)):
            done[b] = 0
            continue
        f = min(first, k)
        last = k - f if weights is None else min(recent, k - f)
        end = -(-k // P)
        need = [j for j in range(f // P, end) if shared[old[b, j]]] if f < k else []
        room -= len(need)
        if need and room < 0:
            done[b] = 0
            continue
        for j in need:
            refs[old[b, j]] -= 1
            table[b, j] = free.pop(0)
            refs[table[b, j]] = 1
        for j in range(end, M):
            if 0 <= old[b, j] < N:
                refs[old[b, j]] -= 1
            table[b, j] = -1
        lens[b], stay[b] = k, []
        for layer in range(layers):
            stay[b].append([])
            for g in range(Hkv):
                between = list(range(f, n - last))
                if was is not None:
                    key = [-math.inf if math.isnan(x) else -x
                           for x in was[layer, b, g, f:n - last].tolist()]
                    nan = [math.isnan(x) for x in was[layer, b, g, f:n - last].tolist()]
                    between.sort(key=lambda r: (not nan[r - f], key[r - f], r))
                between = between[:k - f - last]
                rows = sorted(list(range(f)) + between + list(range(n - last, n)))
                stay[b][-1].append(rows)
                for i, r in enumerate(rows):
                    moves.append((layer, g, (old[b, r // P], r % P), (table[b, i // P], i % P)))
                    if was is not None:
                        weights[layer, b, g, i] = was[layer, b, g, r]
    return table, lens, refs, done, weights, moves, stay
