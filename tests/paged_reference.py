"""Plain 64-bit forms of the paged serving operators, one conversation, node
and page at a time, for the tests."""
import math

import numpy as np

from trained_kv_prefix_gb300 import synth

HALF_BF16 = 2.0 ** -8   # largest relative error of a rounding to bf16


def rope(x, pos, theta=synth.ROPE_THETA):
    """Rotate-half rotation of the head row x [d] at position pos."""
    h = x.shape[-1] // 2
    ang = pos * theta ** (-np.arange(h) / h)
    c, s = np.cos(ang), np.sin(ang)
    return np.concatenate([x[..., :h] * c - x[..., h:] * s, x[..., h:] * c + x[..., :h] * s], -1)


def page_at(table_row, r, N, P):
    """(page, row in it) of a conversation's row r, or None."""
    if r < 0 or r // P >= len(table_row):
        return None
    page = int(table_row[r // P])
    return (page, r % P) if 0 <= page < N else None


def used_nodes(parents, L, table_row, N, P, nodes):
    """Per node the list of its ancestors and itself from the root, or None."""
    paths = []
    for t in range(nodes):
        up = t - 1 if parents is None else int(parents[t])
        path = None
        if L >= 0 and -1 <= up < t and page_at(table_row, min(L, len(table_row) * P) + t, N, P):
            if up == -1:
                path = [t]
            elif paths[up] is not None:
                path = paths[up] + [t]
        paths.append(path)
    return paths


def tree(q, k_new, v_new, kc, vc, k_pages, v_pages, table, lens, parents, window=0, scale=None,
         theta=synth.ROPE_THETA):
    """(o, bound on an implementation's error, {(page, row): (key, value)} of
    the rows written).  All inputs are fp64 arrays.

    The bound holds for bf16 operands with f32 sums: each of the rotated
    query, the rotated new keys, the weights and the output is rounded once
    to bf16 (2^-8 relative), a weight's relative error from the logits' error
    e is at most exp(2 e) - 1 (numerator and sum), and 1e-5 covers the f32
    sums and angles."""
    B, T, Hq, d = q.shape
    Hkv, p = k_new.shape[2], kc.shape[0]
    N, P = k_pages.shape[:2]
    G = Hq // Hkv
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o, bound, wrote = np.zeros(q.shape), np.zeros(q.shape), {}
    for b in range(B):
        L = int(lens[b])
        paths = used_nodes(None if parents is None else parents[b], L, table[b], N, P, T)
        L = min(L, table.shape[1] * P)
        rows = [(p + r, page_at(table[b], r, N, P)) for r in range(max(L, 0))]
        rows = [(pos, at) for pos, at in rows if at]
        for t in range(T):
            if paths[t] is None:
                continue
            wrote[page_at(table[b], L + t, N, P)] = (
                rope(k_new[b, t], p + L + len(paths[t]) - 1, theta), v_new[b, t])
        for t in range(T):
            if paths[t] is None:
                continue
            pos = p + L + len(paths[t]) - 1
            first = pos - window + 1 if window else 0
            seen = [at for x, at in rows if x >= first]
            mine = [n for n in paths[t] if p + L + len(paths[n]) - 1 >= first]
            kn = [rope(k_new[b, n], p + L + len(paths[n]) - 1, theta) for n in mine]
            for g in range(Hkv):
                k = np.concatenate([kc[max(first, 0):, g]] + [k_pages[x][None, g] for x in seen] +
                                   [x[None, g] for x in kn])
                v = np.concatenate([vc[max(first, 0):, g]] + [v_pages[x][None, g] for x in seen] +
                                   [v_new[b, n][None, g] for n in mine])
                for h in range(g * G, (g + 1) * G):
                    x = rope(q[b, t, h], pos, theta)
                    s = scale * (k @ x)
                    w = np.exp(s - s.max())
                    w /= w.sum()
                    o[b, t, h] = w @ v
                    e = scale * (np.abs(k) @ np.abs(x)) * (2 * HALF_BF16 + 1e-5)
                    rel = np.expm1(2 * e.max()) + HALF_BF16 + 1e-5
                    bound[b, t, h] = (w @ np.abs(v)) * rel * (1 + HALF_BF16) + \
                        HALF_BF16 * np.abs(o[b, t, h])
    return o, bound, wrote


def fork(table, lens, refs, src, dst, rows, P):
    table, lens, refs = table.copy(), lens.copy(), refs.copy()
    B, M = table.shape
    old_table, old_lens, done = table.copy(), lens.copy(), np.zeros(len(src), np.int32)
    for f, (a, z) in enumerate(zip(src, dst)):
        others = [x for i, x in enumerate(dst) if i != f]
        if not (0 <= a < B and 0 <= z < B) or z in others or z in src:
            continue
        n = old_lens[a] if rows is None else min(rows[f], old_lens[a])
        n = max(0, min(n, M * P))
        new = [old_table[a, k] if k * P < n else -1 for k in range(M)]
        for x, by in [(x, -1) for x in table[z]] + [(x, 1) for x in new]:
            if 0 <= x < len(refs):
                refs[x] += by
        table[z], lens[z], done[f] = new, n, 1
    return table, lens, refs, done


def reserve(table, lens, refs, rows, P):
    """... and the copies [(from page, to page, rows)]."""
    table, lens, refs = table.copy(), lens.copy(), refs.copy()
    B, M = table.shape
    N = len(refs)
    asks = [0 <= n <= M * P for n in rows]
    for b in range(B):
        if asks[b]:
            for k in range(-(-int(rows[b]) // P), M):
                if 0 <= table[b, k] < N:
                    refs[table[b, k]] -= 1
                table[b, k] = -1
            lens[b] = min(max(lens[b], 0), rows[b])
    free = [i for i in range(N) if refs[i] <= 0]
    shared = refs > 1
    room, at, copies, done = len(free), 0, [], np.zeros(B, np.int32)
    for b in range(B):
        if not asks[b]:
            continue
        need = [k for k in range(lens[b] // P, -(-int(rows[b]) // P))
                if not 0 <= table[b, k] < N or shared[table[b, k]]]
        room -= len(need)
        if need and room < 0:
            continue
        done[b] = 1
        for k in need:
            old, new = table[b, k], free[at]
            at += 1
            if 0 <= old < N:
                refs[old] -= 1
                if k == lens[b] // P and lens[b] % P:
                    copies.append((old, new, lens[b] % P))
            table[b, k], refs[new] = new, 1
    return table, lens, refs, done, copies


def accept(table, lens, parents, node, N, P, nodes):
    """(new lens, moves [((page, row) from, (page, row) to)])"""
    out, moves = lens.copy(), []
    for b in range(len(lens)):
        paths = used_nodes(None if parents is None else parents[b], int(lens[b]), table[b], N, P,
                           nodes)
        n = int(node[b])
        path = paths[n] if 0 <= n < nodes else None
        if path is None:
            continue
        L = min(int(lens[b]), table.shape[1] * P)
        out[b] = L + len(path)
        moves += [(page_at(table[b], L + t, N, P), page_at(table[b], L + i, N, P))
                  for i, t in enumerate(path) if t != i]
    return out, moves


def compact(table, refs):
    """(table, refs, moved, live, copies)"""
    N = len(refs)
    pages = [i for i in range(N) if refs[i] > 0]
    n = len(pages)
    moved = np.array([i if refs[i] > 0 else -1 for i in range(N)], np.int32)
    new = np.where(refs > 0, refs, 0).astype(np.int32)
    copies = list(zip([i for i in pages if i >= n], [i for i in range(n) if refs[i] <= 0]))
    for a, z in copies:
        moved[a], new[z], new[a] = z, refs[a], 0
    out = np.array([[moved[x] if 0 <= x < N else -1 for x in row] for row in table], np.int32)
    return out, new, moved, n, copies
