"""GPU parity of the operators that hold a paged cache to a budget of rows
(append, weights of keys, evict, the single-token step) with plain 64-bit
forms."""
import numpy as np
import pytest
import torch

from tests import budget_reference as bref
from tests import paged_reference as ref
from trained_kv_prefix_gb300 import cartattn as ca
from trained_kv_prefix_gb300 import synth

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(np.ascontiguousarray(x), dtype=torch.int32, device="cuda")


def _f32(x):
    return torch.tensor(np.ascontiguousarray(x), dtype=torch.float32, device="cuda")


def _bf16(rng, shape, std=0.5):
    return torch.from_numpy(rng.standard_normal(shape) * std).to(torch.bfloat16)


def _tables(rng, lens, more, P, spare=3, extra=1):
    lens = np.asarray(lens, np.int32)
    M = max(1, -(-(int(lens.max(initial=0)) + more) // P)) + extra
    need = [-(-(int(n) + more) // P) if n >= 0 else 0 for n in lens]
    N = sum(need) + spare
    ids, table, at = rng.permutation(N), np.full((len(lens), M), -1, np.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, N


def f64(x):
    return synth.f64(x)


# --------------------------------------------------------------- append ----
APPENDS = [
    # id, B, n, Hkv, d, p, lens, P, positions, packed
    ("one_token", 2, 1, 2, 64, 5, (0, 16), 16, False, False),
    ("odd", 3, 7, 3, 64, 0, (15, 1, 40), 16, False, False),
    ("d128", 2, 33, 8, 128, 300, (0, 63), 64, False, False),
    ("idle", 3, 5, 1, 128, 9, (-1, 3, 127), 128, False, False),
    ("positions", 3, 6, 2, 64, 9, (0, 3, 20), 32, True, False),
    ("packed", 4, 9, 2, 128, 17, (0, 31, 5, 2), 32, False, True),
    ("packed_positions", 3, 40, 1, 64, 17, (0, 31, 5), 16, True, True),
]


@pytest.mark.parametrize("case", APPENDS, ids=[c[0] for c in APPENDS])
def test_append_parity(case):
    _, B, n, Hkv, d, p, lens, P, positions, packed = case
    rng = np.random.default_rng(n)
    table, N = _tables(rng, lens, n, P)
    pos = rng.integers(0, 100000, size=B) if positions else None
    cu = None
    if packed:                              # runs of 0 to n tokens
        runs = rng.integers(0, n + 1, size=B)
        runs[0], runs[-1] = n, 0
        cu = np.concatenate([[0], np.cumsum(runs)])
    shape = (int(cu[-1]), Hkv, d) if packed else (B, n, Hkv, d)
    k, v = _bf16(rng, shape), _bf16(rng, shape)
    kp, vp = _bf16(rng, (N, P, Hkv, d)), _bf16(rng, (N, P, Hkv, d))
    gk, gv = kp.cuda(), vp.cuda()
    got = ca.cart_pages_append(k.cuda(), v.cuda(), gk, gv, _i32(table), _i32(lens), p=p,
                               pos=None if pos is None else _i32(pos),
                               cu_seqlens=None if cu is None else _i32(cu))
    assert got[0] is gk and got[1] is gv and ca.device_status() == 0
    wrote, lost = bref.append(f64(k), f64(v), table, np.array(lens), pos, p, N, P, cu)
    assert not lost
    kr, vr = f64(kp), f64(vp)
    off = np.zeros(kr.shape)
    for at, (a, b, raw) in wrote.items():
        kr[at], vr[at] = a, b
        # one rounding to bf16, and angles good to 1e-6
        off[at] = ref.HALF_BF16 * np.abs(a) + 2e-6 * np.abs(raw).max()
    np.testing.assert_array_equal(f64(gv), vr)
    assert (np.abs(f64(gk) - kr) <= off).all()


def test_append_drops_what_has_no_place():
    """Rows without a page and tokens in no run are dropped and reported; the
    others arrive."""
    rng = np.random.default_rng(1)
    table, lens, P, N = np.array([[3, -1], [1, 9]], np.int32), [14, 0], 16, 4
    k = _bf16(rng, (2, 6, 1, 64))
    pools = [torch.zeros(N, P, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ca.cart_pages_append(k.cuda(), k.cuda(), *pools, _i32(table), _i32(lens), p=2)
    assert ca.device_status() == 1 << 7
    np.testing.assert_array_equal(f64(pools[1])[3, 14:], f64(k)[0, :2])
    np.testing.assert_array_equal(f64(pools[1])[1, :6], f64(k)[1])
    assert (f64(pools[1])[[0, 2]] == 0).all() and (f64(pools[1])[3, :14] == 0).all()
    flat, cu = k.view(12, 1, 64).cuda(), _i32([3, 5, 4])     # neither from 0 nor rising to 12
    pools = [torch.zeros(N, P, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ca.cart_pages_append(flat, flat, *pools, _i32(table), _i32(lens), p=2, cu_seqlens=cu)
    assert ca.device_status() == 1 << 6
    np.testing.assert_array_equal(f64(pools[1])[3, 14:], f64(flat)[3:5])
    assert (f64(pools[1])[[0, 1, 2]] == 0).all()


# -------------------------------------------------------------- weights ----
def make_weigh(seed, B, T, Hq, Hkv, d, p, lens, P, positions=False, hole=False):
    rng = np.random.default_rng(seed)
    table, N = _tables(rng, lens, 0, P)
    if hole:
        table[-1, 0] = N + 7
    t = dict(q=_bf16(rng, (B, T, Hq, d), 1.5), kc=_bf16(rng, (p, Hkv, d), 1.0),
             k_pages=_bf16(rng, (N, P, Hkv, d), 1.0))
    lse = (rng.standard_normal((B, Hq, T)) + 3).astype(np.float32)
    pos = rng.integers(0, 90000, size=B) if positions else None
    return t, lse, table, np.asarray(lens, np.int32), pos


def check_weigh(t, lse, table, lens, pos, window=0, sinks=0, accumulate=False, W=0, **kw):
    P, Hkv, p, B = t["k_pages"].shape[1], t["kc"].shape[1], t["kc"].shape[0], len(lens)
    rng = np.random.default_rng(9)
    W = W or table.shape[1] * P
    old = rng.random((B, Hkv, W)).astype(np.float32)
    cart = rng.random((B, Hkv, p)).astype(np.float32)
    T = t["q"].shape[1]
    gw, gc = ca.cart_attn_weights(t["q"].cuda(), _f32(lse), t["kc"].cuda(), t["k_pages"].cuda(),
                                  _i32(table), _i32(lens), _f32(old), _f32(cart),
                                  pos=None if pos is None else _i32(pos), window=window, sinks=sinks,
                                  accumulate=accumulate, **kw)
    assert ca.device_status() == 0
    a = {k: f64(v) for k, v in t.items()}
    kept = {k: kw[k] for k in ("scale", "theta") if k in kw}
    w, bound, held = bref.weigh(a["q"], lse.astype(np.float64), a["kc"], a["k_pages"], table, lens, pos,
                                window, sinks, **kept)
    gw, gc = f64(gw), f64(gc)
    base = cart if accumulate else 0
    # (an addition rounds once more)
    off = bound[..., :p] + 2.0 ** -24 * np.abs(base + w[..., :p])
    assert (np.abs(gc - base - w[..., :p]) <= off).all()
    for b in range(B):
        n = int(held[b])
        was = np.where(np.arange(n) < n - T, old[b, :, :n], 0) if accumulate else 0
        want = was + w[b, :, p:p + n]
        assert (np.abs(gw[b, :, :n] - want) <=
                bound[b, :, p:p + n] + 2.0 ** -24 * np.abs(want)).all(), b
        np.testing.assert_array_equal(gw[b, :, n:], old[b, :, n:])
    return gw, gc


WEIGHS = [
    # id, B, T, Hq, Hkv, d, p, lens, P, window, sinks, accumulate, positions
    ("one_query", 3, 1, 4, 2, 64, 20, (1, 16, 33), 16, 0, 0, False, False),
    ("one_query_g1_d128", 2, 1, 2, 2, 128, 130, (5, 200), 64, 0, 0, True, False),
    ("few", 3, 9, 8, 2, 128, 70, (9, 130, 64), 32, 0, 0, False, False),
    ("more_queries_than_rows", 3, 40, 4, 1, 64, 33, (3, 0, 41), 16, 0, 0, True, False),
    ("idle", 2, 5, 4, 2, 64, 5, (-1, 6), 16, 0, 0, False, False),
    ("no_cartridge", 2, 6, 4, 4, 64, 0, (130, 7), 16, 0, 0, False, False),
    ("g7", 2, 20, 14, 2, 128, 129, (100, 20), 64, 0, 0, False, False),
    ("g8", 2, 37, 8, 1, 64, 128, (128, 129), 128, 0, 0, True, True),
    ("g5_many", 1, 100, 5, 1, 64, 257, (260,), 64, 0, 0, False, True),
    ("window", 2, 30, 4, 2, 64, 200, (190, 40), 32, 77, 0, False, False),
    ("window_sinks", 2, 30, 6, 2, 128, 300, (190, 40), 32, 90, 131, True, False),
    ("window_one", 2, 4, 4, 2, 64, 9, (19, 4), 16, 1, 0, False, False),
    ("sinks_in_rows", 2, 8, 4, 2, 64, 9, (150, 300), 16, 20, 40, False, False),
    ("long", 1, 3, 2, 1, 64, 700, (2500,), 128, 0, 0, False, False),
]


@pytest.mark.parametrize("case", WEIGHS, ids=[c[0] for c in WEIGHS])
def test_weights_parity(case):
    _, B, T, Hq, Hkv, d, p, lens, P, window, sinks, accumulate, positions = case
    check_weigh(*make_weigh(T + B, B, T, Hq, Hkv, d, p, lens, P, positions), window=window,
                sinks=sinks, accumulate=accumulate)


def test_weights_rows_that_are_not_there():
    s = make_weigh(3, 2, 5, 4, 2, 64, 12, (40, 50), 16, hole=True)
    gw, _ = check_weigh(*s)
    assert (gw[1, :, :16] == 0).all()
    check_weigh(*s, accumulate=True, W=100)
    check_weigh(*make_weigh(3, 2, 5, 4, 2, 64, 12, (40, 50), 16), scale=0.3, theta=1e4)


def test_weights_keep_what_is_not_seen_apart():
    """NaN and infinities in queries that are not there, in keys behind a
    window, in rows behind the end and in unused pages reach nothing."""
    t, lse, table, lens, _ = make_weigh(5, 2, 12, 4, 2, 64, 30, (70, 5), 16)
    want = ca.cart_attn_weights(t["q"].cuda(), _f32(lse), t["kc"].cuda(), t["k_pages"].cuda(),
                                _i32(table), _i32(lens), torch.zeros(2, 2, 96, device="cuda"),
                                window=20)
    k, q, kc = t["k_pages"].clone(), t["q"].clone(), t["kc"].clone()
    used = {int(x) for x in table[table >= 0]}
    for page in set(range(k.shape[0])) - used:
        k[page] = float("nan")
    q[1, :7], lse = float("inf"), lse.copy()
    lse[1, :, :7] = np.nan
    k[table[0, 4], 6:] = float("nan")                # behind row 69
    k[table[0, 2], :7] = float("inf")                # below place 70 - 12 - 19 + 30
    kc[:5] = float("nan")                            # below place 30 + 5 - 12 + 7 - 19
    got = ca.cart_attn_weights(q.cuda(), _f32(lse), kc.cuda(), k.cuda(), _i32(table), _i32(lens),
                               torch.zeros(2, 2, 96, device="cuda"), window=20)
    for a, b in zip(got, want):
        np.testing.assert_array_equal(f64(a), f64(b))


# ---------------------------------------------------------------- evict ----
def make_evict(seed, B, layers, Hkv, d, P, lens, share=1, dtype=torch.bfloat16, spare=40, ties=False):
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, np.int32)
    M = max(1, -(-int(lens.max()) // P)) + 1
    n = -(-np.maximum(lens, 0) // P)
    first = np.arange(B) // share * share
    N = int(n.sum()) + spare
    ids, table, at = rng.permutation(N), np.full((B, M), -1, np.int32), 0
    for b in range(B):
        c = 0 if b == first[b] else min(n[b], n[first[b]])
        table[b, :c] = table[first[b], :c]
        table[b, c:n[b]] = ids[at:at + n[b] - c]
        at += n[b] - c
    refs = np.bincount(table[table >= 0], minlength=N).astype(np.int32)
    W = M * P + 5
    w = rng.random((layers, B, Hkv, W)).astype(np.float32) ** 6
    if ties:
        w = np.round(w * 3) / 3
    pools = [torch.from_numpy(rng.standard_normal((layers, N, P, Hkv, d))).to(dtype) for _ in range(2)]
    return pools, table, lens, refs, w


def check_evict(pools, table, lens, refs, w, keep, first=0, recent=0, **kw):
    g = [x.cuda() for x in pools]
    gt, gl, gr, gw = _i32(table), _i32(lens), _i32(refs), None if w is None else _f32(w)
    layers, _, P, Hkv, _ = pools[0].shape
    done = ca.cart_pages_evict(*g, gt, gl, gr, gw, _i32(keep), first=first, recent=recent, **kw)
    assert ca.device_status() == 0
    t, n, r, dn, w2, moves, stay = bref.evict(table, lens, refs, w, keep, first, recent, layers, Hkv, P)
    np.testing.assert_array_equal(done.cpu().numpy(), dn)
    np.testing.assert_array_equal(gt.cpu().numpy(), t)
    np.testing.assert_array_equal(gl.cpu().numpy(), n)
    np.testing.assert_array_equal(gr.cpu().numpy(), r)
    if w is not None:
        np.testing.assert_array_equal(gw.cpu().numpy(), w2)
    for x, y in zip(pools, g):
        want = x.clone()
        for layer, h, a, z in moves:
            want[(layer,) + z + (h,)] = x[(layer,) + a + (h,)]
        assert torch.equal(want.view(torch.uint8), y.cpu().view(torch.uint8))
    return done, stay


EVICTS = [
    # id, B, layers, Hkv, d, P, lens, keep, first, recent, share, ties
    ("one_row_out", 1, 1, 1, 64, 16, (17,), (16,), 0, 0, 1, False),
    ("to_one", 2, 2, 2, 64, 16, (17, 1), (1, 1), 0, 0, 1, False),
    ("to_none", 2, 1, 2, 64, 16, (17, 40), (0, 0), 3, 5, 1, False),
    ("some_left", 5, 2, 2, 64, 32, (100, 7, 64, -1, 65), (50, 50, -1, 3, 64), 4, 20, 1, False),
    ("ties", 3, 2, 4, 64, 16, (100, 90, 33), (40, 41, 30), 2, 7, 1, True),
    ("first_alone", 2, 1, 2, 64, 16, (60, 70), (20, 33), 100, 0, 1, False),
    ("recent_alone", 2, 1, 2, 64, 16, (60, 70), (20, 33), 0, 100, 1, False),
    ("both_more_than_keep", 2, 1, 2, 64, 16, (60, 70), (20, 33), 15, 18, 1, False),
    ("shared", 6, 2, 2, 128, 16, (100, 90, 120, 33, 50, 60), (40, 41, 50, 20, 50, 7), 20, 7, 3, False),
    ("shared_first_pages_stay", 4, 1, 2, 64, 16, (100, 100, 90, 20), (40,) * 4, 32, 0, 2, False),
    ("shared_nothing_changes", 2, 1, 1, 64, 16, (40, 40), (20, 20), 20, 0, 2, False),
    ("long", 2, 1, 2, 128, 128, (6000, 4500), (3000, 4499), 5, 1000, 1, False),
    ("long_ties", 1, 1, 2, 64, 64, (5000,), (700,), 0, 0, 1, True),
    ("d96", 2, 1, 2, 96, 16, (50, 70), (33, 41), 1, 1, 1, False),
]


@pytest.mark.parametrize("case", EVICTS, ids=[c[0] for c in EVICTS])
def test_evict_parity(case):
    _, B, layers, Hkv, d, P, lens, keep, first, recent, share, ties = case
    s = make_evict(B + layers, B, layers, Hkv, d, P, lens, share, ties=ties)
    check_evict(*s, keep, first, recent)


def test_evict_other_types_and_no_weights():
    check_evict(*make_evict(1, 3, 2, 2, 64, 16, (70, 50, 33), dtype=torch.float32), (30, 20, 33), 2, 9)
    pools, table, lens, refs, _ = make_evict(2, 3, 2, 2, 64, 16, (70, 50, 33), share=2)
    check_evict(pools, table, lens, refs, None, (30, 20, 40), 4, 1)
    # one layer's pool with one layer's weights
    pools, table, lens, refs, w = make_evict(3, 2, 1, 2, 64, 16, (70, 50))
    g = [x[0].cuda() for x in pools]
    gw = _f32(w[0])
    done = ca.cart_pages_evict(*g, _i32(table), _i32(lens), _i32(refs), gw, _i32((20, 20)))
    w2 = bref.evict(table, lens, refs, w, (20, 20), 0, 0, 1, 2, 16)[4]
    assert done.tolist() == [1, 1]
    np.testing.assert_array_equal(gw.cpu().numpy(), w2[0])


def test_evict_weights_of_any_kind():
    """Negative ones, infinities, both zeros (equal) and NaN (most of all)."""
    s = make_evict(5, 2, 2, 2, 64, 16, (90, 60))
    w = s[4]
    rng = np.random.default_rng(0)
    kinds = np.array([0.0, -0.0, -1.5, np.inf, -np.inf, np.nan, 1e-42, 3.0], np.float32)
    w[:] = rng.choice(kinds, size=w.shape)
    check_evict(*s, (41, 22), 3, 4)
    w[:] = np.nan
    check_evict(*s, (41, 22), 3, 4)


def test_evict_without_pages():
    """Too few free pages: the conversation and all later ones that need any are
    left as they are; a page that is not there leaves its conversation too."""
    pools, table, lens, refs, w = make_evict(7, 6, 1, 2, 64, 16, (90, 90, 80, 80, 70, 70), share=2,
                                             spare=0)
    N = len(refs)
    free = [i for i in range(N) if refs[i] == 0]
    refs[free] = 1                          # somebody else's, all but four
    refs[free[-4:]] = 0
    done, _ = check_evict(pools, table, lens, refs, w, (40, 40, 40, -1, 17, 70), 0, 5)
    assert done.tolist() == [1, 0, 0, 1, 0, 1]
    table[0, 3] = -1
    table[3, 1] = N + 4
    done, _ = check_evict(pools, table, lens, refs, w, (40, 40, 40, 0, 17, 70), 0, 5)
    assert done.tolist() == [0, 1, 0, 0, 0, 1]
    table[5, 4:] = table[0, 0]              # pages behind the rows are not looked at
    check_evict(pools, table, lens, refs, w, (40, 40, 40, 0, 17, 60), 0, 5)


# --------------------------------------------------------------- decode ----
def make_step(seed, B, Hq, Hkv, d, p, lens, P, positions=False, std=1.0):
    rng = np.random.default_rng(seed)
    table, N = _tables(rng, lens, 1, P)
    t = dict(q=_bf16(rng, (B, Hq, d), 1.5 * std), k_new=_bf16(rng, (B, Hkv, d), std),
             v_new=_bf16(rng, (B, Hkv, d)), kc=_bf16(rng, (p, Hkv, d), std), vc=_bf16(rng, (p, Hkv, d)),
             k_pages=_bf16(rng, (N, P, Hkv, d), std), v_pages=_bf16(rng, (N, P, Hkv, d)))
    pos = rng.integers(0, 90000, size=B) if positions else None
    return t, table, np.asarray(lens, np.int32), pos


def run_step(t, table, lens, pos=None, weights=None, **kw):
    g = {k: v.cuda() for k, v in t.items()}
    o = ca.cart_attn_decode_paged(g["q"], g["k_new"], g["v_new"], g["kc"], g["vc"], g["k_pages"],
                                  g["v_pages"], _i32(table), _i32(lens),
                                  pos=None if pos is None else _i32(pos), weights=weights, **kw)
    torch.cuda.synchronize()
    return o, g


def check_step(t, table, lens, pos=None, window=0, sinks=0, weights=True, status=0, **kw):
    B, Hkv, P = len(lens), t["k_new"].shape[1], t["k_pages"].shape[1]
    rows = table.shape[1] * P
    old = np.random.default_rng(4).random((B, Hkv, rows + 3)).astype(np.float32)
    gw = _f32(old) if weights else None
    o, g = run_step(t, table, lens, pos, gw, window=window, sinks=sinks, **kw)
    assert ca.device_status() == status
    a = {k: f64(v) for k, v in t.items()}
    kept = {k: kw[k] for k in ("scale", "theta") if k in kw}
    want, ob, w, wb, wrote, lost = bref.decode(**a, table=table, lens=lens, pos=pos, window=window,
                                               sinks=sinks, **kept)
    off = np.abs(f64(o) - want)
    assert np.isfinite(off).all() and (off <= ob).all(), float((off - ob).max())
    k, v, kb = a["k_pages"].copy(), a["v_pages"].copy(), np.zeros(a["k_pages"].shape)
    for at, (kr, vr) in wrote.items():
        k[at], v[at] = kr, vr
        kb[at] = ref.HALF_BF16 * np.abs(kr) + 2e-6 * np.abs(a["k_new"]).max()
    np.testing.assert_array_equal(f64(g["v_pages"]), v)
    assert (np.abs(f64(g["k_pages"]) - k) <= kb).all()
    if weights:
        got = f64(gw)
        for b in range(B):
            n = min(int(lens[b]), rows)
            if n < 0 or ref.page_at(table[b], n, t["k_pages"].shape[0], P) is None:
                np.testing.assert_array_equal(got[b], old[b])
                continue
            x = w[b].copy()
            x[:, :n] += old[b, :, :n]
            assert (np.abs(got[b, :, :n + 1] - x[:, :n + 1]) <=
                    wb[b, :, :n + 1] + 2.0 ** -24 * np.abs(x[:, :n + 1])).all(), b
            np.testing.assert_array_equal(got[b, :, n + 1:], old[b, :, n + 1:])
    return o


STEPS = [
    # id, B, Hq, Hkv, d, p, lens, P, window, sinks, positions
    ("first_token", 1, 4, 2, 64, 0, (0,), 16, 0, 0, False),
    ("small", 3, 8, 2, 128, 70, (0, 1, 200), 64, 0, 0, False),
    ("d64", 4, 4, 2, 64, 16, (0, 15, 16, 17), 16, 0, 0, True),
    ("no_cartridge", 3, 4, 4, 128, 0, (0, 127, 129), 32, 0, 0, True),
    ("idle", 4, 8, 2, 64, 20, (-1, 5, -3, 0), 16, 0, 0, False),
    ("g1", 2, 3, 3, 64, 130, (33, 128), 16, 0, 0, False),
    ("g3", 2, 6, 2, 128, 128, (255, 256), 64, 0, 0, False),
    ("g5_h9", 2, 45, 9, 64, 40, (255, 17), 64, 0, 0, True),
    ("g7", 3, 28, 4, 128, 300, (120, 310, 0), 32, 0, 0, False),
    ("g8_one_head", 2, 8, 1, 64, 257, (190, 63), 16, 0, 0, False),
    ("h16", 2, 16, 16, 64, 100, (500, 3), 32, 0, 0, False),
    ("h11", 2, 22, 11, 128, 33, (200, 99), 128, 0, 0, False),
    ("many", 40, 4, 2, 64, 140, tuple(range(0, 200, 5)), 16, 0, 0, False),
    ("window_in_rows", 3, 8, 2, 128, 300, (0, 255, 599), 64, 100, 0, False),
    ("window_in_cartridge", 4, 4, 2, 64, 400, (0, 17, 200, 300), 32, 350, 0, True),
    ("window_one_key", 2, 4, 4, 64, 64, (69, 3), 16, 1, 0, False),
    ("sinks", 3, 8, 2, 128, 300, (0, 255, 599), 64, 100, 7, False),
    ("sinks_all_cartridge", 3, 4, 2, 64, 300, (0, 255, 599), 64, 100, 300, True),
    ("sinks_in_rows", 3, 4, 2, 64, 30, (0, 255, 599), 64, 50, 75, False),
    ("sinks_meet_window", 2, 4, 2, 64, 200, (50, 20), 16, 60, 180, False),
    ("long_rows", 2, 4, 1, 64, 30, (5003, 2048), 128, 0, 0, False),
    ("long_cartridge", 1, 4, 2, 64, 4500, (40,), 64, 0, 0, False),
    ("long_d128", 1, 32, 8, 128, 513, (3001,), 64, 0, 0, True),
    # more tiles and rows than CTAs: several a CTA, in pieces of several segments
    ("runs_of_tiles", 3, 8, 8, 64, 2700, (40, 7, 0), 16, 0, 0, False),
    ("runs_across", 3, 8, 8, 128, 2700, (40, 7, 0), 16, 0, 0, False),
    ("runs_of_both", 34, 32, 8, 128, 1500, tuple(range(0, 680, 20)), 64, 0, 0, False),
    ("runs_wide", 20, 35, 5, 64, 2900, tuple(range(9, 609, 30)), 32, 0, 0, True),
    ("runs_window", 20, 32, 8, 64, 1500, tuple(range(0, 2000, 100)), 32, 700, 70, False),
]


@pytest.mark.parametrize("case", STEPS, ids=[c[0] for c in STEPS])
def test_step_parity(case):
    _, B, Hq, Hkv, d, p, lens, P, window, sinks, positions = case
    s = make_step(B + d, B, Hq, Hkv, d, p, lens, P, positions)
    check_step(*s, window=window, sinks=sinks)
    check_step(*s, window=window, sinks=sinks, weights=False)


def test_step_with_one_key_far_ahead():
    """Logits of hundreds: one key takes all, the others' weights leave f32."""
    check_step(*make_step(3, 3, 8, 2, 128, 90, (0, 77, 200), 16, std=9.0), scale=0.5, theta=1e4)


def test_step_is_the_tree_of_one_node():
    t, table, lens, _ = make_step(6, 5, 8, 2, 128, 130, (0, 64, 63, 200, -1), 64)
    for window in (0, 90):
        o, g = run_step(t, table, lens, window=window)
        h = {k: v.cuda() for k, v in t.items()}
        o2 = ca.cart_attn_decode_tree(h["q"][:, None].contiguous(), h["k_new"][:, None].contiguous(),
                                      h["v_new"][:, None].contiguous(), h["kc"], h["vc"],
                                      h["k_pages"], h["v_pages"], _i32(table), _i32(lens),
                                      window=window)
        # both within two roundings to bf16 and the weights' of the values' size
        assert np.abs(f64(o) - f64(o2)[:, 0]).max() <= 6 * ref.HALF_BF16 * np.abs(f64(o)).max()
        assert torch.equal(g["v_pages"], h["v_pages"]) and (o[4] == 0).all()


def test_step_without_a_page():
    """Bad tables, lengths beyond them, rows that are not there."""
    t, table, lens, _ = make_step(7, 4, 4, 2, 64, 20, (20, 16, 40, 33), 16)
    table[0, 0], table[1, 1], table[3, 0] = 1000, -5, -1      # 1: the new row's page
    lens[2] = 10000
    check_step(t, table, lens, status=1 << 7)
    o, _ = run_step(t, table, lens)
    assert (o[1] == 0).all() and (o[2] == 0).all() and ca.device_status() == 1 << 7


def test_step_keeps_what_is_not_seen_apart():
    t, table, lens, _ = make_step(9, 3, 8, 2, 128, 200, (70, 5, 300), 16)
    W = table.shape[1] * 16
    w0, w1 = (torch.zeros(3, 2, W, device="cuda") for _ in range(2))
    want, _ = run_step(t, table, lens, weights=w0, window=50, sinks=3)
    k, v = t["k_pages"].clone(), t["v_pages"].clone()
    for page in set(range(k.shape[0])) - {int(x) for x in table[table >= 0]}:
        k[page], v[page] = float("nan"), float("inf")
    for b, n in enumerate((70, 5, 300)):
        k[table[b, n // 16], n % 16:], v[table[b, n // 16], n % 16:] = float("nan"), float("nan")
    for r in range(300 - 49):
        k[table[2, r // 16], r % 16], v[table[2, r // 16], r % 16] = float("inf"), float("nan")
    kc, vc = t["kc"].clone(), t["vc"].clone()
    kc[3:150], vc[3:150] = float("nan"), float("-inf")        # places 3 .. 149 < 200 + 5 - 49
    got, _ = run_step(dict(t, k_pages=k, v_pages=v, kc=kc, vc=vc), table, lens, weights=w1, window=50,
                      sinks=3)
    assert torch.equal(want, got) and torch.equal(w0, w1)


def test_step_passes_on_what_is_not_finite():
    """A value that is not finite reaches the queries that see it, as in IEEE
    sums, and a NaN key its conversation's weights; others stay as they are."""
    t, table, lens, _ = make_step(10, 3, 4, 2, 64, 30, (40, 33, 20), 16)
    w0, w1 = (torch.zeros(3, 2, table.shape[1] * 16, device="cuda") for _ in range(2))
    want, _ = run_step(t, table, lens, weights=w0)
    v, k = t["v_pages"].clone(), t["k_pages"].clone()
    v[table[0, 1], 3, 0, 5] = float("inf")
    k[table[1, 0], 2, 1] = float("nan")
    got, _ = run_step(dict(t, v_pages=v, k_pages=k), table, lens, weights=w1)
    g, w = f64(got), f64(want)
    assert np.isinf(g[0, :2, 5]).all()
    np.testing.assert_array_equal(np.delete(g[0, :2], 5, 1), np.delete(w[0, :2], 5, 1))
    np.testing.assert_array_equal(g[0, 2:], w[0, 2:])
    assert np.isnan(g[1, 2:]).all() and torch.equal(got[1, :2], want[1, :2])
    assert torch.equal(got[2], want[2]) and torch.equal(w1[0], w0[0]) and torch.equal(w1[2], w0[2])
    assert torch.isnan(w1[1, 1, :34]).all() and torch.equal(w1[1, 0], w0[1, 0])


def test_step_rows_of_minus_infinity():
    """Every logit -inf: o = 0 and no weight is given."""
    t, table, lens, _ = make_step(11, 2, 4, 2, 64, 3, (2, 0), 16)
    for x in ("q", "k_new", "kc", "k_pages"):
        t[x] = torch.zeros_like(t[x])
    # position 0 turns nothing; the products of element 0 are below f32's range
    t["q"][:, :, 0] = 1e30
    for x in ("kc", "k_pages", "k_new"):
        t[x][..., 0] = -3.0e38
    w = torch.ones(2, 2, table.shape[1] * 16, device="cuda")
    o, _ = run_step(t, table, lens, pos=np.zeros(2), weights=w)
    assert (o == 0).all()
    assert (w[0, :, :2] == 1).all() and (w[0, :, 2] == 0).all() and (w[1, :, 0] == 0).all()


# ------------------------------------------------------------- together ----
def test_a_prompt_held_to_a_budget():
    """Prompts through the training forward, their rows appended, weighed by the
    last queries, evicted, and decoded on, twice, with room reserved between;
    each call against the plain form on the state it met."""
    rng = np.random.default_rng(12)
    layers, B, n, Hq, Hkv, d, p, P, M = 2, 3, 96, 8, 2, 64, 40, 16, 12
    T, budget = 24, 50
    N = B * M + 4
    kp, vp = (torch.zeros(layers, N, P, Hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.full((B, M), -1, dtype=torch.int32, device="cuda")
    lens, refs = _i32([0] * B), _i32([0] * N)
    weights = torch.zeros(layers, B, Hkv, M * P, device="cuda")
    kc, vc = (_bf16(rng, (layers, p, Hkv, d)).cuda() for _ in range(2))
    assert ca.cart_pages_reserve(kp, vp, table, lens, refs, _i32([n] * B)).tolist() == [1] * B
    for i in range(layers):
        q, k, v = _bf16(rng, (B, n, Hq, d), 1.5), _bf16(rng, (B, n, Hkv, d)), _bf16(rng, (B, n, Hkv, d))
        _, lse = ca.cart_attn_fwd(q.cuda(), k.cuda(), v.cuda(), kc[i], vc[i])
        ca.cart_pages_append(k.cuda(), v.cuda(), kp[i], vp[i], table, lens, p=p)
        held = lens + n
        qo, lo = q[:, -T:].contiguous(), lse[:, :, -T:].contiguous()
        ca.cart_attn_weights(qo.cuda(), lo, kc[i], kp[i], table, held, weights[i])
        w, bound, _ = bref.weigh(f64(qo), f64(lo), f64(kc[i]), f64(kp[i]), table.cpu().numpy(),
                                 held.cpu().numpy())
        assert (np.abs(f64(weights[i])[..., :n] - w[..., p:p + n]) <= bound[..., p:p + n] + 1e-7).all()
    lens, pos = lens + n, _i32([p + n] * B)
    for step in range(2):
        before = [x.cpu() for x in (kp, vp)]
        t0, l0, r0, w0 = (x.cpu().numpy() for x in (table, lens, refs, weights))
        done = ca.cart_pages_evict(kp, vp, table, lens, refs, weights, _i32([budget] * B), first=2,
                                   recent=10)
        t, ln, r, dn, w, moves, _ = bref.evict(t0, l0, r0, w0, [budget] * B, 2, 10, layers, Hkv, P)
        assert done.tolist() == [1] * B and lens.tolist() == [budget] * B
        np.testing.assert_array_equal(table.cpu().numpy(), t)
        np.testing.assert_array_equal(refs.cpu().numpy(), r)
        np.testing.assert_array_equal(weights.cpu().numpy(), w)
        for x, y in zip(before, (kp, vp)):
            want = x.clone()
            for layer, h, a, z in moves:
                want[(layer,) + z + (h,)] = x[(layer,) + a + (h,)]
            assert torch.equal(want, y.cpu())
        ask = torch.where(done == 1, lens + 3, -1)
        assert ca.cart_pages_reserve(kp, vp, table, lens, refs, ask.int()).tolist() == [1] * B
        for token in range(3):
            for i in range(layers):
                q, k, v = _bf16(rng, (B, Hq, d), 1.5), _bf16(rng, (B, Hkv, d)), _bf16(rng, (B, Hkv, d))
                kb, vb, wb = kp[i].clone(), vp[i].clone(), f64(weights[i])
                o = ca.cart_attn_decode_paged(q.cuda(), k.cuda(), v.cuda(), kc[i], vc[i], kp[i], vp[i],
                                              table, lens, pos=pos, weights=weights[i])
                want, ob, w, wbd, wrote, lost = bref.decode(
                    f64(q), f64(k), f64(v), f64(kc[i]), f64(vc[i]), f64(kb), f64(vb),
                    table.cpu().numpy(), lens.cpu().numpy(), pos.cpu().numpy())
                assert not lost and (np.abs(f64(o) - want) <= ob).all()
                m = int(lens[0])
                wb[..., m:] = 0
                got = f64(weights[i])[..., :m + 1]
                assert (np.abs(got - (wb + w)[..., :m + 1]) <=
                        wbd[..., :m + 1] + 2.0 ** -24 * np.abs(got)).all()
                assert torch.equal(kp[i][int(table[0, 0])], kb[int(table[0, 0])])
            lens, pos = lens + 1, pos + 1
    assert ca.device_status() == 0
