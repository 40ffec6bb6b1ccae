"""Edges of the paged operators on the GPU, against the plain 64-bit forms."""
import numpy as np
import pytest
import torch

from tests import paged_reference as ref
from tests.test_paged_gpu import _bf16, _i32, _pool, check_tree, make_tables, make_tree, run_tree
from trained_kv_prefix_gb300 import cartattn as ca
from trained_kv_prefix_gb300 import synth

pytestmark = pytest.mark.gpu

BAD = (float("inf"), -float("inf"), float("nan"))

WINDOWS = [
    # id, B, nodes, Hq, Hkv, d, p, lens, P, kind, window
    ("chain", 1, 2, 4, 2, 64, 30, (77,), 16, "chain", 40),
    ("window_in_tree", 2, 8, 4, 2, 128, 30, (77, 3), 16, "chain", 5),
    ("across_tiles", 2, 40, 2, 2, 64, 50, (240, 390), 32, "chain", 128),
    ("two_query_tiles", 2, 64, 8, 1, 128, 64, (190, 400), 64, "random", 100),
    ("most_nodes", 1, 64, 2, 2, 64, 0, (500,), 16, "chain", 400),
    ("from_the_cartridge", 3, 30, 4, 2, 64, 64, (60, 20, 75), 16, "chain", 70),
    ("stacked", 6, 9, 8, 2, 128, 1200, (100, 300, 129, 250, 64, 31), 16, "chain", 60),
    ("cut_among_ctas", 1, 12, 8, 2, 128, 30, (9003,), 128, "chain", 8800),
    ("tree", 2, 33, 4, 1, 64, 40, (100, 300), 32, "wide", 90),
]


@pytest.mark.parametrize("case", WINDOWS, ids=[c[0] for c in WINDOWS])
@pytest.mark.parametrize("with_key", [False, True])
def test_values_that_a_deeper_node_has_left_behind(case, with_key):
    """Cached rows in the window of the shallowest node and out of a deeper
    one's that are not finite: they reach the nodes that see them, in the
    elements that are not finite, and no other."""
    _, B, nodes, Hq, Hkv, d, p, lens, P, kind, window = case
    t, table, lens, parents = make_tree(81, B, nodes, Hq, Hkv, d, p, lens, P, kind)
    t["v_pages"], t["k_pages"] = t["v_pages"].clone(), t["k_pages"].clone()
    n = 0
    for b in range(B):
        for r in range(max(lens[b] - window, 0), min(lens[b] - window + nodes + 2, lens[b])):
            page, row = table[b, r // P], r % P
            t["v_pages"][page, row, r % Hkv, 5 * r % d] = BAD[r % 3]
            n += 1
        if with_key:
            r = lens[b] - window + 1
            if 0 <= r < lens[b]:
                t["k_pages"][table[b, r // P], r % P, 0, 3] = float("nan")
    assert n > 1
    o, g = run_tree(t, table, lens, parents, window=window)
    assert ca.device_status(clear=True) == 0
    a = {k: synth.f64(v) for k, v in t.items()}
    with np.errstate(invalid="ignore"):
        o_ref, bound, _ = ref.tree(**a, table=table, lens=lens, parents=parents, window=window)
    got, finite = synth.f64(o), np.isfinite(o_ref)
    assert finite.any() and not finite.all()
    np.testing.assert_array_equal(got[~finite], o_ref[~finite])
    assert (np.abs(got[finite] - o_ref[finite]) <= bound[finite]).all()
    # the cached rows stay as they are
    for b in range(B):
        for r in range(lens[b]):
            at = table[b, r // P], r % P
            np.testing.assert_array_equal(synth.f64(g["v_pages"][at]), a["v_pages"][at])


def test_window_of_single_tokens_equals_their_chain():
    """A chain with a window is the single-token steps in order, whatever the
    rows that each step has left behind hold."""
    window, nodes = 40, 6
    t, table, lens, parents = make_tree(82, 2, nodes, 4, 2, 64, 30, (77, 160), 16, "chain")
    t["v_pages"] = t["v_pages"].clone()
    for b in range(2):
        for i in range(nodes):
            r = lens[b] - window + 1 + i
            t["v_pages"][table[b, r // 16], r % 16, 0, i] = BAD[i % 3]
    o, _ = run_tree(t, table, lens, parents, window=window)
    a = {k: synth.f64(v) for k, v in t.items()}
    with np.errstate(invalid="ignore"):
        _, bound, _ = ref.tree(**a, table=table, lens=lens, parents=parents, window=window)
    g = {k: v.cuda() for k, v in t.items()}
    tb = torch.tensor(table, dtype=torch.int32, device="cuda")
    for i in range(nodes):
        ln = torch.tensor(lens + i, dtype=torch.int32, device="cuda")
        one = ca.cart_attn_decode_tree(*(g[k][:, i:i + 1].contiguous() for k in
                                         ("q", "k_new", "v_new")), g["kc"], g["vc"], g["k_pages"],
                                       g["v_pages"], tb, ln, window=window)
        x, y = synth.f64(one[:, 0]), synth.f64(o[:, i])
        same = np.isfinite(x)
        np.testing.assert_array_equal(np.isfinite(y), same)
        np.testing.assert_array_equal(x[~same], y[~same])
        # each within its bound of one value
        assert (np.abs(x[same] - y[same]) <= 2 * bound[:, i][same]).all()
    assert ca.device_status(clear=True) == 0


@pytest.mark.parametrize("window", [1, 5, 39, 40, 90])
def test_windows_of_idle_empty_and_full_conversations(window):
    t, table, lens, parents = make_tree(83, 4, 40, 4, 2, 64, 30, (50, 0, 8, 60), 16, "random")
    lens[0] = -1
    check_tree(t, table, lens, parents, window=window)
    lens[3] = table.shape[1] * 16           # no node of it fits
    check_tree(t, table, lens, parents, window=window, status=128)


@pytest.mark.parametrize("B,nodes,p,lens", [(1, 3, 900, (40,)), (1, 2, 0, (5,)), (3, 5, 30, (0, 9, 200)),
                                            (6, 4, 1100, (0, 9, 200, 40, 3, 1)),
                                            (2, 40, 300, (4000, 17))])
def test_logits_of_minus_infinity(B, nodes, p, lens):
    """Rows whose every logit is -inf are 0, whether one CTA walked their keys
    or several did.  One dimension of the slowest angle holds the queries and,
    negated, the keys: 2^100 * -2^100 is -inf in f32, and so is the product of
    what the rotation moves to the dimension's other half."""
    d = 64
    t, table, lens, parents = make_tree(84, B, nodes, 4, 2, d, p, lens, 16, "random")
    for name in ("q", "k_new", "kc", "k_pages"):
        x = torch.zeros_like(t[name])
        x[..., d // 2 - 1] = 2.0 ** 100 if name == "q" else -2.0 ** 100
        t[name] = x
    o, _ = run_tree(t, table, lens, parents)
    assert ca.device_status(clear=True) == 0
    assert not torch.isnan(o).any() and not o.any()


NOTHING_TO_APPEND = [
    # id, table, lens, refs, rows -> table, lens, refs, done, copies (from, to, rows); 16 rows a page
    # two that share their part page ask for what they hold: each gets its own
    ("free", [[0, -1], [0, -1]], [5, 5], [2, 0, 0], [5, 5],
     [[1, -1], [2, -1]], [5, 5], [0, 1, 1], [1, 1], [(0, 1, 5), (0, 2, 5)]),
    # without a free page they keep it, and have their rows
    ("full", [[0, -1], [0, 1]], [5, 20], [2, 1], [5, 20],
     [[0, -1], [0, 1]], [5, 20], [2, 1], [1, 1], []),
    # a rewind into the part page that both share; nothing is given back
    ("rewind_full", [[0, -1], [0, -1], [1, -1]], [9, 9, 16], [2, 1], [3, -1, 16],
     [[0, -1], [0, -1], [1, -1]], [3, 9, 16], [2, 1], [1, 0, 1], []),
    # a rewind that gives back a page of its own takes that one
    ("rewind", [[0, 1], [0, -1]], [20, 9], [2, 1], [3, -1],
     [[1, -1], [0, -1]], [3, 9], [1, 1], [1, 0], [(0, 1, 3)]),
    # rows that end with a page need no other
    ("whole_pages", [[0, 1], [0, 1]], [32, 20], [2, 2], [32, 16],
     [[0, 1], [0, -1]], [32, 16], [2, 1], [1, 1], []),
    # one that has nothing to append does not keep back the answer of one that has
    ("both", [[0, -1], [0, -1], [1, -1]], [5, 5, 16], [2, 1], [5, 6, 17],
     [[0, -1], [0, -1], [1, -1]], [5, 5, 16], [2, 1], [1, 0, 0], []),
]


@pytest.mark.parametrize("case", NOTHING_TO_APPEND, ids=[c[0] for c in NOTHING_TO_APPEND])
def test_reserve_with_nothing_to_append(case):
    _, table, lens, refs, rows, wt, wl, wr, wd, copies = case
    k, v = (_pool((2, len(refs), 16, 1, 64), torch.bfloat16, s) for s in (1, 2))
    tb, ln, rf = _i32(table), _i32(lens), _i32(refs)
    before = k.clone(), v.clone()
    done = ca.cart_pages_reserve(k, v, tb, ln, rf, _i32(rows))
    assert done.tolist() == wd and ln.tolist() == wl
    assert tb.tolist() == wt and rf.tolist() == wr
    for now, old in zip((k, v), before):
        want = old.clone()
        for a, z, n in copies:
            want[:, z, :n] = old[:, a, :n]
        assert torch.equal(now, want)


def test_a_step_sat_out():
    """A conversation without room is idle for a step, keeps its rows, and goes
    on once there is room."""
    rng = np.random.default_rng(85)
    t, _, _, _ = make_tree(85, 3, 2, 2, 1, 64, 4, (0, 0, 0), 16, "chain")
    k, v = (_bf16(rng, (1, 3, 16, 1, 64)).cuda() for _ in range(2))
    table, lens, refs = _i32([[0, -1], [0, -1], [1, -1]]), _i32([5, 5, 16]), _i32([2, 1, 0])
    parents = _i32([[-1, 0]] * 3)
    g = {n: x.cuda() for n, x in t.items()}

    def step(rows):
        nonlocal lens
        done = ca.cart_pages_reserve(k, v, table, lens, refs, rows)
        now = torch.where((done == 1) & (rows > lens), lens, -1)
        before = k.clone(), v.clone()
        o = ca.cart_attn_decode_tree(g["q"], g["k_new"], g["v_new"], g["kc"], g["vc"], k[0], v[0],
                                     table, now, parents)
        a = {n: synth.f64(x) for n, x in t.items() if n not in ("k_pages", "v_pages")}
        o_ref, bound, wrote = ref.tree(**a, k_pages=synth.f64(before[0][0]),
                                       v_pages=synth.f64(before[1][0]),
                                       table=table.cpu().numpy(), lens=now.cpu().numpy(),
                                       parents=parents.cpu().numpy())
        assert (np.abs(synth.f64(o) - o_ref) <= bound).all()
        left = torch.ones(3, 16, dtype=torch.bool)
        for page, row in wrote:
            left[page, row] = False
        assert torch.equal(k[0].cpu()[left], before[0][0].cpu()[left])
        new = ca.cart_pages_accept(k, v, table, now, parents, _i32([1, 1, 1]))
        lens = torch.where(now < 0, lens, new)
        return done.tolist()

    assert step(lens + 2) == [1, 0, 0] and lens.tolist() == [7, 5, 16]
    assert table.tolist() == [[2, -1], [0, -1], [1, -1]] and refs.tolist() == [1, 1, 1]
    # the second's page is its own now; the first leaves, and the third takes its page
    assert step(_i32([0, 7, 18])) == [1, 1, 1] and lens.tolist() == [0, 7, 18]
    assert table.tolist() == [[-1, -1], [0, -1], [1, 2]]
    assert ca.device_status(clear=True) == 0


def test_reserve_takes_a_missing_page_as_it_is():
    """The page of row lens is missing: a free one is taken, nothing is copied,
    and its rows below lens are seen again, with what the page holds."""
    k, v = (_pool((1, 3, 16, 1, 64), torch.bfloat16, s) for s in (1, 2))
    before = k.clone(), v.clone()
    tb, ln, rf = _i32([[0, -1]]), _i32([21]), _i32([1, 0, 0])
    done = ca.cart_pages_reserve(k, v, tb, ln, rf, _i32([22]))
    assert done.tolist() == [1] and tb.tolist() == [[0, 1]] and rf.tolist() == [1, 1, 0]
    assert torch.equal(k, before[0]) and torch.equal(v, before[1])


def test_largest_tables_and_lists():
    """65535 conversations: 8192 forks at once, then room for all of them."""
    B, M, P, F, N = 65535, 2, 16, 8192, 90000
    rng = np.random.default_rng(86)
    table, lens, refs = make_tables(rng, B, M, P, N, share=0.6)
    src, dst = np.split(rng.permutation(B)[:2 * F].astype(np.int32), 2)
    src[5], dst[9], dst[11] = -1, B, dst[12]
    bad = {5, 9, 11, 12}
    tb, ln, rf = _i32(table), _i32(lens), _i32(refs)
    done = ca.cart_pages_fork(tb, ln, rf, _i32(src), _i32(dst), page_rows=P)
    good = np.array([f not in bad for f in range(F)])
    np.testing.assert_array_equal(done.cpu().numpy(), good.astype(np.int32))
    # no destination is a source: all rows move at once
    a, z = src[good], dst[good]
    n = np.maximum(lens[a], 0)
    new = np.where(np.arange(M) * P < n[:, None], table[a], -1)
    for pages, by in ((table[z], -1), (new, 1)):
        np.add.at(refs, pages[pages >= 0], by)
    table[z], lens[z] = new, n
    for got, w in ((tb, table), (ln, lens), (rf, refs)):
        np.testing.assert_array_equal(got.cpu().numpy(), w)
    rows = np.where(lens < 0, -1, np.minimum(lens + 3, M * P)).astype(np.int32)
    k, v = (_pool((1, N, P, 1, 8), torch.bfloat16, s) for s in (1, 2))
    k0 = k.clone()
    done = ca.cart_pages_reserve(k, v, tb, ln, rf, _i32(rows))
    wt, wl, wr, wd, copies = ref.reserve(table, lens, refs, rows, P)
    wd = np.where((rows >= 0) & (rows == lens), 1, wd)      # nothing to append
    assert 0 < wd.sum() < B and len(copies) > 1000
    for got, w in zip((tb, ln, rf, done), (wt, wl, wr, wd)):
        np.testing.assert_array_equal(got.cpu().numpy(), w)
    want = k0.clone()
    fr, to, n = (torch.tensor(x, device="cuda") for x in np.array(copies).T)
    part = (torch.arange(P, device="cuda") < n[:, None])[None, :, :, None, None]
    want[:, to] = torch.where(part, k0[:, fr], k0[:, to])
    assert torch.equal(k, want)
