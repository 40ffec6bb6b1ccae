"""GPU parity of the paged serving operators (tree attention over paged
private rows, fork, reserve, accept, compact) with plain 64-bit forms."""
import numpy as np
import pytest
import torch

from tests import paged_reference as ref
from trained_kv_prefix_gb300 import cartattn as ca
from trained_kv_prefix_gb300 import synth

pytestmark = pytest.mark.gpu


def _gpu(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)) if isinstance(x, np.ndarray) else x
    return (t if dtype is None else t.to(dtype)).cuda()


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _bf16(rng, shape, std=0.5):
    return torch.from_numpy(rng.standard_normal(shape) * std).to(torch.bfloat16)


def random_tree(rng, nodes, kind):
    t = np.arange(nodes)
    if kind == "chain":
        return t - 1
    if kind == "star":                      # every node follows the cached rows
        return np.full(nodes, -1)
    if kind == "wide":                      # four children each
        return (t - 1) // 4
    up = np.floor(rng.random(nodes) * t).astype(int)
    up[0] = -1
    if kind == "ragged":                    # unused tail, an unused node inside, bad parents
        up[max(1, nodes - nodes // 3):] = -2
        if nodes > 4:
            up[2], up[3], up[4] = 3, -7, 1000
    return up


def make_tree(seed, B, nodes, Hq, Hkv, d, p, lens, P, kind="random", spare_pages=3, hole=False):
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, np.int32)
    assert lens.shape == (B,)
    M = max(1, -(-(int(lens.max(initial=0)) + nodes) // P)) + 1
    need = [-(-(max(int(n), 0) + nodes) // P) for n in lens]
    N = sum(need) + spare_pages
    ids, table, at = rng.permutation(N), np.full((B, M), -1, np.int32), 0
    for b in range(B):
        table[b, :need[b]] = ids[at:at + need[b]]
        at += need[b]
    if hole:                                # a page that is not there, inside
        table[B - 1, 0] = -1
        table[0, min(1, M - 1)] = N + 5
    parents = np.stack([random_tree(rng, nodes, kind) for _ in range(B)]).astype(np.int32)
    t = dict(q=_bf16(rng, (B, nodes, Hq, d)), k_new=_bf16(rng, (B, nodes, Hkv, d)),
             v_new=_bf16(rng, (B, nodes, Hkv, d)), kc=_bf16(rng, (p, Hkv, d)),
             vc=_bf16(rng, (p, Hkv, d)), k_pages=_bf16(rng, (N, P, Hkv, d)),
             v_pages=_bf16(rng, (N, P, Hkv, d)))
    return t, table, lens, parents


def run_tree(t, table, lens, parents, window=0, **kw):
    g = {k: v.cuda() for k, v in t.items()}
    o = ca.cart_attn_decode_tree(g["q"], g["k_new"], g["v_new"], g["kc"], g["vc"], g["k_pages"],
                                 g["v_pages"], _i32(table), _i32(lens),
                                 None if parents is None else _i32(parents), window=window, **kw)
    torch.cuda.synchronize()
    return o, g


def check_tree(t, table, lens, parents, window=0, status=0, **kw):
    o, g = run_tree(t, table, lens, parents, window, **kw)
    assert ca.device_status(clear=True) == status
    a = {k: synth.f64(v) for k, v in t.items()}
    o_ref, bound, wrote = ref.tree(**a, table=table, lens=lens, parents=parents, window=window)
    off = np.abs(synth.f64(o) - o_ref)
    assert np.isfinite(off).all()
    assert (off <= bound).all(), float((off - bound).max())
    assert (synth.f64(o)[bound == 0] == 0).all()
    # the rows written, and no other
    k, v = a["k_pages"].copy(), a["v_pages"].copy()
    kb = np.zeros(k.shape)
    for at, (kr, vr) in wrote.items():
        k[at], v[at] = kr, vr
        # one rounding to bf16, and angles good to 1e-6
        kb[at] = ref.HALF_BF16 * np.abs(kr) + 2e-6 * np.abs(a["k_new"]).max()
    np.testing.assert_array_equal(synth.f64(g["v_pages"]), v)
    assert (np.abs(synth.f64(g["k_pages"]) - k) <= kb).all()
    return o


TREES = [
    # id, B, nodes, Hq, Hkv, d, p, lens, P, kind, window
    ("one_token", 3, 1, 8, 2, 128, 70, (0, 1, 200), 64, "chain", 0),
    ("one_token_d64", 4, 1, 4, 2, 64, 16, (0, 15, 16, 17), 16, "chain", 0),
    ("no_cartridge", 3, 5, 4, 4, 128, 0, (0, 127, 129), 32, "random", 0),
    ("no_rows_at_all", 2, 7, 4, 4, 64, 0, (0, 0), 16, "random", 0),
    ("one_row_cartridge", 2, 3, 8, 1, 128, 1, (0, 5), 128, "random", 0),
    ("g1", 2, 9, 3, 3, 64, 130, (33, 128), 16, "random", 0),
    ("g2", 2, 16, 4, 2, 128, 128, (255, 256), 64, "wide", 0),
    ("g8_many_rows", 2, 20, 16, 2, 64, 200, (120, 310), 32, "random", 0),
    ("g8_full", 1, 64, 8, 1, 128, 257, (190,), 16, "random", 0),
    ("g4_full", 3, 64, 8, 2, 64, 300, (0, 63, 400), 64, "wide", 0),
    ("g4_48", 2, 48, 4, 1, 128, 129, (128, 77), 128, "random", 0),
    ("deep_chain", 2, 64, 2, 2, 64, 40, (100, 3), 16, "chain", 0),
    ("star", 2, 33, 4, 1, 64, 40, (100, 31), 32, "star", 0),
    ("ragged", 5, 13, 8, 2, 128, 66, (0, 3, 129, 250, 64), 16, "ragged", 0),
    ("many_small", 19, 3, 4, 2, 64, 140, tuple(range(0, 190, 10)), 16, "random", 0),
    ("window_in_rows", 3, 6, 8, 2, 128, 300, (0, 255, 599), 64, "random", 100),
    ("window_in_cartridge", 4, 9, 4, 2, 64, 400, (0, 17, 200, 300), 32, "random", 350),
    ("window_one_key", 2, 8, 4, 4, 64, 64, (69, 3), 16, "chain", 1),
    ("window_in_tree", 2, 40, 4, 1, 64, 20, (130, 0), 16, "chain", 7),
    ("window_wide_rows", 2, 64, 8, 1, 64, 500, (130, 700), 16, "random", 333),
    ("long_rows", 2, 6, 4, 1, 64, 30, (5003, 2048), 128, "random", 0),
    ("long_cartridge", 1, 4, 4, 2, 64, 4500, (40,), 64, "random", 0),
    # cartridges long enough that the rows of all conversations walk them together
    ("stacked_tokens", 5, 1, 8, 2, 128, 700, (0, 1, 200, 64, 333), 64, "chain", 0),
    ("stacked_g1", 7, 9, 2, 2, 64, 640, (0, 15, 16, 17, 300, 1, 128), 16, "random", 0),
    ("stacked_g2", 4, 16, 4, 2, 128, 1100, (255, 256, 0, 31), 64, "wide", 0),
    ("stacked_g8", 9, 20, 8, 1, 64, 2700, (0, 5, 128, 310, 64, 77, 1, 90, 12), 32, "random", 0),
    ("stacked_two_tiles", 8, 36, 4, 1, 64, 2500, (3, 0, 127, 130, 40, 9, 250, 64), 16, "wide", 0),
    ("stacked_ragged", 6, 13, 8, 2, 128, 1200, (0, 3, 129, 250, 64, 31), 16, "ragged", 0),
    ("stacked_many", 40, 3, 4, 2, 64, 520, tuple(range(0, 200, 5)), 16, "random", 0),
    ("stacked_window_in_rows", 5, 6, 8, 2, 64, 700, (0, 255, 599, 90, 101), 64, "random", 100),
    ("stacked_window_in_cartridge", 5, 9, 4, 2, 64, 900, (0, 17, 200, 300, 5), 32, "random", 350),
    ("stacked_window_wide", 8, 36, 4, 1, 64, 2500, (3, 0, 700, 130, 40, 9, 250, 64), 64, "random",
     333),
]


@pytest.mark.parametrize("case", TREES, ids=[c[0] for c in TREES])
def test_tree_parity(case):
    _, B, nodes, Hq, Hkv, d, p, lens, P, kind, window = case
    check_tree(*make_tree(B + nodes, B, nodes, Hq, Hkv, d, p, lens, P, kind), window=window)


def test_tree_chains_without_parents_equal_given_chains():
    t, table, lens, parents = make_tree(3, 3, 6, 8, 2, 128, 90, (0, 77, 200), 32, "chain")
    a = check_tree(t, table, lens, parents)
    b, _ = run_tree(t, table, lens, None)
    assert torch.equal(a, b)


@pytest.mark.parametrize("p", [200, 900])
@pytest.mark.parametrize("nodes,G", [(1, 4), (4, 4), (3, 2), (8, 1)])
def test_tree_chain_agrees_with_span_verify(nodes, G, p):
    """A chain over pages is the span verify over a dense cache."""
    rng = np.random.default_rng(5)
    B, Hkv, d, P, rows = 4, 2, 128, 32, 320
    lens = np.array([0, 31, 150, rows - nodes], np.int32)
    x = {k: _bf16(rng, s).cuda() for k, s in dict(
        q=(B, nodes, G * Hkv, d), k_new=(B, nodes, Hkv, d), v_new=(B, nodes, Hkv, d),
        kc=(p, Hkv, d), vc=(p, Hkv, d), k=(B, rows, Hkv, d), v=(B, rows, Hkv, d)).items()}
    table = np.arange(B * rows // P, dtype=np.int32).reshape(B, -1)
    kp, vp = (x[n].clone().view(B * rows // P, P, Hkv, d) for n in "kv")
    a = ca.cart_attn_decode_tree(x["q"], x["k_new"], x["v_new"], x["kc"], x["vc"], kp, vp,
                                 _i32(table), _i32(lens))
    b = ca.cart_attn_decode_span(x["q"], x["k_new"], x["v_new"], x["kc"], x["vc"], x["k"], x["v"],
                                 _i32(lens))
    torch.cuda.synchronize()
    # both are within 2^-8 (weights) + 2^-8 (output) of one value, relative to
    # sum w |v| <= max |v|; the queries are rotated alike up to angles of 1e-6
    vmax = float(torch.cat([x["v"].flatten(), x["vc"].flatten(), x["v_new"].flatten()]).abs().max())
    assert float((a.float() - b.float()).abs().max()) <= 4 * ref.HALF_BF16 * vmax
    # stored keys: one rounding each of values that differ by 1e-6
    assert torch.equal(vp.view_as(x["v"]), x["v"])
    assert float((kp.view_as(x["k"]).float() - x["k"].float()).abs().max()) <= \
        2 * ref.HALF_BF16 * 2 * float(x["k_new"].abs().max())


@pytest.mark.parametrize("p", [50, 900])
def test_tree_idle_and_pageless_conversations(p):
    """Idle slots, missing pages among the cached rows (not seen) and under
    new nodes (unused, reported)."""
    t, table, lens, parents = make_tree(11, 4, 7, 8, 2, 64, p, (40, 0, 33, 60), 16, "random",
                                        hole=True)
    lens = lens.copy()
    lens[1] = -1
    table[2, 2] = -1       # rows 32..47: the last cached row and all new nodes
    check_tree(t, table, lens, parents, status=128)


def test_tree_lens_beyond_the_table():
    """More rows than the table names count as its rows; no node fits."""
    t, table, lens, parents = make_tree(12, 2, 3, 4, 2, 64, 20, (30, 30), 16, "chain")
    lens = np.array([30, 1 << 30], np.int32)
    check_tree(t, table, lens, parents, status=128)


@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("nodes,Hq,Hkv,d,p", [(6, 4, 2, 64, 30), (64, 8, 1, 128, 30),
                                               (13, 8, 1, 128, 30), (6, 4, 2, 64, 900)])
def test_tree_masked_places_may_hold_anything(nodes, Hq, Hkv, d, p, window):
    """NaN and infinities in rows behind the sequence, in pages of nobody, in
    rows left behind by the window, and in other branches."""
    t, table, lens, parents = make_tree(21, 3, nodes, Hq, Hkv, d, p, (0, 77, 130), 16, "star")
    parents[1] = random_tree(np.random.default_rng(1), nodes, "ragged")
    clean = check_tree(t, table, lens, parents, window=window)
    bad = [float("nan"), float("inf"), -float("inf"), 3e38]
    for name in ("k_pages", "v_pages"):
        x = t[name] = t[name].clone()
        held = np.zeros(x.shape[:2], bool)
        for b in range(3):
            first = lens[b] - window + 1 if window else 0     # of the shallowest node
            for r in range(max(first, 0), lens[b]):
                held[table[b, r // 16], r % 16] = True
        spots = torch.from_numpy(np.argwhere(~held))
        x[spots[:, 0], spots[:, 1]] = torch.tensor(bad, dtype=torch.bfloat16).repeat(
            len(spots))[:len(spots), None, None]
    o, g = run_tree(t, table, lens, parents, window=window)
    assert torch.equal(o, clean)
    # one branch of conversation 2 goes wrong: the others do not notice
    for name in ("k_new", "v_new"):
        t[name] = t[name].clone()
        t[name][2, 3] = float("nan")
        t[name][2, 4, 0, :2] = float("inf")
        t[name][2, 5, :, 1] = -float("inf")
    o, g = run_tree(t, table, lens, parents, window=window)
    keep = [n for n in range(nodes) if n not in (3, 4, 5)]
    assert torch.equal(o[:2], clean[:2])
    assert torch.equal(o[2, keep], clean[2, keep])
    assert torch.isnan(o[2, 3]).all()
    ca.device_status(clear=True)


@pytest.mark.parametrize("B,p", [(1, 30), (4, 900)])
def test_tree_visible_infinities_reach_the_nodes_that_see_them(B, p):
    """A value of an ancestor that is infinite or NaN reaches its descendants
    in that element alone."""
    t, table, lens, parents = make_tree(22, B, 6, 2, 1, 64, p, (50,) * B, 16, "chain")
    parents[0] = [-1, 0, 1, -1, 3, 4]
    clean, _ = run_tree(t, table, lens, parents)
    t["v_new"] = t["v_new"].clone()
    t["v_new"][0, 1, 0, 5] = float("inf")
    t["v_new"][0, 4, 0, 7] = float("nan")
    o, _ = run_tree(t, table, lens, parents)
    want = clean.clone()
    want[0, [1, 2], :, 5] = float("inf")
    want[0, [4, 5], :, 7] = float("nan")
    torch.testing.assert_close(o, want, rtol=0, atol=0, equal_nan=True)


@pytest.mark.parametrize("fill", [0, 255, 127])
@pytest.mark.parametrize("B,nodes,p", [(3, 5, 200), (1, 5, 200), (2, 64, 200), (3, 5, 0), (3, 5, 900)])
def test_tree_workspace_needs_no_initial_value(B, nodes, p, fill):
    """Any bytes in the workspace, for stacked and fused segments; then every
    conversation idle over what that call left there, and over any bytes."""
    t, table, lens, parents = make_tree(25, B, nodes, 8, 2, 64, p, (300, 5, 90)[:B], 16, "random")
    want, _ = run_tree(t, table, lens, parents)
    n = ca.decode_tree_workspace_size(B, nodes, 8, 2, 64, p, 16, table.shape[1])
    ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
    o, _ = run_tree(t, table, lens, parents, workspace=ws)
    assert torch.equal(o, want)
    idle = np.full(B, -1, np.int32)
    for again in range(2):
        o, g = run_tree(t, table, idle, parents, workspace=ws)
        assert not o.any() and torch.equal(g["k_pages"].cpu(), t["k_pages"])
        ws.fill_(fill)
    assert ca.device_status(clear=True) == 0


@pytest.mark.parametrize("p,nodes", [(70, 1), (0, 2), (130, 3), (700, 2)])
def test_tree_many_conversations(p, nodes):
    """More conversations than the schedule's blocks have threads."""
    B = 530 if nodes == 1 else 300
    lens = np.random.default_rng(B).integers(-1, 60, B)
    check_tree(*make_tree(24 + nodes, B, nodes, 2, 1, 64, p, lens, 16, "random"))


@pytest.mark.parametrize("p", [150, 2900])
def test_tree_windows_that_cut_nothing(p):
    """Up to the largest window, bit for bit as without one."""
    t, table, lens, parents = make_tree(26, 3, 40, 8, 2, 64, p, (90, 0, 301), 16, "random")
    want, _ = run_tree(t, table, lens, parents)
    for window in (p + 600, 2 ** 24 - 1, 2 ** 24, 2 ** 31 - 1):
        o, _ = run_tree(t, table, lens, parents, window=window)
        assert torch.equal(o, want), window
    assert ca.device_status(clear=True) == 0


@pytest.mark.parametrize("p", [3, 600])
def test_tree_largest_batch(p):
    """The most conversations a call takes, a few of them checked."""
    B = 65535
    lens = np.random.default_rng(27).integers(-1, 15, B)
    t, table, lens, _ = make_tree(27, B, 1, 2, 1, 64, p, lens, 16, "chain")
    o, _ = run_tree(t, table, lens, None)
    assert ca.device_status(clear=True) == 0
    some = np.r_[0, 1, 255, 256, 257, 32767, 65533, 65534, np.arange(5, B, 997)]
    a = {k: synth.f64(v) for k, v in t.items() if k in ("kc", "vc")}
    pages = table[some][:, :1]
    a |= {k: synth.f64(t[k][some]) for k in ("q", "k_new", "v_new")}
    a |= {k: synth.f64(t[k][pages[:, 0]]) for k in ("k_pages", "v_pages")}
    own = np.arange(len(some), dtype=np.int32)[:, None]
    o_ref, bound, _ = ref.tree(**a, table=own, lens=lens[some], parents=None, window=0)
    assert (np.abs(synth.f64(o[torch.from_numpy(some).cuda()]) - o_ref) <= bound).all()


def test_tree_most_heads():
    check_tree(*make_tree(28, 1, 64, 1024, 128, 64, 130, (140,), 16, "wide"))


@pytest.mark.parametrize("p", [200, 900])
def test_tree_large_logits(p):
    """Logits of hundreds: the weights are all on a few keys."""
    t, table, lens, parents = make_tree(23, 2, 9, 4, 2, 64, p, (90, 300), 32, "random")
    t["q"] = (t["q"].float() * 64).to(torch.bfloat16)
    o, g = run_tree(t, table, lens, parents)
    assert torch.isfinite(o).all()
    vmax = max(float(t[n].float().abs().max()) for n in ("vc", "v_new", "v_pages"))
    assert float(o.float().abs().max()) <= vmax * (1 + 2 * ref.HALF_BF16)


def test_tree_pool_beyond_32_bits():
    """Pages whose byte offsets pass 2^32."""
    B, nodes, Hq, Hkv, d, P, p = 2, 5, 8, 8, 128, 128, 40
    N = 20000                               # 5.2 GB per pool
    rng = np.random.default_rng(31)
    lens = np.array([300, 90], np.int32)
    M = 4
    table = np.full((B, M), -1, np.int32)
    table[0, :3], table[1, :1] = [19999, 16385, 17000], [19321]
    kp = torch.zeros((N, P, Hkv, d), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    ids = [int(x) for x in table[table >= 0]]
    small = {k: _bf16(rng, (len(ids), P, Hkv, d)) for k in ("k", "v")}
    for i, page in enumerate(ids):
        kp[page], vp[page] = small["k"][i].cuda(), small["v"][i].cuda()
    t = dict(q=_bf16(rng, (B, nodes, Hq, d)), k_new=_bf16(rng, (B, nodes, Hkv, d)),
             v_new=_bf16(rng, (B, nodes, Hkv, d)), kc=_bf16(rng, (p, Hkv, d)),
             vc=_bf16(rng, (p, Hkv, d)))
    parents = np.tile(np.array([-1, 0, 0, 1, 2], np.int32), (B, 1))
    g = {k: v.cuda() for k, v in t.items()}
    o = ca.cart_attn_decode_tree(g["q"], g["k_new"], g["v_new"], g["kc"], g["vc"], kp, vp,
                                 _i32(table), _i32(lens), _i32(parents))
    torch.cuda.synchronize()
    local = np.full_like(table, -1)
    for i, page in enumerate(ids):
        local[table == page] = i
    a = {k: synth.f64(v) for k, v in t.items()}
    o_ref, bound, wrote = ref.tree(**a, k_pages=synth.f64(small["k"]), v_pages=synth.f64(small["v"]),
                                   table=local, lens=lens, parents=parents)
    assert (np.abs(synth.f64(o) - o_ref) <= bound).all()
    for (page, row), (_, v) in wrote.items():
        np.testing.assert_array_equal(synth.f64(vp[ids[page], row]), v)
    # reserve, accept and compact over the same pool
    refs = np.zeros(N, np.int32)
    for page in ids:
        refs[page] += 1
    pools = kp[None], vp[None]
    before = vp[19321, :90].clone()
    tb, ln, rf = _i32(table), _i32(lens), _i32(refs)
    new = ca.cart_pages_accept(*pools, tb, ln, _i32(parents), _i32([3, 4]))
    assert new.tolist() == [303, 93]
    moved, live = ca.cart_pages_compact(*pools, tb, rf)
    assert int(live) == len(ids) and int(tb.max()) == len(ids) - 1
    assert torch.equal(vp[tb[1, 0], :90], before)
    del kp, vp, pools
    torch.cuda.empty_cache()


@pytest.mark.parametrize("B,window", [(1, 0), (2, 0), (2, 9_000_001)])
def test_tree_longest_rows(B, window):
    """The most rows a conversation can have; its table names eight pages over
    and over, so the plain form weighs each key by how often it is there."""
    M, P, p, nodes, d, N = 131071, 128, 20, 3, 64, 10
    rng = np.random.default_rng(33)
    table = np.full((B, M), -1, np.int32)
    table[0] = np.arange(M) % 8
    table[0, -1] = 8
    lens = np.array([M * P - 5, 77][:B], np.int32)
    if B > 1:
        table[1, 0] = 9
    t = dict(q=_bf16(rng, (B, nodes, 4, d)), k_new=_bf16(rng, (B, nodes, 1, d)),
             v_new=_bf16(rng, (B, nodes, 1, d)), kc=_bf16(rng, (p, 1, d)),
             vc=_bf16(rng, (p, 1, d)), k_pages=_bf16(rng, (N, P, 1, d)),
             v_pages=_bf16(rng, (N, P, 1, d)))
    parents = np.tile(np.array([-1, 0, 0], np.int32), (B, 1))
    o, g = run_tree(t, table, lens, parents, window=window)
    assert ca.device_status(clear=True) == 0
    a = {k: synth.f64(v) for k, v in t.items()}
    L, G = int(lens[0]), 4
    first_new = [ref.rope(a["k_new"][0, n], p + L + (n > 0)) for n in range(nodes)]
    for n in range(nodes):
        pos = p + L + (n > 0)
        first = pos - window + 1 if window else 0
        r0 = max(first - p, 0)                      # the first row it sees
        times = np.zeros((9, P))
        pages, rows = np.unique(np.arange(r0 // P + 1, M - 1) % 8, return_counts=True)
        times[pages] += rows[:, None]
        times[(r0 // P) % 8, r0 % P:] += 1
        times[8, :P - 5] = 1
        seen = [0, n] if n else [0]
        k = np.concatenate([a["k_pages"][:9, :, 0].reshape(-1, d),
                            a["kc"][first:, 0] if first < p else np.zeros((0, d))] +
                           [first_new[x] for x in seen])
        v = np.concatenate([a["v_pages"][:9, :, 0].reshape(-1, d),
                            a["vc"][first:, 0] if first < p else np.zeros((0, d))] +
                           [a["v_new"][0, x] for x in seen])
        c = np.concatenate([times.ravel(), np.ones(len(k) - times.size)])
        for h in range(G):
            x = ref.rope(a["q"][0, n, h], pos)
            s = d ** -0.5 * (k @ x)
            w = c * np.exp(s - s.max())
            w /= w.sum()
            # as ref.tree: each of the rotated query and key, the weights and
            # the output rounded once; 2e-4 for f32 sums of 2^24 rows in 2^17
            # tiles (2^-24 of the sum at each of at most 2^9 steps of a run,
            # 2^7 terms each, and of the runs' merge)
            e = d ** -0.5 * (np.abs(k) @ np.abs(x)) * (2 * ref.HALF_BF16 + 1e-5)
            rel = np.expm1(2 * e.max()) + ref.HALF_BF16 + 2e-4
            bound = rel * (w @ np.abs(v)) + ref.HALF_BF16 * np.abs(w @ v) + 1e-6
            off = np.abs(synth.f64(o[0, n, h]) - w @ v)
            assert (off <= bound).all(), (n, h, float((off - bound).max()))
    if B > 1:                                       # its neighbour is not disturbed
        one = {k: v if k in ("kc", "vc", "k_pages", "v_pages") else v[1:] for k, v in t.items()}
        alone, _ = run_tree(one, table[1:], lens[1:], parents[1:], window=window)
        o_ref, bound, _ = ref.tree(**{k: synth.f64(v) for k, v in one.items()},
                                   table=table[1:, :2], lens=lens[1:], parents=parents[1:],
                                   window=window)
        assert (np.abs(synth.f64(o[1:]) - o_ref) <= bound).all()
        assert (np.abs(synth.f64(alone) - o_ref) <= bound).all()


# ------------------------------------------------------------ page operators
def make_tables(rng, B, M, P, N, share=0.4):
    """Random tables: conversations that hold rows of their own and of others,
    an idle one, one without pages."""
    table, refs = np.full((B, M), -1, np.int32), np.zeros(N, np.int32)
    lens, ids = np.zeros(B, np.int32), list(rng.permutation(N))
    for b in range(B):
        n = int(rng.integers(0, M + 1))
        for k in range(n):
            if b and rng.random() < share and table[b - 1, k] >= 0 and (k == 0 or
                                                                         table[b, k - 1] == table[b - 1, k - 1]):
                table[b, k] = table[b - 1, k]
            elif len(ids) > N // 4:
                table[b, k] = ids.pop()
            else:
                n = k
                break
            refs[table[b, k]] += 1
        lens[b] = rng.integers(0, n * P + 1)
    lens[0] = -1
    return table, lens, refs


FORKS = [(3, 2, 16, 2), (40, 9, 64, 25), (300, 70, 16, 120), (7, 1, 128, 3)]


@pytest.mark.parametrize("B,M,P,F", FORKS)
@pytest.mark.parametrize("with_rows", [True, False])
def test_fork(B, M, P, F, with_rows):
    rng = np.random.default_rng(B)
    table, lens, refs = make_tables(rng, B, M, P, B * M + 5)
    src, dst = rng.integers(-1, B + 1, F).astype(np.int32), rng.integers(-1, B + 1, F).astype(np.int32)
    dst[: F // 2] = rng.permutation(B)[: F // 2]
    rows = rng.integers(-2, M * P + 9, F).astype(np.int32) if with_rows else None
    want = ref.fork(table, lens, refs, src, dst, rows, P)
    tb, ln, rf = _i32(table), _i32(lens), _i32(refs)
    done = ca.cart_pages_fork(tb, ln, rf, _i32(src), _i32(dst),
                              None if rows is None else _i32(rows), page_rows=P)
    for got, w in zip((tb, ln, rf, done), want):
        np.testing.assert_array_equal(got.cpu().numpy(), w)


RESERVES = [
    # B, M, P, pages, layers, Hkv, d, dtype
    (2, 3, 16, 9, 1, 1, 64, torch.bfloat16),
    (23, 6, 16, 150, 3, 2, 64, torch.bfloat16),
    (23, 6, 16, 60, 2, 2, 64, torch.float32),       # the pool runs out
    (70, 5, 64, 400, 2, 8, 128, torch.bfloat16),
    (1500, 3, 16, 9000, 1, 1, 64, torch.bfloat16),  # more than one pass of the plan
    (5, 120, 32, 700, 1, 1, 64, torch.bfloat16),    # many pages each
    (9, 4, 128, 40, 1, 3, 8, torch.bfloat16),       # a row of 48 bytes
]


def _pool(shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("case", RESERVES, ids=[str(c[:4]) for c in RESERVES])
def test_reserve(case):
    B, M, P, N, layers, Hkv, d, dtype = case
    rng = np.random.default_rng(B + M)
    table, lens, refs = make_tables(rng, B, M, P, N)
    rows = np.where(rng.random(B) < 0.15, rng.integers(-1, 1, B),
                    np.maximum(lens, 0) + rng.integers(-P, 2 * P, B)).astype(np.int32)
    if B > 3:
        rows[1], rows[2] = M * P, M * P + 1
        lens[3], table[3, 0], rows[3] = 5, -1, 9        # a hole in the page to write
        refs = np.bincount(table[table >= 0], minlength=N).astype(np.int32)
    k, v = (_pool((layers, N, P, Hkv, d), dtype, s) for s in (1, 2))
    k0, v0 = k.clone(), v.clone()
    tb, ln, rf = _i32(table), _i32(lens), _i32(refs)
    done = ca.cart_pages_reserve(k, v, tb, ln, rf, _i32(rows))
    wt, wl, wr, wd, copies = ref.reserve(table, lens, refs, rows, P)
    for got, w in zip((tb, ln, rf, done), (wt, wl, wr, wd)):
        np.testing.assert_array_equal(got.cpu().numpy(), w)
    for got, old in ((k, k0), (v, v0)):
        want = old.clone()
        for a, z, n in copies:
            want[:, z, :n] = old[:, a, :n]
        assert torch.equal(got, want)


def test_reserve_frees_before_it_takes():
    """A full pool: what one conversation gives back another gets."""
    P, N = 16, 4
    table = _i32([[0, 1], [2, 3], [-1, -1]])
    lens, refs = _i32([20, 30, 0]), _i32([1, 1, 1, 1])
    k, v = _pool((1, N, P, 1, 64), torch.bfloat16, 1), _pool((1, N, P, 1, 64), torch.bfloat16, 2)
    done = ca.cart_pages_reserve(k, v, table, lens, refs, _i32([0, -1, 20]))
    assert done.tolist() == [1, 0, 1]
    assert table.tolist() == [[-1, -1], [2, 3], [0, 1]]
    assert lens.tolist() == [0, 30, 0] and refs.tolist() == [1, 1, 1, 1]


ACCEPTS = [
    # B, nodes, M, P, layers, Hkv, d, dtype, kind
    (1, 1, 2, 16, 1, 1, 64, torch.bfloat16, "chain"),
    (6, 9, 5, 16, 3, 2, 64, torch.bfloat16, "random"),
    (9, 64, 9, 16, 2, 8, 128, torch.bfloat16, "wide"),
    (5, 64, 3, 64, 1, 1, 64, torch.float32, "star"),
    (4, 33, 2, 128, 2, 3, 8, torch.bfloat16, "ragged"),
    (4, 64, 6, 16, 1, 5, 128, torch.float32, "deep"),
]


@pytest.mark.parametrize("case", ACCEPTS, ids=[str(c[:4]) for c in ACCEPTS])
def test_accept(case):
    B, nodes, M, P, layers, Hkv, d, dtype, kind = case
    rng = np.random.default_rng(nodes)
    N = B * M + 3
    table = rng.permutation(N)[:B * M].reshape(B, M).astype(np.int32)
    lens = rng.integers(0, M * P - nodes + 1, B).astype(np.int32)
    if kind == "deep":      # paths whose nodes lie where earlier nodes go to
        parents = np.tile(np.r_[-1, -1, np.arange(1, nodes - 1)], (B, 1)).astype(np.int32)
    else:
        parents = np.stack([random_tree(rng, nodes, kind) for _ in range(B)]).astype(np.int32)
    node = rng.integers(nodes // 2, nodes, B).astype(np.int32)
    if B > 3:
        node[0], lens[1], node[2] = -1, -1, nodes - 1
        table[3, -1] = -1
        node[B - 1] = nodes if kind == "wide" else node[B - 1]
    k, v = (_pool((layers, N, P, Hkv, d), dtype, s) for s in (1, 2))
    k0, v0 = k.clone(), v.clone()
    got = ca.cart_pages_accept(k, v, _i32(table), _i32(lens), _i32(parents), _i32(node))
    want, moves = ref.accept(table, lens, parents, node, N, P, nodes)
    np.testing.assert_array_equal(got.cpu().numpy(), want)
    for now, old in ((k, k0), (v, v0)):
        w = old.clone()
        for (a, x), (z, y) in moves:
            w[:, z, y] = old[:, a, x]
        assert torch.equal(now, w)


def test_accept_chains():
    """Chains need no moves: the accepted number is the last node's + 1."""
    k, v = _pool((2, 6, 16, 2, 64), torch.bfloat16, 1), _pool((2, 6, 16, 2, 64), torch.bfloat16, 2)
    k0 = k.clone()
    table = _i32([[0, 1, 2], [3, 4, 5]])
    new = ca.cart_pages_accept(k, v, table, _i32([7, 30]), 4, _i32([2, -1]))
    assert new.tolist() == [10, 30] and torch.equal(k, k0)


COMPACTS = [
    # B, M, P, pages, layers, Hkv, d, dtype, live share
    (1, 1, 16, 1, 1, 1, 64, torch.bfloat16, 1.0),
    (4, 3, 16, 9, 1, 1, 64, torch.bfloat16, 0.0),
    (6, 8, 16, 30, 2, 2, 64, torch.float32, 0.5),
    (6, 8, 16, 30, 2, 2, 64, torch.bfloat16, 1.0),
    (40, 12, 64, 300, 3, 8, 128, torch.bfloat16, 0.6),
    (300, 60, 16, 20011, 1, 1, 64, torch.bfloat16, 0.7),
    (5, 4, 32, 24, 1, 3, 8, torch.bfloat16, 0.3),
]


@pytest.mark.parametrize("case", COMPACTS, ids=[str(c[:4]) for c in COMPACTS])
def test_compact(case):
    B, M, P, N, layers, Hkv, d, dtype, share = case
    rng = np.random.default_rng(N)
    live = rng.permutation(N)[:int(N * share)]
    table = np.full((B, M), -1, np.int32)
    if len(live):
        pick = rng.choice(live, size=(B, M))
        table = np.where(rng.random((B, M)) < 0.7, pick, rng.integers(-3, 0, (B, M))).astype(np.int32)
        table[0, 0] = N + 3
    refs = np.bincount(table[(table >= 0) & (table < N)], minlength=N).astype(np.int32)
    refs[live[: len(live) // 9]] += 1           # a caller's own holds
    if N > 5:
        refs[rng.integers(0, N)] = -4           # free as well
    table0 = table.copy()
    k, v = (_pool((layers, N, P, Hkv, d), dtype, s) for s in (1, 2))
    k0, v0 = k.clone(), v.clone()
    tb, rf = _i32(table), _i32(refs)
    moved, n = ca.cart_pages_compact(k, v, tb, rf)
    wt, wr, wm, wn, copies = ref.compact(table0, refs)
    for got, w in zip((tb, rf, moved), (wt, wr, wm)):
        np.testing.assert_array_equal(got.cpu().numpy(), w)
    assert int(n) == wn
    for now, old in ((k, k0), (v, v0)):
        w = old.clone()
        for a, z in copies:
            w[:, z] = old[:, a]
        assert torch.equal(now, w)


# --------------------------------------------------------------- together --
class Server:
    """A few conversations served with the paged operators, and the same rows
    kept per conversation in plain lists."""

    def __init__(self, seed, B=6, layers=2, P=16, M=12, N=60, Hq=8, Hkv=2, d=64, p=40):
        rng = self.rng = np.random.default_rng(seed)
        self.B, self.layers, self.P, self.N, self.p = B, layers, P, N, p
        self.Hq, self.Hkv, self.d = Hq, Hkv, d
        self.k, self.v = (torch.full((layers, N, P, Hkv, d), float("nan"), dtype=torch.bfloat16,
                                     device="cuda") for _ in range(2))
        self.table, self.lens = _i32(np.full((B, M), -1)), _i32(np.full(B, -1))
        self.refs = _i32(np.zeros(N))
        self.kc, self.vc = (_bf16(rng, (layers, p, Hkv, d)).cuda() for _ in range(2))
        self.rows = {}                      # conversation -> per layer lists of (key, value) rows

    def reserve(self, room):
        rows = self.lens.clone().clamp(min=0) + room
        rows = torch.tensor([int(rows[b]) if b in self.rows else 0 for b in range(self.B)],
                            dtype=torch.int32, device="cuda")
        done = ca.cart_pages_reserve(self.k, self.v, self.table, self.lens, self.refs, rows)
        assert done.all()

    def step(self, parents, node):
        """One tree step in every layer; accepts the path to node[b]."""
        T = parents.shape[1]
        live = _i32([int(self.lens[b]) if b in self.rows else -1 for b in range(self.B)])
        for l in range(self.layers):
            x = {k: _bf16(self.rng, (self.B, T, h, self.d)) for k, h in
                 (("q", self.Hq), ("k_new", self.Hkv), ("v_new", self.Hkv))}
            o = ca.cart_attn_decode_tree(x["q"].cuda(), x["k_new"].cuda(), x["v_new"].cuda(),
                                         self.kc[l], self.vc[l], self.k[l], self.v[l], self.table,
                                         live, _i32(parents))
            self.check(l, x, o, parents, node)
        new = ca.cart_pages_accept(self.k, self.v, self.table, live, _i32(parents), _i32(node))
        for b in self.rows:
            self.lens[b] = new[b]

    def check(self, l, x, o, parents, node):
        """The layer's outputs against dense rows kept apart."""
        a = {k: synth.f64(v) for k, v in x.items()}
        for b, layers in self.rows.items():
            rows = layers[l]
            n, T = len(rows), parents.shape[1]
            kp, vp = np.zeros((1, n + T, self.Hkv, self.d)), np.zeros((1, n + T, self.Hkv, self.d))
            for i, (k, v) in enumerate(rows):
                kp[0, i], vp[0, i] = k, v
            o_ref, bound, wrote = ref.tree(
                a["q"][b:b + 1], a["k_new"][b:b + 1], a["v_new"][b:b + 1], synth.f64(self.kc[l]),
                synth.f64(self.vc[l]), kp, vp, np.zeros((1, 1), np.int32),
                np.array([n], np.int32), parents[b:b + 1])
            assert (np.abs(synth.f64(o[b:b + 1]) - o_ref) <= bound).all(), (b, l)
            t, path = int(node[b]), []
            while t >= 0:
                path.append(t)
                t = int(parents[b, t])
            for t in reversed(path):
                k, v = wrote[(0, n + t)]
                # the cache holds the rounded key
                rows.append((synth.f64(torch.from_numpy(k).to(torch.bfloat16)), v))


def test_served_together():
    """Admit, draft, accept, branch, rewind, retire and compact, over two
    layers, against rows kept densely per conversation."""
    s = Server(41)
    rng = np.random.default_rng(7)
    for b in (0, 2, 3):
        s.rows[b] = [[] for _ in range(s.layers)]

    def draft(T, kind="random"):
        parents = np.stack([random_tree(rng, T, kind) for _ in range(s.B)]).astype(np.int32)
        s.reserve(T)
        s.step(parents, rng.integers(-1, T, s.B).astype(np.int32))

    draft(20, "wide")
    draft(9)
    # conversation 0 branches into 1 and 5, at its end and at an earlier row
    n = int(s.lens[0])
    done = ca.cart_pages_fork(s.table, s.lens, s.refs, _i32([0, 0]), _i32([1, 5]),
                              _i32([n, max(n - 2, 0)]), page_rows=s.P)
    assert done.tolist() == [1, 1]
    s.rows[1] = [list(r) for r in s.rows[0]]
    s.rows[5] = [list(r)[:max(n - 2, 0)] for r in s.rows[0]]
    draft(17)
    # 2 retires; the pool is compacted; 3 is rewound into rows that 4 shares
    ca.cart_pages_fork(s.table, s.lens, s.refs, _i32([3]), _i32([4]), page_rows=s.P)
    s.rows[4] = [list(r) for r in s.rows[3]]
    del s.rows[2]
    back = max(0, int(s.lens[3]) - 3)
    s.lens[3] = back
    s.rows[3] = [r[:back] for r in s.rows[3]]
    draft(8)
    moved, live = ca.cart_pages_compact(s.k, s.v, s.table, s.refs)
    assert int((s.refs > 0).sum()) == int(live) and int(s.table.max()) < int(live)
    assert int(s.refs.sum()) == int((s.table >= 0).sum())
    draft(30, "wide")
    draft(1, "chain")
    assert ca.device_status(clear=True) == 0
    s.rows.clear()
    s.reserve(0)
    assert int(s.refs.abs().sum()) == 0 and int(s.table.max()) == -1


def test_no_room_sits_the_step_out():
    """A pool that runs out: the conversation without room takes no part, and
    the page that it shares stays as it is."""
    rng = np.random.default_rng(43)
    k = _bf16(rng, (1, 3, 16, 1, 64)).cuda()
    v = _bf16(rng, (1, 3, 16, 1, 64)).cuda()
    table, lens, refs = _i32([[0, -1], [0, -1], [1, -1]]), _i32([5, 5, 16]), _i32([2, 1, 0])
    k0, v0 = k.clone(), v.clone()
    done = ca.cart_pages_reserve(k, v, table, lens, refs, lens + 2)
    assert done.tolist() == [1, 0, 0]       # one free page: the first's copy
    assert table.tolist() == [[2, -1], [0, -1], [1, -1]] and refs.tolist() == [1, 1, 1]
    parents = torch.where(done[:, None] == 1, _i32([[-1, 0]] * 3), -2)
    q = _bf16(rng, (3, 2, 2, 64)).cuda()
    new = _bf16(rng, (3, 2, 1, 64)).cuda()
    c = _bf16(rng, (4, 1, 64)).cuda()
    o = ca.cart_attn_decode_tree(q, new, new, c, c, k[0], v[0], table, lens, parents)
    assert ca.device_status(clear=True) == 0
    assert o[0].any() and not o[1:].any()
    assert torch.equal(k[:, :2], k0[:, :2]) and torch.equal(v[:, :2], v0[:, :2])
    assert torch.equal(k[0, 2, :5], k0[0, 0, :5]) and torch.equal(v[0, 2, 5:7], new[0])
    after = ca.cart_pages_accept(k, v, table, lens, parents, _i32([1, 1, 1]))
    assert after.tolist() == [7, 5, 16]


def test_captured_step_replays():
    """A step of reserve, tree attention and accept captured into a graph
    gives the same results as eager calls, replay after replay."""
    def make():
        t, table, lens, parents = make_tree(51, 5, 7, 8, 2, 64, 40, (3, 40, 0, 17, 90), 16, "random")
        N = 64
        g = {k: v.cuda() for k, v in t.items()}
        for k in ("k_pages", "v_pages"):
            x = torch.zeros((N, 16, 2, 64), dtype=torch.bfloat16, device="cuda")
            x[:g[k].shape[0]] = g[k]
            g[k] = x
        wide = np.full((5, 12), -1, np.int32)
        wide[:, :table.shape[1]] = table
        g.update(table=_i32(wide), lens=_i32(lens), parents=_i32(parents),
                 refs=_i32(np.bincount(wide[wide >= 0], minlength=N)), node=_i32([0, 3, 6, -1, 5]))
        return g

    def step(g):
        rows = g["lens"] + 7
        ca.cart_pages_reserve(g["k_pages"][None], g["v_pages"][None], g["table"], g["lens"],
                              g["refs"], rows)
        o = ca.cart_attn_decode_tree(g["q"], g["k_new"], g["v_new"], g["kc"], g["vc"],
                                     g["k_pages"], g["v_pages"], g["table"], g["lens"],
                                     g["parents"])
        g["lens"].copy_(ca.cart_pages_accept(g["k_pages"][None], g["v_pages"][None], g["table"],
                                             g["lens"], g["parents"], g["node"]))
        return o

    a, b = make(), make()
    want = [step(a).clone() for _ in range(4)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    warm = make()
    step(warm)                                # lazy set-up before the capture
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        o = step(b)
    for w in want:
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, w)
    for k in ("table", "lens", "refs"):
        assert torch.equal(a[k], b[k])
    assert ca.device_status(clear=True) == 0


def test_calls_on_another_stream():
    """A stream given by the caller: outputs and workspaces belong to it."""
    t, table, lens, parents = make_tree(52, 4, 9, 8, 2, 128, 300, (3, 400, 0, 170), 64, "random")
    want, _ = run_tree(t, table, lens, parents)
    g = {k: v.cuda() for k, v in t.items()}
    tb, ln, up = _i32(table), _i32(lens), _i32(parents)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        o = ca.cart_attn_decode_tree(g["q"], g["k_new"], g["v_new"], g["kc"], g["vc"],
                                     g["k_pages"], g["v_pages"], tb, ln, up, stream=side)
        junk = torch.full((1 << 22,), float("nan"), device="cuda")   # reuses freed memory
        del junk
    side.synchronize()
    assert torch.equal(o, want)


@pytest.mark.parametrize("nodes", [24, 4])
def test_tree_repeats_bit_for_bit(nodes):
    t, table, lens, parents = make_tree(53, 9, nodes, 16, 2, 128, 700,
                                        (3, 400, 0, 170, 1000, 5, 90, 333, 64), 32, "random")
    a, _ = run_tree(t, table, lens, parents)
    for _ in range(3):
        b, _ = run_tree(t, table, lens, parents)
        assert torch.equal(a, b)


@pytest.mark.parametrize("p", [500, 1500])
def test_tree_calls_do_not_share_scratch(p):
    """Two calls in flight on two streams, each with a workspace of its own."""
    cases = [make_tree(60 + i, 6, 12, 8, 2, 128, p, (900, 2, 77, 300, 0, 640), 64, "random")
             for i in range(2)]
    want = [run_tree(*c)[0] for c in cases]
    gs = [{k: v.cuda() for k, v in c[0].items()} for c in cases]
    ints = [[_i32(x) for x in c[1:]] for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(6):
        for g, (tb, ln, up), s in zip(gs, ints, streams):
            with torch.cuda.stream(s):
                outs.append(ca.cart_attn_decode_tree(
                    g["q"], g["k_new"], g["v_new"], g["kc"], g["vc"], g["k_pages"], g["v_pages"],
                    tb, ln, up))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o, want[i % 2])
