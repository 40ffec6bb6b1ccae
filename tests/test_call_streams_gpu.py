"""Calls on a stream that the caller names, while the current stream still has
work to do on memory that it has freed."""
import numpy as np
import pytest
import torch

from tests import paged_reference as ref
from tests.test_paged_gpu import _i32, _pool, make_tables, make_tree, run_tree
from trained_kv_prefix_gb300 import cartattn as ca
from trained_kv_prefix_gb300 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture
def busy():
    """Makes the current stream busy for some milliseconds and leaves freed
    blocks of the sizes asked for, which it has yet to fill, in its cache."""
    x = torch.randn(8192, 8192, device="cuda").to(torch.bfloat16)
    y = torch.empty_like(x)

    def go(*sizes):
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
        for _ in range(20):
            torch.matmul(x, x, out=y)
        for b in blocks:
            b.fill_(255)

    yield go
    torch.cuda.synchronize()


@pytest.mark.parametrize("p", [300, 1500])
def test_tree_beside_a_busy_stream(busy, p):
    t, table, lens, parents = make_tree(71, 6, 9, 8, 2, 128, p, (3, 400, 0, 170, 60, 9), 64,
                                        "random")
    want, _ = run_tree(t, table, lens, parents)
    g = {k: v.cuda() for k, v in t.items()}
    tb, ln, up = _i32(table), _i32(lens), _i32(parents)
    need = ca.decode_tree_workspace_size(6, 9, 8, 2, 128, p, 64, table.shape[1])
    side = torch.cuda.Stream()
    busy(need, want.numel() * 2)
    outs = [ca.cart_attn_decode_tree(g["q"], g["k_new"], g["v_new"], g["kc"], g["vc"],
                                     g["k_pages"], g["v_pages"], tb, ln, up, stream=side)
            for _ in range(3)]
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)
    assert ca.device_status(clear=True) == 0


def test_reserve_accept_and_compact_beside_a_busy_stream(busy):
    B, M, P, N, nodes = 70, 5, 64, 400, 3
    rng = np.random.default_rng(72)
    table, lens, refs = make_tables(rng, B, M, P, N)
    rows = np.where(lens < 0, -1, np.minimum(lens + nodes, M * P)).astype(np.int32)
    k, v = (_pool((2, N, P, 2, 64), torch.bfloat16, s) for s in (1, 2))
    wk, wv = k.clone(), v.clone()
    wt, wl, wr, wd, copies = ref.reserve(table, lens, refs, rows, P)
    assert copies
    for x in (wk, wv):
        before = x.clone()
        for a, z, n in copies:
            x[:, z, :n] = before[:, a, :n]
    # the last node's row to the front where the conversation has room
    parents = np.tile(np.array([-1, -1, -1], np.int32), (B, 1))
    node = np.where(wd == 1, 2, -1).astype(np.int32)
    step = np.where(wd == 1, wl, -1).astype(np.int32)
    wn, moves = ref.accept(wt, step, parents, node, N, P, nodes)
    for x in (wk, wv):
        before = x.clone()
        for (a, i), (z, j) in moves:
            x[:, z, j] = before[:, a, i]
    ct, cr, cm, cn, copies = ref.compact(wt, wr)
    for x in (wk, wv):
        before = x.clone()
        for a, z in copies:
            x[:, z] = before[:, a]
    tb, ln, rf, rw = _i32(table), _i32(lens), _i32(refs), _i32(rows)
    up, nd, st = _i32(parents), _i32(node), _i32(step)
    side = torch.cuda.Stream()
    busy(ca.pages_workspace_size(B, M, N), 4 * B, 4 * N, 4)
    done = ca.cart_pages_reserve(k, v, tb, ln, rf, rw, stream=side)
    after = ca.cart_pages_accept(k, v, tb, st, up, nd, stream=side)
    moved, live = ca.cart_pages_compact(k, v, tb, rf, stream=side)
    torch.cuda.synchronize()
    for got, w in ((done, wd), (ln, wl), (after, wn), (tb, ct), (rf, cr), (moved, cm)):
        np.testing.assert_array_equal(got.cpu().numpy(), w)
    assert int(live) == cn
    assert torch.equal(k, wk) and torch.equal(v, wv)


def test_fork_beside_a_busy_stream(busy):
    B, M, P, N = 40, 9, 64, 400
    rng = np.random.default_rng(73)
    table, lens, refs = make_tables(rng, B, M, P, N)
    order = rng.permutation(B).astype(np.int32)
    src, dst = order[:15], order[15:30]
    want = ref.fork(table, lens, refs, src, dst, None, P)
    tb, ln, rf, a, z = _i32(table), _i32(lens), _i32(refs), _i32(src), _i32(dst)
    side = torch.cuda.Stream()
    busy(4 * 15)
    done = ca.cart_pages_fork(tb, ln, rf, a, z, page_rows=P, stream=side)
    torch.cuda.synchronize()
    for got, w in zip((tb, ln, rf, done), want):
        np.testing.assert_array_equal(got.cpu().numpy(), w)


def test_training_step_beside_a_busy_stream(busy):
    """Forward and backward that add to gradients of their own: the same bits
    as on the current stream."""
    s = synth.TrainShape("side", B=2, n=150, Hq=4, Hkv=2, d=64, p=40, dtype="bf16", seed=74)
    g = {k: v.cuda() for k, v in synth.train_inputs(s).items()}
    args = [g[k] for k in ("q", "k", "v", "kc", "vc")]

    def step(**kw):
        o, lse = ca.cart_attn_fwd(*args, **kw)
        return (o, lse) + ca.cart_attn_bwd(*args, o, lse, g["do"], accumulate=True, **kw)

    want = step()
    side = torch.cuda.Stream()
    geom = ca.geom(2, 150, 4, 2, 64, 40)
    busy(ca.fwd_workspace_size(geom, 0, 1), ca.bwd_workspace_size(geom, 0, 1),
         *(t.numel() * t.element_size() for t in want))
    got = step(stream=side)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert ca.device_status(clear=True) == 0


def test_decode_step_beside_a_busy_stream(busy):
    s = synth.DecodeShape("side", B=3, Hq=4, Hkv=2, d=128, p=400, max_private=90, seed=75,
                          fixed_len=(0, 7, 90))
    g = {k: v.cuda() for k, v in synth.decode_inputs(s).items()}
    args = [g[k] for k in ("q", "k_new", "v_new", "kc", "vc", "k_cache", "v_cache", "lens")]
    want = ca.cart_attn_decode(*args)
    side = torch.cuda.Stream()
    busy(ca.decode_workspace_size(3, 4, 2, 128, 400, g["k_cache"].shape[1]), want.numel() * 2)
    got = ca.cart_attn_decode(*args, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_captured_on_a_forked_stream():
    """A capture that hands the calls to a stream of its own: what they allocate
    lives as long as the graph."""
    t, table, lens, parents = make_tree(76, 4, 9, 8, 2, 128, 700, (3, 400, 0, 170), 64, "random")
    want, _ = run_tree(t, table, lens, parents)
    g = {k: v.cuda() for k, v in t.items()}
    tb, ln, up = _i32(table), _i32(lens), _i32(parents)
    refs = _i32(np.bincount(table[table >= 0], minlength=g["k_pages"].shape[0]))
    rows = ln + 9
    side = torch.cuda.Stream()

    def step(**kw):
        done = ca.cart_pages_reserve(g["k_pages"][None], g["v_pages"][None], tb, ln, refs, rows, **kw)
        return done, ca.cart_attn_decode_tree(g["q"], g["k_new"], g["v_new"], g["kc"], g["vc"],
                                              g["k_pages"], g["v_pages"], tb, ln, up, **kw)

    step(stream=side)                         # lazy set-up before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        now = torch.cuda.current_stream()
        side.wait_stream(now)
        done, o = step(stream=side)
        now.wait_stream(side)
    for _ in range(3):
        o.fill_(float("nan"))
        done.fill_(7)
        graph.replay()
        junk = torch.full((1 << 24,), float("nan"), device="cuda")
        del junk
        torch.cuda.synchronize()
        assert torch.equal(o, want) and done.tolist() == [1] * 4
    assert ca.device_status(clear=True) == 0
