"""CPU-only checks of the operators that hold a paged cache to a budget: what
they refuse, and the plain 64-bit forms that the GPU tests compare with."""
import ctypes
import math

import numpy as np
import pytest
import torch

from tests import budget_reference as bref
from tests import paged_reference as ref
from trained_kv_prefix_gb300 import build as cbuild
from trained_kv_prefix_gb300 import cartattn as ca

AL, ODD, ODD4 = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1002), ctypes.c_void_p(0x1004)
BIG = 1 << 40
BF, I32, F32 = torch.bfloat16, torch.int32, torch.float32


@pytest.fixture(scope="module")
def lib():
    cbuild.build()
    return ca.lib()


def append(lib, *, B=2, n=3, total=6, cu=None, Hkv=2, d=64, p=5, theta=1e6, k=AL, v=AL, kp=AL, vp=AL,
           N=8, P=16, table=AL, M=4, lens=AL, pos=None):
    return lib.cart_pages_append(B, n, total, cu, Hkv, d, p, theta, k, v, kp, vp, N, P, table, M,
                                 lens, pos, None)


def weigh(lib, *, B=2, T=3, window=0, sinks=0, Hq=4, Hkv=2, d=64, p=5, scale=0.1, theta=1e6, q=AL,
          lse=AL, kc=AL, kp=AL, N=8, P=16, table=AL, M=4, lens=AL, pos=None, acc=0, w=AL, W=64,
          cart=AL, ws=AL, ws_bytes=BIG):
    return lib.cart_attn_weights(B, T, window, sinks, Hq, Hkv, d, p, scale, theta, q, lse, kc, kp, N,
                                 P, table, M, lens, pos, acc, w, W, cart, ws, ws_bytes, None)


def evict(lib, *, B=2, layers=2, Hkv=2, d=64, dtype=0, kp=AL, vp=AL, N=8, P=16, table=AL, M=4,
          lens=AL, refs=AL, w=AL, W=64, keep=AL, first=1, recent=2, done=AL, ws=AL, ws_bytes=BIG):
    return lib.cart_pages_evict(B, layers, Hkv, d, dtype, kp, vp, N, P, table, M, lens, refs, w, W,
                                keep, first, recent, done, ws, ws_bytes, None)


def decode(lib, *, B=2, window=0, sinks=0, Hq=4, Hkv=2, d=64, p=5, scale=0.1, theta=1e6, q=AL,
           k_new=AL, v_new=AL, kc=AL, vc=AL, kp=AL, vp=AL, N=8, P=16, table=AL, M=4, lens=AL,
           pos=None, w=AL, W=64, o=AL, ws=AL, ws_bytes=BIG):
    return lib.cart_attn_decode_paged(B, window, sinks, Hq, Hkv, d, p, scale, theta, q, k_new, v_new,
                                      kc, vc, kp, vp, N, P, table, M, lens, pos, w, W, o, ws,
                                      ws_bytes, None)


@pytest.mark.parametrize("bad", [dict(B=0), dict(B=65536), dict(M=0), dict(N=0), dict(P=12),
                                 dict(P=256), dict(M=1 << 20), dict(N=(1 << 30) + 1)])
def test_tables_are_refused(lib, bad):
    for call in (append, weigh, evict, decode):
        assert call(lib, **bad) == -1, call.__name__


@pytest.mark.parametrize("bad", [
    dict(window=-1), dict(sinks=-1), dict(Hq=5), dict(Hq=18, Hkv=2), dict(Hkv=0), dict(d=96),
    dict(p=-1), dict(p=1 << 24), dict(scale=0.0), dict(scale=float("nan")), dict(theta=0.0),
    dict(theta=float("inf")), dict(W=63)])
def test_attention_geometry_is_refused(lib, bad):
    assert weigh(lib, **bad) == -1 and decode(lib, **bad) == -1


def test_append_refuses(lib):
    for bad in (dict(d=96), dict(p=-1), dict(p=1 << 24), dict(theta=0.0), dict(n=0, total=0),
                dict(total=5), dict(total=0, cu=AL)):
        assert append(lib, **bad) == -1, bad
    for name in ("k", "v", "kp", "vp"):
        assert append(lib, **{name: None}) == -2 and append(lib, **{name: ODD4}) == -2
    for name in ("table", "lens"):
        assert append(lib, **{name: None}) == -2 and append(lib, **{name: ODD}) == -2
    assert append(lib, cu=ODD) == -2 and append(lib, pos=ODD) == -2


def test_weights_refuse(lib):
    assert weigh(lib, T=0) == -1 and weigh(lib, T=1 << 24) == -1 and weigh(lib, acc=2) == -1
    for name in ("q", "kc", "kp", "w", "cart"):
        assert weigh(lib, **{name: None}) == -2 and weigh(lib, **{name: ODD4}) == -2
    for name in ("lse", "table", "lens"):
        assert weigh(lib, **{name: None}) == -2 and weigh(lib, **{name: ODD}) == -2
    assert weigh(lib, pos=ODD) == -2
    need = ca.weights_workspace_size(2, 3, 4, 2, 64, 5, 16, 4)
    assert need > 0 and ca.weights_workspace_size(2, 0, 4, 2, 64, 5, 16, 4) == 0
    assert weigh(lib, ws=None) == -4 and weigh(lib, ws_bytes=need - 1) == -4


def test_evict_refuses(lib):
    for bad in (dict(layers=0), dict(first=-1), dict(recent=-1), dict(W=63), dict(Hkv=4, d=4),
                dict(layers=32767, B=65535, Hkv=2)):
        assert evict(lib, **bad) == -1, bad
    assert evict(lib, dtype=5) == -3
    for name in ("kp", "vp"):
        assert evict(lib, **{name: None}) == -2 and evict(lib, **{name: ODD4}) == -2
    for name in ("table", "lens", "refs", "keep", "done"):
        assert evict(lib, **{name: None}) == -2 and evict(lib, **{name: ODD}) == -2
    assert evict(lib, w=ODD4) == -2
    need = ca.evict_workspace_size(2, 4, 8)
    assert need > 0 and ca.evict_workspace_size(2, 0, 8) == 0
    assert evict(lib, ws=None) == -4 and evict(lib, ws_bytes=need - 1) == -4


def test_decode_refuses(lib):
    for name in ("q", "k_new", "v_new", "kc", "vc", "kp", "vp", "o"):
        assert decode(lib, **{name: None}) == -2 and decode(lib, **{name: ODD4}) == -2
    for name in ("table", "lens"):
        assert decode(lib, **{name: None}) == -2 and decode(lib, **{name: ODD}) == -2
    assert decode(lib, pos=ODD) == -2 and decode(lib, w=ODD4) == -2
    need = ca.decode_paged_workspace_size(2, 4, 2, 64, 5, 16, 4, True)
    assert need >= ca.decode_paged_workspace_size(2, 4, 2, 64, 5, 16, 4, False) > 0
    assert ca.decode_paged_workspace_size(2, 5, 2, 64, 5, 16, 4, True) == 0
    assert decode(lib, ws=None) == -4 and decode(lib, ws_bytes=need - 1) == -4


def test_valid_arguments_reach_the_device_check(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert append(lib) in (-5, -6) and append(lib, cu=AL, total=5, n=0, pos=AL) in (-5, -6)
    assert weigh(lib) in (-5, -6) and weigh(lib, p=0, kc=None, cart=None, Hq=14) in (-5, -6)
    assert evict(lib) in (-5, -6) and evict(lib, w=None, W=0, dtype=1) in (-5, -6)
    assert decode(lib) in (-5, -6)
    assert decode(lib, p=0, kc=None, vc=None, w=None, W=0, Hq=14) in (-5, -6)


def zeros(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


def test_bindings_check_shapes_and_sizes():
    pool, table, lens = zeros(4, 16, 2, 64), zeros(2, 2, dtype=I32), zeros(2, dtype=I32)
    new, kc = zeros(2, 2, 64), zeros(5, 2, 64)
    w = zeros(2, 2, 32, dtype=F32)
    step = (zeros(2, 4, 64), new, new, kc, kc, pool, pool, table, lens)
    with pytest.raises(ValueError, match="pos"):
        ca.cart_attn_decode_paged(*step, pos=zeros(3, dtype=I32))
    with pytest.raises(TypeError, match="weights"):
        ca.cart_attn_decode_paged(*step, weights=w.double())
    with pytest.raises(ValueError, match="window"):
        ca.cart_attn_decode_paged(*step, window=1 << 32)
    with pytest.raises(ValueError, match="sinks"):
        ca.cart_attn_decode_paged(*step, sinks=-(1 << 31) - 1)
    with pytest.raises(ValueError, match="GPU"):
        ca.cart_attn_decode_paged(*step)
    q, lse = zeros(2, 3, 4, 64), zeros(2, 4, 3, dtype=F32)
    with pytest.raises(ValueError, match="lse"):
        ca.cart_attn_weights(q, zeros(2, 3, 4, dtype=F32), kc, pool, table, lens, w)
    with pytest.raises(ValueError, match="weights"):
        ca.cart_attn_weights(q, lse, kc, pool, table, lens, zeros(2, 4, 32, dtype=F32))
    with pytest.raises(ValueError, match="contiguous"):
        ca.cart_attn_weights(q, lse, kc, pool, table.t(), lens, w)
    with pytest.raises(ValueError, match="sinks"):
        ca.cart_attn_weights(q, lse, kc, pool, table, lens, w, sinks=1 << 31)
    k = zeros(2, 3, 2, 64)
    with pytest.raises(ValueError, match="v must be"):
        ca.cart_pages_append(k, k[:, :2].contiguous(), pool, pool, table, lens, p=5)
    with pytest.raises(TypeError, match="cu_seqlens"):
        ca.cart_pages_append(k[0], k[0], pool, pool, table, lens, p=5, cu_seqlens=zeros(3, dtype=F32))
    with pytest.raises(ValueError, match="p: "):
        ca.cart_pages_append(k, k, pool, pool, table, lens, p=1 << 33)
    refs, keep, layers = zeros(4, dtype=I32), lens, zeros(3, 4, 16, 2, 64)
    with pytest.raises(ValueError, match="weights"):
        ca.cart_pages_evict(layers, layers, table, lens, refs, w, keep)
    with pytest.raises(ValueError, match="recent"):
        ca.cart_pages_evict(layers, layers, table, lens, refs, None, keep, recent=1 << 32)
    with pytest.raises(ValueError, match="keep"):
        ca.cart_pages_evict(layers, layers, table, lens, refs, None, zeros(3, dtype=I32))


# ------------------------------------------------- the plain forms agree ----
def _state(seed, B=3, Hq=4, Hkv=2, d=8, p=7, P=16, M=3, lens=(0, 20, 33)):
    rng = np.random.default_rng(seed)
    N = B * M + 2
    table = rng.permutation(N)[:B * M].reshape(B, M)
    r = rng.standard_normal
    return rng, dict(q=r((B, Hq, d)), k_new=r((B, Hkv, d)), v_new=r((B, Hkv, d)), kc=r((p, Hkv, d)),
                     vc=r((p, Hkv, d)), k_pages=r((N, P, Hkv, d)), v_pages=r((N, P, Hkv, d)),
                     table=table, lens=np.array(lens))


def test_plain_decode_is_the_plain_tree_step():
    """Positions equal to places, no sinks: the tree of one node, with a window
    and without; and the weights of a step sum to the group's heads less the
    cartridge's share."""
    for window in (0, 9, 30):
        _, s = _state(window)
        o, _, w, _, wrote, lost = bref.decode(**s, window=window)
        t = dict(s, q=s["q"][:, None], k_new=s["k_new"][:, None], v_new=s["v_new"][:, None])
        o2, _, wrote2 = ref.tree(**t, parents=None, window=window)
        np.testing.assert_allclose(o, o2[:, 0], rtol=1e-12)
        assert not lost and wrote.keys() == wrote2.keys()
        total = w.sum(-1)
        assert (total <= 2 + 1e-12).all()
        if window == 9:         # the cartridge is out of sight of the longer two
            np.testing.assert_allclose(total[1:], 2.0, rtol=1e-12)


def test_plain_sinks_cut_and_keep():
    """All places sinks is no window; sinks at or below the window change nothing."""
    _, s = _state(5)
    full = bref.decode(**s)[0]
    np.testing.assert_array_equal(bref.decode(**s, window=4, sinks=100)[0], full)
    np.testing.assert_array_equal(bref.decode(**s, window=1000, sinks=3)[0], full)
    a = bref.decode(**s, window=12, sinks=3)[0]
    assert np.abs(a - full).max() > 1e-3 and np.abs(a - bref.decode(**s, window=12)[0]).max() > 1e-3


def test_plain_weights_are_the_steps_weights():
    """The weights of a conversation's last queries are what single-token steps
    of the same tokens add up."""
    rng, s = _state(8)
    P, p, N = 16, 7, s["k_pages"].shape[0]
    B, T, lens = 3, 4, s["lens"].copy()
    q = rng.standard_normal((B, T, 4, 8))
    total, lse = np.zeros((B, 2, 48)), np.zeros((B, 4, T))
    for i in range(T):
        t = dict(s, q=q[:, i], lens=lens + i)
        o, _, w, _, wrote, _ = bref.decode(**t, window=25, sinks=2)
        for at, (k, v) in wrote.items():
            s["k_pages"][at], s["v_pages"][at] = k, v
        total += w
        for b in range(B):      # log-sum-exps from the parts
            n = lens[b] + i
            for h in range(4):
                x = ref.rope(q[b, i, h], p + n)
                ys = list(range(p)) + [p + r for r in range(n + 1)]
                ks = [s["kc"][y, h // 2] if y < p else
                      s["k_pages"][ref.page_at(s["table"][b], y - p, N, P)][h // 2] for y in ys]
                z = [k @ x / math.sqrt(8) for y, k in zip(ys, ks) if bref.sees(p + n, y, 25, 2)]
                lse[b, h, i] = np.log(np.exp(z).sum())
    w, bound, held = bref.weigh(q, lse, s["kc"], s["k_pages"], s["table"], lens + T, window=25, sinks=2)
    np.testing.assert_array_equal(held, lens + T)
    np.testing.assert_allclose(w[..., p:], total, rtol=1e-9, atol=1e-12)
    np.testing.assert_allclose(w.sum((1, 2)), 4 * T, rtol=1e-9)


def test_plain_evict_keeps_order_and_counts():
    rng = np.random.default_rng(3)
    B, M, P, layers, Hkv, N = 4, 4, 16, 2, 2, 24
    table = np.full((B, M), -1, np.int32)
    table[0], table[1], table[2, :2] = [0, 1, 2, 3], [0, 1, 4, 5], [6, 7]
    table[3] = [8, -1, 9, 10]
    refs = np.bincount(table[table >= 0], minlength=N).astype(np.int32)
    lens = np.array([60, 50, 20, 64], np.int32)
    w = rng.random((layers, B, Hkv, M * P)).astype(np.float32)
    out, n, r, done, w2, moves, stay = bref.evict(table, lens, refs, w, np.array([33, 33, 20, 5]), 17,
                                                  5, layers, Hkv, P)
    assert list(done) == [1, 1, 1, 0] and list(n) == [33, 33, 20, 64] and stay[2] is None
    for b in (0, 1):
        for layer in range(layers):
            for g in range(Hkv):
                rows = stay[b][layer][g]
                assert rows == sorted(set(rows)) and len(rows) == 33
                assert rows[:17] == list(range(17)) and rows[-5:] == list(range(lens[b] - 5, lens[b]))
                np.testing.assert_array_equal(w2[layer, b, g, :33], w[layer, b, g, rows])
    assert out[0, 0] == 0 and out[1, 0] == 0 and out[0, 1] == 11 and out[1, 1] == 12
    assert out[0, 2] == 2 and out[0, 3] == -1 and r[3] == 0 and r[0] == 2 and r[1] == 0
