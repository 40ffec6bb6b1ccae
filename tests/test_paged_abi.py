"""CPU-only checks of the paged serving entry points: what they refuse, and
the plain 64-bit forms that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

from tests import paged_reference as ref
from trained_kv_prefix_gb300 import build as cbuild
from trained_kv_prefix_gb300 import cartattn as ca

AL, ODD = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1002)
ODD4 = ctypes.c_void_p(0x1004)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    cbuild.build()
    return ca.lib()


def tree(lib, *, B=2, nodes=4, window=0, Hq=8, Hkv=2, d=128, p=16, scale=0.1, theta=1e6, q=AL,
         k_new=AL, v_new=AL, kc=AL, vc=AL, kp=AL, vp=AL, N=8, P=16, table=AL, M=4, lens=AL,
         parents=AL, o=AL, ws=AL, ws_bytes=BIG):
    return lib.cart_attn_decode_tree(B, nodes, window, Hq, Hkv, d, p, scale, theta, q, k_new, v_new,
                                     kc, vc, kp, vp, N, P, table, M, lens, parents, o, ws, ws_bytes,
                                     None)


@pytest.mark.parametrize("bad", [
    dict(B=0), dict(nodes=0), dict(nodes=65), dict(window=-1), dict(Hq=6, Hkv=2), dict(Hq=32, Hkv=2),
    dict(Hkv=3), dict(d=96), dict(p=-1), dict(scale=0.0), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(theta=0.0), dict(theta=float("nan")), dict(N=0), dict(P=8),
    dict(P=48), dict(P=256), dict(M=0), dict(M=1 << 20), dict(p=1 << 24), dict(B=2000, nodes=64),
    dict(N=(1 << 30) + 1)])
def test_tree_refuses_geometry(lib, bad):
    assert tree(lib, **bad) == -1


@pytest.mark.parametrize("name", ["q", "k_new", "v_new", "kc", "vc", "kp", "vp", "o"])
def test_tree_refuses_pointers(lib, name):
    assert tree(lib, **{name: None}) == -2
    assert tree(lib, **{name: ODD4}) == -2


def test_tree_refuses_tables_and_workspaces(lib):
    for name in ("table", "lens"):
        assert tree(lib, **{name: None}) == -2
        assert tree(lib, **{name: ODD}) == -2
    assert tree(lib, parents=ODD) == -2
    need = ca.decode_tree_workspace_size(2, 4, 8, 2, 128, 16, 16, 4)
    assert need > 0
    assert tree(lib, ws=None) == -4 and tree(lib, ws_bytes=need - 1) == -4
    assert tree(lib, ws=ODD4) == -4
    assert ca.decode_tree_workspace_size(2, 65, 8, 2, 128, 16, 16, 4) == 0
    assert ca.decode_tree_workspace_size(2, 4, 8, 2, 128, 16, 24, 4) == 0


def test_valid_arguments_reach_the_device_check(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert tree(lib) in (-5, -6)
    assert tree(lib, kc=None, vc=None, p=0, parents=None) in (-5, -6)
    assert fork(lib) in (-5, -6) and reserve(lib) in (-5, -6)
    assert accept(lib) in (-5, -6) and compact(lib) in (-5, -6)


def fork(lib, *, B=2, table=AL, M=4, lens=AL, refs=AL, N=8, P=16, src=AL, dst=AL, rows=None, F=1,
         done=AL):
    return lib.cart_pages_fork(B, table, M, lens, refs, N, P, src, dst, rows, F, done, None)


def reserve(lib, *, B=2, layers=1, Hkv=2, d=64, dtype=0, kp=AL, vp=AL, N=8, P=16, table=AL, M=4,
            lens=AL, refs=AL, rows=AL, done=AL, ws=AL, ws_bytes=BIG):
    return lib.cart_pages_reserve(B, layers, Hkv, d, dtype, kp, vp, N, P, table, M, lens, refs, rows,
                                  done, ws, ws_bytes, None)


def accept(lib, *, B=2, nodes=4, layers=1, Hkv=2, d=64, dtype=0, kp=AL, vp=AL, N=8, P=16, table=AL,
           M=4, lens=AL, parents=AL, node=AL, new=ctypes.c_void_p(0x2000)):
    return lib.cart_pages_accept(B, nodes, layers, Hkv, d, dtype, kp, vp, N, P, table, M, lens,
                                 parents, node, new, None)


def compact(lib, *, B=2, layers=1, Hkv=2, d=64, dtype=0, kp=AL, vp=AL, N=8, P=16, table=AL, M=4,
            refs=AL, moved=AL, live=AL, ws=AL, ws_bytes=BIG):
    return lib.cart_pages_compact(B, layers, Hkv, d, dtype, kp, vp, N, P, table, M, refs, moved, live,
                                  ws, ws_bytes, None)


@pytest.mark.parametrize("bad", [dict(B=0), dict(B=65536), dict(M=0), dict(N=0), dict(P=12),
                                 dict(P=256), dict(M=1 << 20), dict(N=(1 << 30) + 1)])
def test_page_operators_refuse_tables(lib, bad):
    for call in (fork, reserve, accept, compact):
        assert call(lib, **bad) == -1, call.__name__


def test_page_operators_refuse_pools(lib):
    for call in (reserve, accept, compact):
        assert call(lib, layers=0) == -1
        assert call(lib, Hkv=1, d=4) == -1            # a row of 8 bytes
        assert call(lib, dtype=5) == -3
        assert call(lib, kp=None) == -2 and call(lib, vp=ODD4) == -2
    for call in (reserve, compact):
        assert call(lib, ws=None) == -4 and call(lib, ws_bytes=64) == -4
        assert call(lib, table=ODD) == -2 and call(lib, refs=None) == -2
    assert ca.pages_workspace_size(2, 4, 8) > 0 and ca.pages_workspace_size(0, 4, 8) == 0


def test_page_operators_refuse_lists(lib):
    assert fork(lib, F=0) == -1 and fork(lib, F=8193) == -1
    for name in ("table", "lens", "refs", "src", "dst", "done"):
        assert fork(lib, **{name: None}) == -2 and fork(lib, **{name: ODD}) == -2
    assert fork(lib, rows=ODD) == -2
    assert reserve(lib, rows=None) == -2 and reserve(lib, done=None) == -2
    assert accept(lib, nodes=65) == -1 and accept(lib, nodes=0) == -1
    assert accept(lib, node=None) == -2 and accept(lib, parents=ODD) == -2
    assert accept(lib, new=AL) == -2                  # lens itself
    assert compact(lib, moved=None) == -2 and compact(lib, live=ODD) == -2


def _tree_tensors():
    bf, i32 = torch.bfloat16, torch.int32
    return dict(q=torch.zeros(2, 3, 4, 64, dtype=bf), k_new=torch.zeros(2, 3, 2, 64, dtype=bf),
                v_new=torch.zeros(2, 3, 2, 64, dtype=bf), kc=torch.zeros(5, 2, 64, dtype=bf),
                vc=torch.zeros(5, 2, 64, dtype=bf), k_pages=torch.zeros(4, 16, 2, 64, dtype=bf),
                v_pages=torch.zeros(4, 16, 2, 64, dtype=bf), table=torch.zeros(2, 2, dtype=i32),
                lens=torch.zeros(2, dtype=i32), parents=torch.zeros(2, 3, dtype=i32))


@pytest.mark.parametrize("name", list(_tree_tensors()))
def test_tree_binding_refuses_types_shapes_and_strides(lib, name):
    t = _tree_tensors()
    with pytest.raises(TypeError):
        ca.cart_attn_decode_tree(**{**t, name: t[name].double()})
    wide = torch.zeros(*t[name].shape[:-1], 2 * t[name].shape[-1], dtype=t[name].dtype)
    with pytest.raises(ValueError):
        ca.cart_attn_decode_tree(**{**t, name: wide[..., ::2]})
    if name not in ("q", "table"):
        with pytest.raises(ValueError):
            ca.cart_attn_decode_tree(**{**t, name: torch.cat([t[name], t[name]], -1)})


def test_page_bindings_refuse_types_shapes_and_strides(lib):
    t = _tree_tensors()
    k, v, table, lens = t["k_pages"][None], t["v_pages"][None], t["table"], t["lens"]
    refs, rows, up, node = torch.zeros(4, dtype=torch.int32), lens, t["parents"], lens
    with pytest.raises(ValueError):
        ca.cart_pages_reserve(k, v[:, :3], table, lens, refs, rows)
    with pytest.raises(TypeError):
        ca.cart_pages_reserve(k, v.float(), table, lens, refs, rows)
    with pytest.raises(TypeError):
        ca.cart_pages_reserve(k.half(), v.half(), table, lens, refs, rows)
    with pytest.raises(ValueError):
        ca.cart_pages_reserve(k, v, table, lens, refs[:3], rows)
    with pytest.raises(TypeError):
        ca.cart_pages_accept(k, v, table, lens.long(), up, node)
    with pytest.raises(ValueError):
        ca.cart_pages_accept(k, v, table, lens, up[:, ::2], node)
    with pytest.raises(ValueError):
        ca.cart_pages_compact(k.transpose(1, 2), v.transpose(1, 2), table, refs)
    with pytest.raises(ValueError):
        ca.cart_pages_fork(table, lens, refs, lens, lens[:1], page_rows=16)
    with pytest.raises(TypeError):
        ca.cart_pages_fork(table.float(), lens, refs, lens, lens, page_rows=16)


# ------------------------------------------------- the plain forms themselves
def test_reference_chain_equals_the_span_oracle(oracle_lib):
    """The tree form over a chain is the oracle's span verify over the same
    rows kept densely."""
    rng = np.random.default_rng(1)
    B, nodes, Hq, Hkv, d, p, rows, P = 3, 4, 4, 2, 64, 9, 48, 16
    x = {k: rng.standard_normal(s) for k, s in dict(
        q=(B, nodes, Hq, d), k_new=(B, nodes, Hkv, d), v_new=(B, nodes, Hkv, d), kc=(p, Hkv, d),
        vc=(p, Hkv, d), k=(B, rows, Hkv, d), v=(B, rows, Hkv, d)).items()}
    lens = np.array([0, 17, rows - nodes], np.int32)
    table = np.arange(B * rows // P).reshape(B, -1)
    for window in (0, 20):
        o, _, _ = ref.tree(x["q"], x["k_new"], x["v_new"], x["kc"], x["vc"],
                           x["k"].reshape(-1, P, Hkv, d), x["v"].reshape(-1, P, Hkv, d), table,
                           lens, None, window=window)
        want, _, _ = oracle_lib.decode_span(x["q"], x["k_new"], x["v_new"], x["kc"], x["vc"],
                                            x["k"], x["v"], lens, theta=1e6, window=window)
        assert np.abs(o - want).max() <= 1e-10


def test_reference_path_equals_its_chain():
    """A node attends to what the chain of its ancestors would."""
    rng = np.random.default_rng(2)
    B, nodes, Hq, Hkv, d, p, P = 1, 7, 2, 1, 64, 5, 16
    x = {k: rng.standard_normal(s) for k, s in dict(
        q=(B, nodes, Hq, d), k_new=(B, nodes, Hkv, d), v_new=(B, nodes, Hkv, d), kc=(p, Hkv, d),
        vc=(p, Hkv, d), k_pages=(3, P, Hkv, d), v_pages=(3, P, Hkv, d)).items()}
    table, lens = np.array([[2, 0]]), np.array([20], np.int32)
    parents = np.array([[-1, 0, 0, 1, -1, 3, 2]])
    o, bound, wrote = ref.tree(**x, table=table, lens=lens, parents=parents)
    path = [0, 1, 3, 5]
    chain = {**x, **{k: x[k][:, path] for k in ("q", "k_new", "v_new")}}
    want, _, _ = ref.tree(**chain, table=table, lens=lens, parents=None)
    assert np.abs(o[:, path] - want).max() <= 1e-12
    assert (bound > 0).all() and len(wrote) == nodes


def test_reference_reserve_and_compact_keep_the_counts():
    table = np.array([[0, 1, -1], [0, 1, -1], [3, -1, -1]], np.int32)
    refs = np.array([2, 2, 0, 1, 0, 0], np.int32)
    t, l, r, done, copies = ref.reserve(table, np.array([20, 20, 3]), refs, [33, -1, 0], 16)
    assert copies == [(1, 2, 4)] and done.tolist() == [1, 0, 1]
    assert t.tolist() == [[0, 2, 3], [0, 1, -1], [-1, -1, -1]] and r.tolist() == [2, 1, 1, 1, 0, 0]
    t, r, moved, n, copies = ref.compact(np.array([[4, 1], [4, 5]]), np.array([0, 1, 0, 0, 2, 1]))
    assert n == 3 and copies == [(4, 0), (5, 2)] and t.tolist() == [[0, 1], [0, 2]]
    assert r.tolist() == [2, 1, 1, 0, 0, 0] and moved.tolist() == [-1, 1, -1, -1, 0, 2]
