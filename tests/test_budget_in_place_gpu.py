"""Outputs of the calls that hold a paged cache to a budget in the place of inputs
that they are allowed to be."""
import numpy as np
import pytest
import torch

from tests.test_budget_gpu import _f32, _i32, make_evict, make_step
from trained_kv_prefix_gb300 import cartattn as ca

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads", [(32, 8), (8, 8), (8, 1)])
def test_step_writes_over_its_queries(heads):
    """... with a table so wide that blocks beside the output's give the rows'
    weights: one or two conversations, and one without a page."""
    for B, lens in ((1, (900,)), (3, (4000, -1, 16 * 260))):
        t, table, n, _ = make_step(41, B, *heads, 128, 70, lens, 16)
        M = max(600, table.shape[1])
        table = np.concatenate([table, np.full((B, M - table.shape[1]), -1, np.int32)], 1)
        if B == 3:
            table[2, 260] = -1                  # the new row's page
        got = []
        for place in (False, True):
            g = {k: v.cuda() for k, v in t.items()}
            w = torch.zeros(B, heads[1], M * 16, device="cuda")
            o = g["q"] if place else torch.empty_like(g["q"])
            for turn in range(4):
                q = t["q"].cuda()
                if place:
                    o.copy_(q)
                r = ca.cart_attn_decode_paged(o if place else q, g["k_new"], g["v_new"], g["kc"],
                                              g["vc"], g["k_pages"], g["v_pages"], _i32(table),
                                              _i32(n), weights=w, o=o)
                assert r is o
            torch.cuda.synchronize()
            got.append((o.clone(), w))
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
        assert ca.device_status(clear=True) == (1 << 7 if B == 3 else 0)


def test_evict_writes_done_over_keep():
    """Many blocks that read keep while others are through."""
    pools, table, lens, refs, w = make_evict(43, 9, 12, 8, 64, 16,
                                             (300, 250, 7, 120, 400, -1, 33, 64, 500), spare=2)
    table[3, 1] = -1                            # a page that is not there
    keep = (100, 250, 9, 40, 39, 5, -1, 1, 0)
    got = []
    for place in (False, True):
        g = [x.cuda() for x in pools]
        gt, gl, gr, gw, k = _i32(table), _i32(lens), _i32(refs), _f32(w), _i32(keep)
        done = ca.cart_pages_evict(*g, gt, gl, gr, gw, k, first=3, recent=9,
                                   done=k if place else None)
        got.append((done, *g, gt, gl, gr, gw))
    assert got[0][0].tolist() == [1, 1, 1, 0, 1, 1, 1, 1, 1]
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(*got))
    assert ca.device_status(clear=True) == 0
