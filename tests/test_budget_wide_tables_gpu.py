"""The step with tables that name many more rows than are held, as an eviction
leaves them: what a narrow table gives, to the joined parts' order."""
import numpy as np
import pytest
import torch

from tests.test_budget_gpu import check_step, make_step, run_step
from trained_kv_prefix_gb300 import cartattn as ca

pytestmark = pytest.mark.gpu


def widen(table, rows, P):
    more = rows // P - table.shape[1]
    return np.concatenate([table, np.full((len(table), more), -1, np.int32)], 1)


@pytest.mark.parametrize("rows", [1024, 16384])
@pytest.mark.parametrize("case", [
    # B, Hq, Hkv, d, p, lens, P, window, sinks
    (1, 32, 8, 128, 512, (201,), 16, 0, 0),
    (3, 8, 2, 64, 1100, (0, 90, 333), 16, 0, 0),
    (20, 8, 2, 128, 700, tuple(range(0, 400, 20)), 64, 0, 0),
    (20, 28, 4, 64, 300, tuple(range(5, 405, 20)), 32, 120, 30),
])
def test_step_parity_in_wide_tables(case, rows):
    B, Hq, Hkv, d, p, lens, P, window, sinks = case
    t, table, n, pos = make_step(51 + B, B, Hq, Hkv, d, p, lens, P)
    check_step(t, widen(table, rows, P), n, pos, window=window, sinks=sinks)


def test_wide_tables_change_no_more_than_the_order_of_sums():
    t, table, n, pos = make_step(52, 16, 32, 8, 128, 2048, tuple(range(10, 810, 50)), 64)
    got = []
    for rows in (table.shape[1] * 64, 8192, 65536):
        w = torch.zeros(16, 8, rows, device="cuda")
        o, _ = run_step(t, widen(table, rows, 64), n, pos, w)
        got.append((o.double(), w[:, :, :768].double()))
    for o, w in got[1:]:
        # outputs round to bf16 once each, to neighbours at most; weights are f32
        # whose log-sum-exp is joined from other parts
        assert ((o - got[0][0]).abs() <= 2.0 ** -7 * got[0][0].abs() + 1e-5).all()
        assert ((w - got[0][1]).abs() <= 1e-5 * got[0][1] + 1e-12).all()
    assert ca.device_status(clear=True) == 0
