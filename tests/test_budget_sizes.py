"""Sizes of the calls that hold a paged cache to a budget, on the CPU."""
import pytest

from trained_kv_prefix_gb300 import build as cbuild
from trained_kv_prefix_gb300 import cartattn as ca


@pytest.fixture(scope="module", autouse=True)
def lib():
    cbuild.build()
    return ca.lib()


@pytest.mark.parametrize("B,Hq,Hkv", [(1, 32, 8), (1, 4, 1), (2, 2, 2), (3, 28, 4)])
@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("M", [1, 2, 3, 13, 14])
def test_step_workspace_holds_the_logits_that_are_walked(B, Hq, Hkv, P, M):
    """Rows are walked in groups of 32, pages of 16 or not: a new token in the
    table's last row has the logits of whole groups read, those of the last
    conversation's last head too."""
    size = [ca.decode_paged_workspace_size(B, Hq, Hkv, 64, 5, P, M, w) for w in (False, True)]
    walked = -(-(M * P - 1) // 32) * 32
    assert size[0] > 0 and size[1] - size[0] >= B * Hq * walked * 4
