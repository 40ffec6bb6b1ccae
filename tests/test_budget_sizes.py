"""Sizes of the calls that hold a paged cache to a budget, on the CPU."""
import types

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


def test_step_workspace_is_the_devices_own(monkeypatch):
    """The work is cut for a device's multiprocessors: a size that was asked for
    on one device, or on none, is not another one's."""
    now = {"device": None}
    cuda = types.SimpleNamespace(is_available=lambda: now["device"] is not None,
                                 current_device=lambda: now["device"])
    size = {None: 100, 0: 4096, 1: 8192}
    monkeypatch.setattr(ca, "torch", types.SimpleNamespace(cuda=cuda))
    monkeypatch.setattr(ca, "lib", lambda: types.SimpleNamespace(
        cart_attn_decode_paged_workspace_size=lambda *args: size[now["device"]]))
    ca.decode_paged_workspace_size.cache_clear()
    for device in (None, 0, 1, 0, None, 1):
        now["device"] = device
        assert ca.decode_paged_workspace_size(2, 4, 2, 64, 5, 16, 3, True) == size[device]
    ca.decode_paged_workspace_size.cache_clear()
