"""The order that the dK / dV kernel's shared-memory rings rely on, read from
its source: a ring slot is loaded again once its empty barrier has all arrivals,
so every reader has to be ahead of an arrival of its own there, or of the one that
the product which arrives there is issued behind.  (A reader behind it sees the
slot's next contents now and then, which no result can be relied on to show.)"""
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "trained_kv_prefix_gb300", "csrc", "bwd.cu")


@pytest.fixture(scope="module")
def kernel():
    with open(SOURCE) as f:
        text = f.read()
    return text[text.index("    dkdv_kernel("):text.index("dQ ======")]


def ring_of(kernel, vec):
    """The ring ("Q" or "Do") whose full barrier the copies of a vector complete."""
    rings = re.findall(r"bulk_load\(" + vec + r" \+ s\w \* 128,[^;]*?&bars\[k(\w+?)Full0 \+ s\w\]\)",
                       kernel)
    assert len(rings) == 1, rings
    return rings[0]


def release(kernel, ring):
    """What a reading warp does last before a slot of the ring can be loaded again:
    its own arrival on the empty barrier, where that counts the 16 warps beside the
    product, or the arrival that the releasing product is issued behind."""
    own = f"mbar_arrive(&bars[k{ring}Empty0 + "
    if f"mbar_init(&bars[k{ring}Empty0 + s], 17)" in kernel:
        assert kernel.count(own) == 1
        return own
    assert f"mbar_init(&bars[k{ring}Empty0 + s], 1)" in kernel and own not in kernel
    at = kernel.index(f"umma_commit_w(&bars[k{ring}Empty0 + ")
    waits = [m for m in re.finditer(r"ok = wait\(&bars\[(kPtFull|kDsFull)\]", kernel) if m.start() < at]
    return f"mbar_arrive(&bars[{waits[-1].group(1)}])"


@pytest.mark.parametrize("vec,address", [("vecL", "lse_s"), ("vecD", "dv_s")])
def test_row_vectors_are_read_before_their_slot_is_released(kernel, vec, address):
    arrive = kernel.index(release(kernel, ring_of(kernel, vec)))
    reads = [m.start() for m in re.finditer(r"lds128\(" + address, kernel)]
    assert reads and max(reads) < arrive


@pytest.mark.parametrize("vec,address", [("vecL", "lse_s"), ("vecD", "dv_s")])
def test_row_vectors_are_read_behind_their_copies(kernel, vec, address):
    """A wait for the ring's full barrier stands before the first read, and the
    address steps with the ring."""
    ring = ring_of(kernel, vec)
    roles = kernel[kernel.index("P^T / dS^T warpgroups 0-3"):]
    assert roles.index(f"mbar_wait(&bars[k{ring}Full0 + ") < roles.index(f"lds128({address}")
    slot = {"Q": "sq", "Do": "sd"}[ring]
    assert f"{address} = smem_u32({vec} + {slot} * 128" in roles


def test_vectors_have_a_slot_for_every_slot_of_their_ring(kernel):
    with open(SOURCE) as f:
        text = f.read()
    area = text[text.index("struct DkdvSmem"):text.index("enum DkdvBar")]
    after = {"vecL": r"kVecD = kVecL \+ kDkdv(\w+)Slots \* 512",
             "vecD": r"kBar = kVecD \+ kDkdv(\w+)Slots \* 512"}
    for vec, pattern in after.items():
        assert re.search(pattern, area).group(1) == ring_of(kernel, vec)
