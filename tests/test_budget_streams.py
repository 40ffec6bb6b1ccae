"""Where the bindings of the calls that hold a cache to a budget allocate what
they make themselves, on the CPU."""
import pytest

from tests.test_call_streams import F32, Device, Stream, check, ints, new, pools
from tests.test_call_streams import fake as _fake  # noqa: F401
from trained_kv_prefix_gb300 import cartattn as ca


@pytest.fixture
def fake(_fake):  # noqa: F811
    sizes = (ca.weights_workspace_size, ca.evict_workspace_size, ca.decode_paged_workspace_size)
    for f in sizes:
        f.cache_clear()
    yield _fake
    for f in sizes:
        f.cache_clear()


CALLS = {
    "weights": lambda **kw: ca.cart_attn_weights(
        new(3, 4, 8, 64), new(3, 8, 4, dtype=F32), new(5, 2, 64), new(8, 16, 2, 64), ints(3, 2),
        ints(3), new(3, 2, 32, dtype=F32), **kw)[1],
    "evict": lambda **kw: ca.cart_pages_evict(
        *pools(), ints(3, 2), ints(3), ints(8), new(2, 3, 2, 32, dtype=F32), ints(3), **kw),
    "decode": lambda **kw: ca.cart_attn_decode_paged(
        new(3, 8, 64), new(3, 2, 64), new(3, 2, 64), new(5, 2, 64), new(5, 2, 64),
        new(8, 16, 2, 64), new(8, 16, 2, 64), ints(3, 2), ints(3),
        weights=new(3, 2, 32, dtype=F32), **kw),
}


def append(**kw):
    return ca.cart_pages_append(new(3, 4, 2, 64), new(3, 4, 2, 64), new(8, 16, 2, 64),
                                new(8, 16, 2, 64), ints(3, 2), ints(3), p=5, **kw)


@pytest.mark.parametrize("name", CALLS)
def test_calls_allocate_on_their_stream(fake, name):
    check(fake, CALLS[name])


def test_append_allocates_nothing(fake):
    append(stream=Stream(9))
    append()
    assert not fake.made and fake.now is fake.default


@pytest.mark.parametrize("name", [*CALLS, "append"])
def test_calls_refuse_a_stream_of_another_device(fake, name):
    other = Stream(9)
    other.device = Device()
    with pytest.raises(ValueError):
        (CALLS.get(name) or append)(stream=other)
    assert not fake.made and fake.now is fake.default
