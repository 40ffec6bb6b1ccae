"""Numbers that do not fit the library's 32 bits, on the CPU: ctypes would pass
their low 32 bits on."""
import pytest
import torch

from trained_kv_prefix_gb300 import cartattn as ca

BF, I32 = torch.bfloat16, torch.int32
WRAPS = 1 << 32


def ints(*shape):
    return torch.zeros(shape, dtype=I32)


def pool(*shape):
    return torch.zeros(shape, dtype=BF)


def wide(*shape):
    """An int32 tensor of that shape without the memory."""
    return ints(1).expand(shape)


@pytest.mark.parametrize("window", [WRAPS, WRAPS + 5, 1 << 31, -(1 << 31) - 1])
def test_tree_refuses_a_window_beyond_32_bits(window):
    new = pool(2, 3, 2, 64)
    with pytest.raises(ValueError, match="window"):
        ca.cart_attn_decode_tree(pool(2, 3, 4, 64), new, new, pool(5, 2, 64), pool(5, 2, 64),
                                 pool(4, 16, 2, 64), pool(4, 16, 2, 64), ints(2, 2), ints(2),
                                 window=window)


@pytest.mark.parametrize("rows", [WRAPS + 16, WRAPS + 128, (1 << 31) + 16])
def test_fork_refuses_a_page_size_beyond_32_bits(rows):
    with pytest.raises(ValueError, match="page_rows"):
        ca.cart_pages_fork(ints(2, 2), ints(2), ints(4), ints(1), ints(1), page_rows=rows)


def test_accept_refuses_a_chain_beyond_32_bits():
    with pytest.raises(ValueError, match="nodes"):
        ca.cart_pages_accept(pool(1, 4, 16, 2, 64), pool(1, 4, 16, 2, 64), ints(2, 2), ints(2),
                             WRAPS + 4, ints(2))


def test_tables_beyond_32_bits_are_refused():
    k = pool(1, 4, 16, 2, 64)
    table, many = wide(1, WRAPS + 2), wide(WRAPS + 2)
    with pytest.raises(ValueError, match="max_pages"):
        ca.cart_pages_reserve(k, k, table, ints(1), ints(4), ints(1))
    with pytest.raises(ValueError, match="max_pages"):
        ca.cart_pages_compact(k, k, table, ints(4))
    with pytest.raises(ValueError, match="max_pages"):
        ca.cart_pages_accept(k, k, table, ints(1), 1, ints(1))
    with pytest.raises(ValueError, match="pages"):
        ca.cart_pages_fork(ints(1, 2), ints(1), many, ints(1), ints(1), page_rows=16)
    with pytest.raises(ValueError, match="forks"):
        ca.cart_pages_fork(ints(1, 2), ints(1), ints(4), many, many, page_rows=16)


def test_numbers_that_fit_are_left_to_the_library():
    ca._fits(window=(1 << 31) - 1, pages=-(1 << 31), zero=0)
    with pytest.raises(ValueError, match="pages: 2147483648"):
        ca._fits(window=0, pages=1 << 31)
