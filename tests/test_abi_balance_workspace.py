"""The size of the balance loss's workspace, as a program that allocates once for its largest batch relies on it (host only)."""
import os

import pytest

from moe_expert_layer_amd import binding as B


@pytest.fixture(scope="module", autouse=True)
def library():
    if not os.path.exists(B.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()


def size(T, E, S):
    return B.moe_balance_workspace_size(B.make_balance_desc(T, E, 2, S))


@pytest.mark.parametrize("E,S", [(1, 1), (129, 24), (256, 1), (1024, 65536)])
def test_no_smaller_batch_needs_more(E, S):
    """A workspace for T tokens serves every smaller number: at the borders of the chunks' sizes (256 chunks of 32 tokens and more, up to
    8192) and around them."""
    at = list(range(0, 20000, 7)) + [256 * c + d for c in (4, 31, 32, 33, 64, 100, 4096, 8191, 8192, 8193, 16384) for d in range(-3, 4)]
    at += [1023, 1024, 1025, 1 << 24, (1 << 30) - (1 << 16)]
    sizes = [size(T, E, S) for T in sorted(at)]
    assert sizes == sorted(sizes)


def test_more_experts_or_sequences_need_no_less():
    for T in (1025, 8192, 8193, 100000):
        assert [size(T, E, 3) for E in range(1, 1025)] == sorted(size(T, E, 3) for E in range(1, 1025))
        s = [size(T, 60, S) for S in (1, 2, 3, 100, 65535, 65536)]
        assert s == sorted(s)


@pytest.mark.parametrize("T,E,S", [(0, 1, 1), (1, 1, 1), (1, 1024, 65536), (1024, 256, 1)])
def test_the_size_is_never_zero(T, E, S):
    """The call wants a workspace, so that what the size asks for has to be something that an allocator gives a pointer to."""
    n = size(T, E, S)
    assert n > 0 and n % 256 == 0
