"""Host checks of lengths near the end of 32 bits (no GPU work is done)."""
import ctypes

import pytest

from tests.test_kv8_host import APPEND, APPEND_OK, COMMIT, COMMIT_OK, L, SHAPE, TREE, TREE_OK, _call  # noqa: F401

INT_MAX = 2 ** 31 - 1


@pytest.mark.parametrize("Lmax", [INT_MAX, INT_MAX - 30, INT_MAX - 126])
def test_caches_whose_last_tile_passes_32_bits_are_refused(L, Lmax):  # noqa: F811
    assert _call(L.eagle_kv8_append, APPEND, APPEND_OK, Lmax=Lmax) == SHAPE
    assert _call(L.eagle_kv8_commit, COMMIT, COMMIT_OK, Lmax=Lmax) == SHAPE
    assert _call(L.eagle_tree_attn_kv8, TREE, TREE_OK, Lmax=Lmax) == SHAPE
    assert L.eagle_tree_attn_kv8_workspace_size(1, 1, 1, 1, 128, Lmax) == 0


def test_workspace_of_the_longest_caches_is_that_of_the_whole_card(L):  # noqa: F811
    size = L.eagle_tree_attn_kv8_workspace_size
    assert isinstance(size(1, 1, 1, 1, 128, 1 << 20), int) and size.restype is ctypes.c_size_t
    assert size(1, 1, 1, 1, 128, INT_MAX - 127) == size(1, 1, 1, 1, 128, 1 << 20) > 0
