"""Host checks of the block operators' C entries and page pool (CPU only), where a value is at the edge of
what an operator takes."""

import ctypes

import pytest

from tests.test_block import ARG, OK, Batch, block, changed, lib  # noqa: F401  (fixtures)

P = 4096


def append(lib, cache, batch, s=128, h=64):  # noqa: F811
    return lib.blk_kv_append(ctypes.byref(cache), ctypes.byref(batch), ctypes.c_void_p(P), ctypes.c_void_p(P),
                             ctypes.c_int64(s), ctypes.c_int64(h), ctypes.c_void_p(0))


def some_cache(block):  # noqa: F811
    return block._Cache(P, P, 16 * 2 * 64, 2 * 64, 64, 8, 16, 2, 64, 0)


@pytest.mark.parametrize("stride,want", [(0, OK), (1, ARG), (3, ARG), (4, OK), (9, OK), (-1, ARG), (-4, ARG)])
def test_table_rows_are_one_or_do_not_overlap(block, lib, stride, want):  # noqa: F811
    assert append(lib, some_cache(block), Batch(P, P, P, stride, 4, 2, 0)) == want
