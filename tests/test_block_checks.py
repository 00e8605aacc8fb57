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


def test_the_stride_of_a_single_entry_is_not_looked_at(block, lib):  # noqa: F811
    # (no GPU: a call that passes its checks goes on to the null pointers)
    from tests.test_block import NULL, Attn, Norm

    vp, ref_ = ctypes.c_void_p, ctypes.byref
    one = changed(some_cache(block), n_pages=1, kv_heads=1, page_stride=-3, head_stride=5)
    batch = Batch(P, P, P, 4, 4, 2, 1)
    for c, want in [(one, NULL), (changed(one, n_pages=2), ARG), (changed(one, kv_heads=2), ARG)]:
        assert lib.blk_kv_append(ref_(c), ref_(batch), None, None, ctypes.c_int64(3), ctypes.c_int64(5), vp(0)) == want
    two = changed(batch, tokens=2)
    assert lib.blk_kv_append(ref_(one), ref_(two), None, None, ctypes.c_int64(3), ctypes.c_int64(5), vp(0)) == ARG
    args = Attn(0, 0, 0, 0, 65, 7, 3, -1, 1, 9, 1, 1, 0, 0.125)
    attn = lambda a, b: lib.blk_attn_run(ref_(one), ref_(b), ref_(a), vp(P), ctypes.c_size_t(1 << 40), vp(0))  # noqa: E731
    assert attn(args, batch) == NULL and attn(args, two) == ARG and attn(changed(args, heads=2), batch) == ARG
    w = block._W4(64, 256, 128, 0, 0)
    run = lambda m, xs, os: lib.blk_w4_run(ref_(w), None, None, ctypes.c_int64(xs), m, None, ctypes.c_int64(os), None)  # noqa: E731
    assert run(1, 13, -1) == NULL and run(2, 13, 64) == ARG and run(2, 256, -1) == ARG
    n = Norm(0, 0, 0, 0, 0, 0, 0, -1, 3, -5, -7, 1 << 41, 64, 0, 2, 1.0, 1e-6)
    assert lib.blk_norm_run(ref_(n), 1, None) == NULL and lib.blk_norm_run(ref_(n), 2, None) == ARG


def test_outputs_that_overlap_themselves_are_refused(block, lib):  # noqa: F811
    # (no GPU: a call that passes its checks goes on to the null pointers)
    from tests.test_block import NULL, Attn, Norm

    vp, ref_ = ctypes.c_void_p, ctypes.byref
    cache = some_cache(block)
    batch = Batch(P, P, P, 4, 4, 2, 3)
    args = Attn(0, 0, 0, 0, 0, 0, 0, 0, 256, 64, 4, 1, 0, 0.125)
    attn = lambda **kw: lib.blk_attn_run(ref_(cache), ref_(batch), ref_(changed(args, **kw)), vp(P),  # noqa: E731
                                         ctypes.c_size_t(1 << 40), vp(0))
    assert attn() == NULL
    for kw in (dict(out_stride=64, out_head_stride=192), dict(out_stride=1000), dict(out_head_stride=80, out_stride=304)):
        assert attn(**kw) == NULL, kw                       # apart, in either order
    for kw in (dict(out_stride=0), dict(out_head_stride=0), dict(out_stride=248), dict(out_head_stride=56),
               dict(out_stride=64), dict(out_stride=64, out_head_stride=184)):
        assert attn(**kw) == ARG, kw
    # keys and values: read through any strides, written only where every place is one
    none = lambda **kw: lib.blk_kv_append(ref_(changed(cache, **kw)), ref_(batch), None, None, ctypes.c_int64(128),  # noqa: E731
                                          ctypes.c_int64(64), vp(0))
    assert none() == NULL and none(token_stride=64, head_stride=1024) == NULL and none(page_stride=4096) == NULL
    for kw in (dict(page_stride=0), dict(head_stride=0), dict(token_stride=64), dict(page_stride=2040)):
        assert none(**kw) == ARG, kw
    shared = Attn(0, 0, 0, 0, 0, 0, 0, 0, 256, 64, 4, 1, 0, 0.125)
    assert lib.blk_attn_run(ref_(changed(cache, head_stride=0)), ref_(batch), ref_(shared), vp(P), ctypes.c_size_t(1 << 40),
                            vp(0)) == NULL
    w = block._W4(64, 256, 128, 0, 0)
    run = lambda m, os: lib.blk_w4_run(ref_(w), None, None, ctypes.c_int64(0), m, None, ctypes.c_int64(os), None)  # noqa: E731
    assert run(2, 64) == NULL and run(2, 63) == ARG and run(2, 0) == ARG and run(1, 0) == NULL
    n = Norm(P, P, 0, 0, P, P, 0, 0, 0, 0, 64, 64, 64, 0, 2, 1.0, 1e-6)
    norm = lambda m, **kw: lib.blk_norm_run(ref_(changed(n, **kw)), m, None)  # noqa: E731
    assert norm(2) == NULL and norm(2, os=63) == ARG and norm(2, ys=0) == ARG and norm(1, os=0, ys=0) == NULL
    assert norm(2, x=0, residual_out=0, ys=0) == NULL


def test_page_numbers_past_32_bits_are_refused(block):  # noqa: F811
    # 2^32 + 1 is not page 1.
    pool = block.PagePool(6)
    pages = pool.alloc(3)
    for bad in ([2 ** 32 + 1], [0, 2 ** 31], [-2 ** 31 - 1], [1.0], ["1"], [None]):
        with pytest.raises(ValueError):
            pool.free(bad)
        with pytest.raises(ValueError):
            pool.fork(bad)
    for call in (lambda: pool.users(2 ** 32 + 1), lambda: pool.alloc(2 ** 32 + 1), lambda: pool.compact(2 ** 32 + 1),
                 lambda: pool.writable([2 ** 32 + 1], 0), lambda: block.PagePool(2 ** 32 + 1), lambda: pool.alloc(1.5)):
        with pytest.raises(ValueError):
            call()
    assert [pool.users(p) for p in range(6)] == [1, 1, 1, 0, 0, 0] and pool.free_pages == 3
    pool.free(pages)
    assert pool.free_pages == 6 and pool.fork([]) == [] and pool.free(()) is None


def test_a_fork_in_a_large_cache_costs_what_it_copies(block):  # noqa: F811
    # The check of the pairs must not take memory by the cache's size: two pairs, 2^31 - 1 pages. In a
    # process of its own, whose peak memory says so.
    import os
    import subprocess
    import sys

    program = """
import ctypes, resource
from gemv_decode_projections_amd import block
lib = block._lib()
cache = block._Cache(4096, 4096, 16 * 64, 64, 64, 2 ** 31 - 1, 16, 1, 64, 0)
pages = ctypes.c_int32 * 2
peak = lambda: resource.getrusage(resource.RUSAGE_SELF).ru_maxrss
before = peak()
for s, d in [((0, 2 ** 31 - 3), (5, 5)), ((0, 2 ** 31 - 2), (2 ** 31 - 2, 9)), ((0, 1), (2 ** 31 - 1, 9))]:
    assert lib.blk_kv_copy_pages(ctypes.byref(cache), pages(*s), pages(*d), 2, None) == -10
print(peak() - before)
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", program], cwd=root, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    assert int(r.stdout) < 64 * 1024, r.stdout        # KB


def test_page_pairs_against_a_plain_check(block, lib):  # noqa: F811
    # Pairs that must be refused are (no GPU: accepted ones fail in the launch, which is another status).
    import random

    import torch

    if torch.cuda.is_available():
        pytest.skip("would launch copies at made-up addresses")
    rng = random.Random(4)
    for pages in (3, 40, 70000, 2 ** 31 - 1):
        cache = block._Cache(P, P, 16 * 64, 64, 64, pages, 16, 1, 64, 0)
        for _ in range(300):
            n = rng.randint(1, 40)
            near = rng.choice([pages, min(pages, 2 * n + 2)])
            src, dst = ([rng.randrange(near) for _ in range(n)] for _ in range(2))
            bad = len(set(dst)) < n or set(src) & set(dst)
            a = (ctypes.c_int32 * n)
            rc = lib.blk_kv_copy_pages(ctypes.byref(cache), a(*src), a(*dst), n, ctypes.c_void_p(0))
            assert (rc == ARG) == bool(bad), (pages, src, dst, rc)
