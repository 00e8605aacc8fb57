"""GPU tests of the paged attention that see single positions: with keys of zeros every position seen
weighs the same, so an output counts positions, exactly, and a position lost, doubled or seen too many
where parts, tiles and waves meet shows in it."""

import math
import random

import pytest
import torch

from tests import block_ref as ref

pytestmark = pytest.mark.gpu

BF, FH = torch.bfloat16, torch.float16
DEV = "cuda"


@pytest.fixture(scope="module")
def block():
    from gemv_decode_projections_amd import block as b

    return b


def say(*a):
    print(*a, flush=True)


def marks(total, kv_heads, dim, code):
    """The element of every position's value that is not zero: positions in turn, or `dim` of them in turn."""
    p = torch.arange(total)[:, None] + 7 * torch.arange(kv_heads)
    return p % dim if code == 0 else p // dim % dim


def counting_batch(block, total, page, kv_heads, dim, dtype, code, seed):
    """Keys of zeros, values of 16 at one element; NaN in the rest of a sequence's last page."""
    need = [-(-t // page) for t in total]
    n_pages = sum(need) + 2
    order = random.Random(seed).sample(range(n_pages), n_pages)
    k = torch.full((n_pages, page, kv_heads, dim), math.nan, dtype=dtype, device=DEV)
    v = k.clone()
    table = torch.full((len(total), max(need)), -1, dtype=torch.int32)
    for b, t in enumerate(total):
        pages = [order.pop() for _ in range(need[b])]
        table[b, :need[b]] = torch.tensor(pages, dtype=torch.int32)
        at = torch.arange(t)
        where = (torch.tensor(pages, dtype=torch.long)[at // page].to(DEV), (at % page).to(DEV))
        k[where] = 0
        hot = torch.zeros(t, kv_heads, dim, dtype=dtype)
        hot.scatter_(2, marks(t, kv_heads, dim, code)[:, :, None], 16.0)
        v[where] = hot.to(DEV)
    return block.KvCache(k, v), table.to(DEV)


def check_counts(block, new, total, heads, kv_heads, dim, dtype, page=64, window=0, max_q=None, ws=None, codes=(0, 1)):
    """The weights are equal and exact, sums are whole numbers below 2^24, so an output is 16 count / n
    but for the division (2^-22) and its rounding to the type; lse is ln n but for one unit of a
    logarithm in base 2 of at most 32 (2^-19) and two roundings: 2^-18 in all."""
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    q_start = torch.tensor(start, dtype=torch.int32, device=DEV)
    kv_len = torch.tensor(total, dtype=torch.int32, device=DEV)
    ws = ws or block.AttnWorkspace(dim)
    gen = torch.Generator(DEV).manual_seed(len(new))
    for code in codes:
        cache, table = counting_batch(block, total, page, kv_heads, dim, dtype, code, 1)
        q = torch.randn(start[-1], heads, dim, generator=gen, device=DEV).to(dtype)
        out, lse = torch.full_like(q, math.nan), torch.full((start[-1], heads), math.nan, device=DEV)
        block.attn_run(q, cache, table, q_start, kv_len, out, ws, max_q=max_q or max(new), window=window, lse=lse)
        torch.cuda.synchronize()
        for b, (n, t) in enumerate(zip(new, total)):
            hot = marks(t, kv_heads, dim, code)
            rows, group = slice(start[b], start[b + 1]), heads // kv_heads
            hi = torch.arange(t - n + 1, t + 1)
            lo = (hi - window).clamp_min(0) if window else torch.zeros_like(hi)
            for h in range(kv_heads):
                before = torch.zeros(t + 1, dim, dtype=torch.int32)
                before[1:].scatter_(1, hot[:, h, None], 1)
                before = before.cumsum(0, dtype=torch.int32)
                want = (16.0 * (before[hi] - before[lo]).double() / (hi - lo)[:, None].double())
                for g in range(h * group, (h + 1) * group):
                    what = "code %d sequence %d head %d" % (code, b, g)
                    ref.assert_within("out " + what, out[rows, g], want,
                                      (ref.U[dtype] + 2.0 ** -22) * want + ref.TINY[dtype] * (want > 0) + 1e-300)
                    ref.assert_within("lse " + what, lse[rows, g], torch.log((hi - lo).double()),
                                      torch.full(hi.shape, 2.0 ** -18, dtype=torch.float64))
    return ws


# new tokens, positions, heads, kv_heads, dim, type, page, window
SEAMS = [
    ([1], [30000], 8, 1, 128, FH, 64, 0), ([1], [30001], 4, 1, 64, FH, 8, 0), ([1], [29999], 8, 1, 256, FH, 16, 0),
    ([1], [20033], 8, 1, 128, FH, 16, 9000), ([1, 1, 1], [25000, 31, 129], 4, 2, 128, FH, 64, 0),
    ([3], [30000], 8, 1, 128, FH, 32, 0), ([2, 3], [18000, 7001], 8, 1, 64, FH, 64, 3001), ([3], [9000], 8, 1, 256, FH, 64, 0),
    ([8], [30000], 8, 1, 128, FH, 64, 0), ([12], [15000], 4, 1, 64, FH, 8, 2999), ([24], [12000], 2, 1, 256, FH, 16, 0),
    ([40], [20000], 4, 1, 64, FH, 64, 0), ([300], [9000], 2, 1, 128, FH, 16, 2500), ([90], [10000], 2, 1, 256, FH, 8, 1000),
    ([130, 70], [6000, 70], 4, 2, 128, BF, 64, 0), ([1], [12000], 8, 1, 128, BF, 64, 0), ([200], [200], 4, 1, 128, BF, 16, 65),
    ([1, 2, 1], [700, 640, 64], 16, 2, 64, BF, 8, 63), ([5], [4097], 6, 1, 128, BF, 128, 1),
]


@pytest.mark.parametrize("case", range(len(SEAMS)))
def test_every_position_counts_once(block, case):
    new, total, heads, kv_heads, dim, dtype, page, window = SEAMS[case]
    say("seams", SEAMS[case])
    check_counts(block, new, total, heads, kv_heads, dim, dtype, page, window)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("max_q", [1, 3, 8, 64])
def test_every_kernel_counts_a_mixed_batch(block, dim, max_q):
    # max_q picks the kernel (16, 32, 64 and 128 rows per tile); any batch is right in each.
    say("seams mixed", dim, max_q)
    check_counts(block, [1, 17, 4], [9001, 3000, 640], 8, 1, dim, FH, 32, 0, max_q)


@pytest.mark.parametrize("new,total,heads,kv_heads,dim", [([1, 1], [164000, 2000], 8, 1, 128), ([1], [164000], 4, 2, 64)])
def test_a_split_alone_at_its_level_touches_no_other_tile(block, new, total, heads, kv_heads, dim):
    # 257 splits: the last one has no partner in the first two levels of joins. The counters of the
    # tile behind it are that tile's alone, and all are zero again afterwards.
    say("seams 257", new, total, heads, kv_heads, dim)
    ws = block.AttnWorkspace(dim)
    for _ in range(3):
        check_counts(block, new, total, heads, kv_heads, dim, FH, 64, ws=ws, codes=(1,))
        assert not bool(ws.buffer[:block.ATTN_ZEROED].any())


@pytest.mark.parametrize("max_q,heads", [(2, 8), (1, 4), (3, 8), (8, 8), (40, 4)])
@pytest.mark.parametrize("seqs", [6, 130])
def test_offsets_that_descend_leave_the_workspace_usable(block, seqs, max_q, heads):
    # Sequences that would overlap: more rows than there are tokens. Every counter of the workspace is
    # zero again, rows are written whole or not at all, and a valid batch on it is right.
    say("descending offsets", seqs, max_q, heads)
    tokens, dim = 16, 128
    total = [1000 + 13 * (b % 7) for b in range(seqs)]
    cache, table = counting_batch(block, total, 64, 1, dim, BF, 0, 2)
    kv_len = torch.tensor(total, dtype=torch.int32, device=DEV)
    ws = block.AttnWorkspace(dim)
    q = torch.randn(tokens, heads, dim, device=DEV).to(BF)
    rng = random.Random(seqs)
    for start in ([0, tokens] * seqs, [tokens, 0] * seqs, [rng.randint(-3, tokens + 3) for _ in range(seqs + 1)],
                  [7, 2 ** 31 - 1, -(2 ** 31)] * seqs):
        q_start = torch.tensor(start[:seqs + 1], dtype=torch.int32, device=DEV)
        out = torch.full_like(q, math.nan)
        block.attn_run(q, cache, table, q_start, kv_len, out, ws, max_q=max_q)
        torch.cuda.synchronize()
        assert not bool(ws.buffer[:block.ATTN_ZEROED].any())
        gone = torch.isnan(out).all(-1)
        assert bool((torch.isnan(out).any(-1) == gone).all())
    check_counts(block, [max_q, 1], [9000, 300], heads, 1, dim, FH, 64, ws=ws)
