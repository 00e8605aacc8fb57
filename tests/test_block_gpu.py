"""GPU tests of the decode-block operators against the 64-bit references of block_ref."""

import math
import random

import pytest
import torch

from tests import block_ref as ref

pytestmark = pytest.mark.gpu

BF, FH, F32 = torch.bfloat16, torch.float16, torch.float32
DEV = "cuda"


@pytest.fixture(scope="module")
def block():
    from gemv_decode_projections_amd import block as b

    return b


def say(*a):
    print(*a, flush=True)


def make_batch(block, new, cached, page, kv_heads, dim, dtype=BF, seed=0, layout="token", spare=3, extra_columns=0):
    """A cache holding NaN wherever no token of the batch lies, its page table (shuffled pages, junk
    behind each sequence's last page) and lengths."""
    rng = random.Random(seed)
    gen = torch.Generator().manual_seed(seed)
    total = [n + c for n, c in zip(new, cached)]
    need = [-(-t // page) for t in total]
    n_pages = sum(need) + spare
    order = rng.sample(range(n_pages), n_pages)
    width = max(max(need), 1) + extra_columns
    table = torch.full((len(new), width), 2 ** 31 - 1, dtype=torch.int32)
    if layout == "token":
        kv = torch.full((2, n_pages, page, kv_heads, dim), math.nan, dtype=dtype)
        k, v = kv[0], kv[1]
    elif layout == "head":              # head-major pages
        kv = torch.full((2, n_pages, kv_heads, page, dim), math.nan, dtype=dtype)
        k, v = kv[0].transpose(1, 2), kv[1].transpose(1, 2)
    else:                               # keys and values of a page next to each other
        kv = torch.full((n_pages, 2, page, kv_heads, dim), math.nan, dtype=dtype)
        k, v = kv[:, 0], kv[:, 1]
    at = 0
    for b, t in enumerate(total):
        for j in range(need[b]):
            table[b, j] = order[at]
            held = min(page, t - j * page)
            k[order[at], :held] = torch.randn(held, kv_heads, dim, generator=gen).to(dtype)
            v[order[at], :held] = torch.randn(held, kv_heads, dim, generator=gen).to(dtype)
            at += 1
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    kd = kv.to(DEV)
    if layout == "token":
        k, v = kd[0], kd[1]
    elif layout == "head":
        k, v = kd[0].transpose(1, 2), kd[1].transpose(1, 2)
    else:
        k, v = kd[:, 0], kd[:, 1]
    return (block.KvCache(k, v), table.to(DEV), torch.tensor(start, dtype=torch.int32, device=DEV),
            torch.tensor(total, dtype=torch.int32, device=DEV), gen)


def run_attn(block, cache, table, q_start, kv_len, q, ws=None, **kw):
    out = torch.full_like(q, math.nan)
    lse = torch.full(q.shape[:2], math.nan, device=DEV)
    block.attn_run(q, cache, table, q_start, kv_len, out, ws or block.AttnWorkspace(cache.head_dim), lse=lse, **kw)
    torch.cuda.synchronize()
    return out, lse


def check_attn(block, cache, table, q_start, kv_len, gen, heads, window=0, gate=False, max_q=None, what=""):
    tokens = int(q_start[-1])
    q = (1.5 * torch.randn(tokens, heads, cache.head_dim, generator=gen)).to(cache.dtype).to(DEV)
    g = torch.randn(tokens, heads, cache.head_dim, generator=gen).to(cache.dtype).to(DEV) if gate else None
    scale = cache.head_dim ** -0.5
    out, lse = run_attn(block, cache, table, q_start, kv_len, q, window=window, gate=g, max_q=max_q)
    ro, rl, bo, bl = ref.attention(q, cache.k, cache.v, table, q_start, kv_len, scale, window, g)
    ref.assert_within("out " + what, out, ro, bo)
    ref.assert_within("lse " + what, lse, rl, bl)
    return out


# (new tokens, cached tokens) per sequence, heads, kv_heads, head_dim, page, dtype, window, gate, layout
ATTN = [
    ([1], [0], 1, 1, 64, 8, BF, 0, False, "token"),
    ([1], [37], 8, 1, 128, 16, BF, 0, True, "token"),
    ([1, 1, 1], [127, 128, 129], 8, 2, 128, 16, FH, 0, False, "head"),
    ([1] * 5, [0, 31, 32, 33, 700], 10, 2, 64, 8, BF, 0, False, "pair"),
    ([1, 1], [515, 64], 7, 1, 256, 32, BF, 0, True, "token"),
    ([1], [3000], 16, 4, 128, 64, BF, 0, False, "token"),
    ([8, 8], [100, 251], 8, 1, 128, 16, BF, 0, True, "token"),
    ([3, 0, 5], [40, 10, 0], 4, 2, 64, 8, FH, 0, False, "token"),
    ([5, 17], [0, 300], 6, 3, 256, 16, FH, 0, False, "head"),
    ([33], [95], 5, 5, 128, 128, BF, 0, False, "token"),
    ([64, 1, 13], [0, 222, 5], 8, 2, 128, 16, BF, 0, False, "pair"),
    ([130], [77], 4, 1, 64, 16, FH, 0, True, "token"),
    ([70, 9], [33, 64], 2, 1, 256, 8, BF, 0, False, "token"),
    ([1, 1], [300, 20], 8, 2, 128, 16, BF, 48, False, "token"),
    ([9, 40], [200, 3], 8, 2, 128, 16, BF, 21, True, "token"),
    ([100], [150], 4, 2, 64, 32, FH, 1, False, "token"),
    ([48], [500], 8, 1, 128, 16, BF, 130, False, "head"),
]


@pytest.mark.parametrize("case", range(len(ATTN)))
def test_attention(block, case):
    new, cached, heads, kv_heads, dim, page, dtype, window, gate, layout = ATTN[case]
    say("attn", ATTN[case])
    cache, table, q_start, kv_len, gen = make_batch(block, new, cached, page, kv_heads, dim, dtype, case, layout)
    check_attn(block, cache, table, q_start, kv_len, gen, heads, window, gate, max(new))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("max_q", [1, 3, 200])
def test_attention_result_does_not_need_max_q(block, dim, max_q):
    # max_q picks the kernel; every kernel takes any batch.
    say("attn max_q", dim, max_q)
    cache, table, q_start, kv_len, gen = make_batch(block, [1, 21, 2], [90, 64, 0], 16, 2, dim, BF, 5)
    check_attn(block, cache, table, q_start, kv_len, gen, 6, max_q=max_q, what="max_q %d" % max_q)
