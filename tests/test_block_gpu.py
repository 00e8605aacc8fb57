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


@pytest.mark.parametrize("new,max_q", [([1, 1, 3], 3), ([9, 40, 70], 70)])
@pytest.mark.parametrize("window", [0, 40])
def test_unmapped_pages_hold_no_tokens(block, new, max_q, window):
    say("attn holes", new, window)
    cached = [100, 70, 0]
    cache, table, q_start, kv_len, gen = make_batch(block, new, cached, 8, 2, 128, BF, 7)
    for b in range(3):
        for j in range(0, (new[b] + cached[b] + 7) // 8, 3):
            table[b, j] = [-1, 2 ** 31 - 1, cache.n_pages][j // 3 % 3]
    table[2] = -1                          # nothing mapped at all: empty rows
    check_attn(block, cache, table, q_start, kv_len, gen, 8, window, max_q=max_q)


@pytest.mark.parametrize("max_q", [1, 40])
def test_rows_that_see_nothing(block, max_q):
    # More new tokens than positions: the first ones stand before position 0. Lengths and offsets
    # outside the tensors are bounded.
    say("attn empty rows", max_q)
    cache, table, q_start, kv_len, gen = make_batch(block, [40, 3, 5], [0, 0, 30], 16, 2, 64, BF, 3)
    kv_len.copy_(torch.tensor([11, 0, 35], dtype=torch.int32))
    out = check_attn(block, cache, table, q_start, kv_len, gen, 4, max_q=max_q)
    assert bool((out[:29] == 0).all()) and bool((out[40:43] == 0).all())
    q = torch.randn(48, 4, 64, generator=gen).to(BF).to(DEV)
    kv_len.copy_(torch.tensor([-5, -(2 ** 31), 2 ** 31 - 1], dtype=torch.int32))
    got, lse = run_attn(block, cache, table, q_start, kv_len, q, max_q=max_q)
    assert bool((got[:43] == 0).all()) and bool((lse[:43] == -math.inf).all())
    rows = [0, 48, 48, 48]                  # one sequence of all tokens, then empty ones
    q_start.copy_(torch.tensor(rows, dtype=torch.int32))
    kv_len.copy_(torch.tensor([33, 5, 0], dtype=torch.int32))
    check_attn(block, cache, table, q_start, kv_len, gen, 4, max_q=max_q)


@pytest.mark.parametrize("dtype", [BF, FH])
@pytest.mark.parametrize("new,heads,dim", [([12], 2, 128), ([2], 8, 64), ([100], 4, 128), ([70], 2, 256), ([90], 1, 64)])
def test_infinities_in_masked_places(block, dtype, new, heads, dim):
    # Tokens that come later hold infinities and NaN; rows before them must not notice, rows that
    # see them get what the definition gives.
    say("attn inf", dtype, new, heads, dim)
    n = new[0]
    cache, table, q_start, kv_len, gen = make_batch(block, new, [45], 8, 1, dim, dtype, 11)
    bad = [45 + n - 1, 45 + n // 2, 45 + n // 2 - 1]
    for i, p in enumerate(bad):
        page, at = int(table[0, p // 8]), p % 8
        cache.v[page, at, 0, 3 + i] = [math.inf, -math.inf, math.nan][i]
        cache.v[page, at, 0, dim - 1 - i] = [math.nan, math.inf, math.inf][i]
    page, at = int(table[0, bad[0] // 8]), bad[0] % 8
    # (even weights: none so small that its type makes it zero)
    q = (0.2 * torch.randn(n, heads, dim, generator=gen)).to(dtype).to(DEV)
    out, lse = run_attn(block, cache, table, q_start, kv_len, q, max_q=n)
    ro, rl, bo, bl = ref.attention(q, cache.k, cache.v, table, q_start, kv_len, dim ** -0.5)
    ref.assert_within("out", out, ro, bo)
    ref.assert_within("lse", lse, rl, bl)
    cache.k[page, at, 0, 5] = math.nan      # the last token's key: only its own row may turn NaN
    out, lse = run_attn(block, cache, table, q_start, kv_len, q, max_q=n)
    assert bool(torch.isnan(lse[n - 1]).all()) and bool(torch.isfinite(lse[:n - 1]).all())
    assert bool(torch.isnan(out[n - 1]).all())


def test_no_tokens(block):
    cache = block.KvCache.empty(4, 8, 2, 64)
    ws = block.AttnWorkspace(64)
    z = torch.zeros(0, dtype=torch.int32, device=DEV)
    one = torch.zeros(1, dtype=torch.int32, device=DEV)
    q = torch.empty(0, 4, 64, dtype=BF, device=DEV)
    kv = torch.empty(0, 2, 64, dtype=BF, device=DEV)
    table0 = torch.zeros(0, 3, dtype=torch.int32, device=DEV)
    block.attn_run(q, cache, table0, one, z, torch.empty_like(q), ws)
    block.kv_append(kv, kv, cache, table0, one, z)
    table1 = torch.zeros(1, 3, dtype=torch.int32, device=DEV)
    two = torch.zeros(2, dtype=torch.int32, device=DEV)
    block.attn_run(q, cache, table1, two, one, torch.empty_like(q), ws)
    block.kv_append(kv, kv, cache, table1, two, one)
    block.kv_copy_pages(cache, [], [])
    torch.cuda.synchronize()


@pytest.mark.parametrize("max_q", [1, 30])
def test_many_sequences(block, max_q):
    # More sequences than lanes of a wave, some without new tokens, some of one page.
    rng = random.Random(5)
    new = [rng.choice([0, 1, 1, 2]) for _ in range(150)]
    cached = [rng.choice([0, 5, 63, 64, 200]) for _ in range(150)]
    say("attn many", max_q)
    cache, table, q_start, kv_len, gen = make_batch(block, new, cached, 8, 1, 64, BF, 9, extra_columns=2)
    check_attn(block, cache, table, q_start, kv_len, gen, 4, max_q=max_q)


@pytest.mark.parametrize("new,heads,dim,window", [([1], 2, 64, 0), ([1], 8, 128, 0), ([3], 8, 128, 0), ([8], 8, 128, 0),
                                                  ([40], 4, 64, 0), ([24], 8, 256, 0), ([1], 4, 128, 9000),
                                                  ([12], 2, 64, 3000), ([300], 2, 128, 2500), ([90], 1, 256, 1000)])
def test_long_contexts_are_split_and_joined(block, new, heads, dim, window):
    say("attn long", new, heads, dim)
    cache, table, q_start, kv_len, gen = make_batch(block, new, [30000], 64, 1, dim, BF, 2)
    check_attn(block, cache, table, q_start, kv_len, gen, heads, window, max_q=new[0])


def test_offsets_past_32_bits(block):
    # Pages beyond 4 GiB in both tensors, appended to, copied and read.
    say("attn large cache")
    page, heads, dim = 64, 8, 256
    n_pages = (5 << 30) // (page * heads * dim * 2)
    cache = block.KvCache.empty(n_pages, page, heads, dim)
    gen = torch.Generator().manual_seed(4)
    pages = [n_pages - 1, 3, n_pages - 2]
    table = torch.tensor([pages], dtype=torch.int32, device=DEV)
    n = 150
    k, v = (torch.randn(n, heads, dim, generator=gen).to(BF).to(DEV) for _ in range(2))
    q_start = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    kv_len = torch.tensor([n], dtype=torch.int32, device=DEV)
    block.kv_append(k, v, cache, table, q_start, kv_len)
    torch.cuda.synchronize()
    for p in range(0, n, 7):
        assert torch.equal(cache.k[pages[p // page], p % page], k[p]) and torch.equal(cache.v[pages[p // page], p % page], v[p])
    block.kv_copy_pages(cache, [n_pages - 1, 3], [n_pages - 5, n_pages - 4])
    table = torch.tensor([[n_pages - 5, n_pages - 4, n_pages - 2]], dtype=torch.int32, device=DEV)
    for m in (1, 5, 20):
        q_start = torch.tensor([0, m], dtype=torch.int32, device=DEV)
        check_attn(block, cache, table, q_start, kv_len, gen, 8, max_q=m)


def fused_case(block, seed):
    """q, k, v and gate as slices of one projection's output; out as a slice of a wider tensor."""
    heads, kv_heads, dim, n = 8, 1, 128, 21
    cache, table, q_start, kv_len, gen = make_batch(block, [n, 3], [50, 130], 16, kv_heads, dim, BF, seed)
    wide = torch.randn(n + 3, 2304, generator=gen).to(BF).to(DEV)
    q, k, v, gate = wide.split([heads * dim, dim, dim, heads * dim], 1)
    tokens = n + 3
    return (cache, table, q_start, kv_len, q.view(tokens, heads, dim), k.view(tokens, 1, dim), v.view(tokens, 1, dim),
            gate.view(tokens, heads, dim))


@pytest.mark.parametrize("max_q", [2, 21])
def test_append_and_attention_on_views_of_one_projection(block, max_q):
    say("fused", max_q)
    cache, table, q_start, kv_len, q, k, v, gate = fused_case(block, 6)
    before_k, before_v = cache.k.clone(), cache.v.clone()
    block.kv_append(k, v, cache, table, q_start, kv_len)
    torch.cuda.synchronize()
    for b, (s, n, length) in enumerate([(0, 21, 71), (21, 3, 133)]):
        for i in range(n):
            p = length - n + i
            before_k[int(table[b, p // 16]), p % 16] = k[s + i]
            before_v[int(table[b, p // 16]), p % 16] = v[s + i]
    assert torch.equal(before_k.view(torch.int16), cache.k.view(torch.int16))
    assert torch.equal(before_v.view(torch.int16), cache.v.view(torch.int16))
    big = torch.full((24, 8, 200), 7.0, dtype=BF, device=DEV)
    out = big[:, :, 40:168]
    block.attn_run(q, cache, table, q_start, kv_len, out, block.AttnWorkspace(128), max_q=max_q, gate=gate)
    torch.cuda.synchronize()
    ro, _, bo, _ = ref.attention(q, cache.k, cache.v, table, q_start, kv_len, 128 ** -0.5, 0, gate)
    ref.assert_within("out", out, ro, bo)
    assert bool((big[:, :, :40] == 7).all()) and bool((big[:, :, 168:] == 7).all())


def test_append_skips_what_has_no_place(block):
    say("append skips")
    cache, table, q_start, kv_len, gen = make_batch(block, [6, 0, 9], [0, 12, 20], 8, 2, 64, FH, 8)
    kv_len.copy_(torch.tensor([4, 12, 29], dtype=torch.int32))     # two tokens before position 0
    table[2, 3] = -1                                               # the page of positions 24..28
    k, v = (torch.randn(15, 2, 64, generator=gen).to(FH).to(DEV) for _ in range(2))
    want_k, want_v = cache.k.clone(), cache.v.clone()
    for i in range(2, 6):
        want_k[int(table[0, 0]), i - 2], want_v[int(table[0, 0]), i - 2] = k[i], v[i]
    for i in range(4):
        want_k[int(table[2, 2]), 4 + i], want_v[int(table[2, 2]), 4 + i] = k[6 + i], v[6 + i]
    block.kv_append(k, v, cache, table, q_start, kv_len)
    torch.cuda.synchronize()
    assert torch.equal(want_k.view(torch.int16), cache.k.view(torch.int16))
    assert torch.equal(want_v.view(torch.int16), cache.v.view(torch.int16))


@pytest.mark.parametrize("layout", ["token", "head", "pair"])
@pytest.mark.parametrize("pages,page,heads,dim,moves", [(40, 16, 3, 128, 9), (70000, 8, 1, 64, 1200), (3000, 8, 1, 64, 1000)])
def test_copy_pages(block, layout, pages, page, heads, dim, moves):
    say("copy", layout, pages)
    if layout == "token":
        kv = torch.randn(2, pages, page, heads, dim, device=DEV).to(BF)
        k, v = kv[0], kv[1]
    elif layout == "head":
        kv = torch.randn(2, pages, heads, page, dim, device=DEV).to(BF)
        k, v = kv[0].transpose(1, 2), kv[1].transpose(1, 2)
    else:
        kv = torch.randn(pages, 2, page, heads, dim, device=DEV).to(BF)
        k, v = kv[:, 0], kv[:, 1]
    order = random.Random(1).sample(range(pages), 2 * moves)
    src, dst = order[:moves], order[moves:]
    src[1] = src[0]                        # one page may be copied to several
    wk, wv = k.clone(), v.clone()
    d, s = torch.tensor(dst, device=DEV), torch.tensor(src, device=DEV)
    wk[d], wv[d] = wk[s], wv[s]
    block.kv_copy_pages(block.KvCache(k, v), src, dst)
    torch.cuda.synchronize()
    assert torch.equal(wk, k) and torch.equal(wv, v)


def test_fork_write_and_compact_keep_what_sequences_read(block):
    # Two sequences share a prefix, one is given a page of its own and goes on, the other is freed,
    # the cache is compacted: attention over the survivor stays the same, bit for bit.
    say("pool")
    page, n_pages = 16, 40
    pool = block.PagePool(n_pages)
    cache = block.KvCache.empty(n_pages, page, 2, 64)
    gen = torch.Generator().manual_seed(2)
    filler = pool.alloc(11)
    a = pool.alloc(3)

    def tables(pages):
        return torch.tensor([pages], dtype=torch.int32, device=DEV)

    def lens(n, total):
        return (torch.tensor([0, n], dtype=torch.int32, device=DEV), torch.tensor([total], dtype=torch.int32, device=DEV))

    def append(pages, n, total):
        k, v = (torch.randn(n, 2, 64, generator=gen).to(BF).to(DEV) for _ in range(2))
        block.kv_append(k, v, cache, tables(pages), *lens(n, total))

    append(a, 40, 40)
    b = pool.fork(a)
    move = pool.writable(b, 2)
    assert move is not None and b[2] != a[2] and pool.writable(b, 2) is None
    block.kv_copy_pages(cache, [move[0]], [move[1]])
    append(b, 5, 45)
    append(a, 3, 43)
    q = torch.randn(2, 4, 64, generator=gen).to(BF).to(DEV)
    ws = block.AttnWorkspace(64)

    def read(pages, total):
        out = torch.empty_like(q)
        block.attn_run(q, cache, tables(pages), *lens(2, total), out, ws, max_q=2)
        torch.cuda.synchronize()
        return out

    before_a, before_b = read(a, 43), read(b, 45)
    ro, _, bo, _ = ref.attention(q, cache.k, cache.v, tables(b), *lens(2, 45), 64 ** -0.5)
    ref.assert_within("fork", before_b, ro, bo)
    pool.free(filler)
    assert torch.equal(read(a, 43), before_a)
    pool.free(a)
    src, dst = pool.compact()
    block.kv_copy_pages(cache, src, dst)
    b = pool.remap(b, src, dst)
    assert max(b) == 2 and pool.free_pages == n_pages - 3
    cache.k[3:] = math.nan
    cache.v[3:] = math.nan
    assert torch.equal(read(b, 45), before_b)


def test_workspace_serves_batches_in_turn(block):
    # One workspace under kernels of every kind, in turn, gives what fresh ones give; past its first
    # bytes it may hold anything.
    say("workspace reuse")
    ws = block.AttnWorkspace(128)
    ws.buffer[block.ATTN_ZEROED:].fill_(255)
    cases = []
    for i, (new, cached, heads) in enumerate([([1], [6000], 8), ([2, 3], [900, 4000], 8), ([8], [3000], 8), ([50], [2000], 4),
                                              ([1] * 20, [700] * 20, 4)]):
        cache, table, q_start, kv_len, gen = make_batch(block, new, cached, 16, 1, 128, BF, 20 + i)
        q = torch.randn(sum(new), heads, 128, generator=gen).to(BF).to(DEV)
        fresh = run_attn(block, cache, table, q_start, kv_len, q, max_q=max(new))
        cases.append((cache, table, q_start, kv_len, q, max(new), fresh))
    for i in [0, 1, 2, 3, 4, 2, 0, 4, 1, 3, 0, 0]:
        cache, table, q_start, kv_len, q, max_q, fresh = cases[i]
        out, lse = run_attn(block, cache, table, q_start, kv_len, q, ws, max_q=max_q)
        assert torch.equal(out, fresh[0]) and torch.equal(lse, fresh[1]), i


def decode_step(block, state):
    """Every operator once, as a decode step runs them."""
    cache, table, q_start, kv_len, wide, w, ws, buf = state
    tokens = wide.shape[0]
    q, k, v, gate = wide.split([1024, 128, 128, 1024], 1)
    block.kv_append(k.view(tokens, 1, 128), v.view(tokens, 1, 128), cache, table, q_start, kv_len)
    block.attn_run(q.view(tokens, 8, 128), cache, table, q_start, kv_len, buf["attn"], ws, max_q=buf["max_q"],
                   gate=gate.view(tokens, 8, 128))
    block.w4_run(w, buf["attn"].view(tokens, 1024), buf["o"])
    block.norm_run(buf["o"], buf["res"], buf["out"], weight_pre=buf["pre"], weight_post=buf["post"], alpha=0.5,
                   residual_out=buf["res_out"])


def step_state(block, new, cached, seed):
    cache, table, q_start, kv_len, gen = make_batch(block, new, cached, 16, 1, 128, BF, seed)
    tokens, width = sum(new), 320
    g = torch.Generator(DEV).manual_seed(seed)
    w = block.w4_prepare(torch.randint(0, 256, (width, 512), generator=g, device=DEV, dtype=torch.uint8),
                         torch.rand(width, 8, generator=g, device=DEV).to(BF) / 64)
    buf = {"max_q": max(new), "attn": torch.empty(tokens, 8, 128, dtype=BF, device=DEV),
           "o": torch.empty(tokens, width, dtype=BF, device=DEV), "out": torch.empty(tokens, width, dtype=BF, device=DEV),
           "res": torch.randn(tokens, width, generator=g, device=DEV), "res_out": torch.empty(tokens, width, device=DEV),
           "pre": torch.rand(width, generator=g, device=DEV).to(BF), "post": torch.rand(width, generator=g, device=DEV).to(BF)}
    wide = torch.randn(tokens, 2304, generator=g, device=DEV).to(BF)
    return cache, table, q_start, kv_len, wide, w, block.AttnWorkspace(128), buf


@pytest.mark.parametrize("new,cached", [([1, 1], [5000, 20]), ([3], [700]), ([8, 2], [3000, 64]), ([30], [1500])])
def test_graph_replays_match_eager(block, new, cached):
    say("graph", new)
    state = step_state(block, new, cached, 31)
    wide, buf = state[4], state[-1]
    decode_step(block, state)               # first launches outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        decode_step(block, state)
    for i in range(4):
        wide.copy_(torch.randn(wide.shape, generator=torch.Generator(DEV).manual_seed(i), device=DEV).to(BF))
        decode_step(block, state)
        torch.cuda.synchronize()
        eager = {k: buf[k].clone() for k in ("attn", "o", "out", "res_out")}
        for k in eager:
            buf[k].fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for k in eager:
            assert torch.equal(eager[k], buf[k]), (i, k)


def test_on_another_stream(block):
    # Inputs made on a side stream, work put on it by argument and as torch's current stream.
    say("streams")
    state = step_state(block, [2, 1], [300, 40], 33)
    wide, buf = state[4], state[-1]
    decode_step(block, state)
    torch.cuda.synchronize()
    want = buf["out"].clone()
    source = wide.clone()
    side = torch.cuda.Stream()
    for _ in range(3):
        wide.zero_()
        buf["out"].zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(2000000)
            wide.copy_(source)
            decode_step(block, state)
        side.synchronize()
        assert torch.equal(buf["out"], want)
    out = torch.zeros_like(buf["attn"])
    with torch.cuda.stream(side):
        torch.cuda._sleep(2000000)
        wide.copy_(source)
    q = wide[:, :1024].view(3, 8, 128)
    block.attn_run(q, state[0], state[1], state[2], state[3], out, state[6], max_q=2, stream=side,
                   gate=wide[:, 1280:].view(3, 8, 128))
    side.synchronize()
    assert torch.equal(out, buf["attn"])


# ------------------------------------------------------------------ 4-bit projections

W4 = [
    # m, n, k, group, zeros, dtype
    (1, 16, 128, 128, False, BF), (1, 2304, 8192, 128, False, BF), (2, 100, 4096, 64, True, FH), (3, 33, 96, 32, True, BF),
    (7, 8192, 1024, 128, True, BF), (16, 257, 5000 // 32 * 32, 32, False, FH), (17, 1000, 2048, 64, True, BF),
    (31, 8200, 512, 128, False, FH), (32, 8192, 320, 64, True, BF), (33, 65, 4160, 32, True, BF), (64, 8192, 256, 32, False, BF),
    (70, 130, 1024, 128, True, FH), (300, 48, 640, 128, False, BF), (1, 1, 32, 32, True, FH), (5, 515, 4128, 32, True, BF),
]


def w4_inputs(m, n, k, group, zeros, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8)
    s = ((0.2 + torch.rand(n, k // group, generator=g)) * k ** -0.5).to(dtype)
    z = torch.randint(0, 16, (n, k // group), generator=g, dtype=torch.uint8) if zeros else None
    x = torch.randn(m, k, generator=g) * (1 + 7 * (torch.rand(m, 1, generator=g) < 0.2)) + (torch.rand(m, 1, generator=g) < 0.3) * 2
    return q, s, z, x.to(dtype)


@pytest.mark.parametrize("case", range(len(W4)))
def test_w4(block, case):
    m, n, k, group, zeros, dtype = W4[case]
    say("w4", W4[case])
    q, s, z, x = w4_inputs(m, n, k, group, zeros, dtype, case)
    w = block.w4_prepare(q.to(DEV), s.to(DEV), z.to(DEV) if zeros else None, group)
    out = torch.full((m, n), math.nan, dtype=dtype, device=DEV)
    block.w4_run(w, x.to(DEV), out)
    torch.cuda.synchronize()
    r, b = ref.w4(q, s, z, group, x)
    ref.assert_within("w4", out, r, b)


@pytest.mark.parametrize("dtype", [BF, FH])
@pytest.mark.parametrize("m", [2, 9, 20, 40])
def test_w4_one_hot_rows_are_exact(block, dtype, m):
    # x = 2^e at one k: the output is one weight times 2^e, rounded once; and strided x and out.
    say("w4 one hot", dtype, m)
    n, k, group = 67, 416, 32
    q, s, z, _ = w4_inputs(m, n, k, group, True, dtype, 3)
    w = block.w4_prepare(q.to(DEV), s.to(DEV), z.to(DEV), group)
    x = torch.zeros(m, k)
    at = [(37 * i + 5) % k for i in range(m)]
    for i in range(m):
        x[i, at[i]] = 2.0 ** (i % 5 - 2)
    xw = torch.full((m, k + 24), math.nan, dtype=dtype, device=DEV)
    xw[:, 8:8 + k] = x.to(dtype).to(DEV)
    ow = torch.full((m, n + 5), 3.0, dtype=dtype, device=DEV)
    block.w4_run(w, xw[:, 8:8 + k], ow[:, 2:2 + n])
    torch.cuda.synchronize()
    r, _ = ref.w4(q, s, z, group, x.to(dtype))
    # (exact in FP32 before the one rounding: weight and activation are a few bits each)
    assert torch.equal(ow[:, 2:2 + n].cpu(), r.float().to(dtype))
    assert bool((ow[:, :2] == 3).all()) and bool((ow[:, 2 + n:] == 3).all())


def test_w4_no_rows(block):
    q, s, _, x = w4_inputs(1, 20, 64, 32, False, BF)
    w = block.w4_prepare(q.to(DEV), s.to(DEV), group=32)
    block.w4_run(w, x.to(DEV)[:0], torch.empty(0, 20, dtype=BF, device=DEV))
    torch.cuda.synchronize()


# ------------------------------------------------------------------ norms around a block

NORM = [
    # m, width, dtype, residual dtype, post, gate, alpha
    (1, 8192, BF, BF, True, "row", 0.7), (3, 1, BF, F32, True, "none", 1.0), (5, 7, FH, FH, True, "token", -2.0),
    (2, 1000, BF, F32, False, "row", 0.5), (9, 1024, FH, F32, True, "token", 1.0), (4, 8200, BF, BF, True, "none", 0.1),
    (2, 32768, FH, FH, True, "row", 1.0), (2, 32761, BF, F32, True, "token", 1.0), (300, 72, BF, BF, False, "none", 1.0),
    (1, 16384, BF, F32, True, "row", 0.3), (2, 8191, FH, F32, True, "none", 1.0),
]


def norm_inputs(m, width, dtype, res, post, gate, seed):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(m, width, generator=g) * (1 + 30 * (torch.rand(m, 1, generator=g) < 0.3))).to(dtype)
    r = (2 * torch.randn(m, width, generator=g)).to(res)
    wp = (1 + 0.2 * torch.randn(width, generator=g)).to(dtype) if post else None
    w = (1 + 0.2 * torch.randn(width, generator=g)).to(dtype)
    gt = {"none": None, "row": torch.randn(width, generator=g).to(dtype), "token": torch.randn(m, width, generator=g).to(dtype)}[gate]
    return x, r, w, wp, gt


@pytest.mark.parametrize("case", range(len(NORM)))
@pytest.mark.parametrize("padded", [False, True])
def test_norm(block, case, padded):
    m, width, dtype, res, post, gate, alpha = NORM[case]
    say("norm", NORM[case], padded)
    x, r, w, wp, gt = norm_inputs(m, width, dtype, res, post, gate, case)
    eps = 1e-5

    def rows(t, fill=math.nan):
        # padded: rows further apart and starting one element off 16 bytes
        if not padded:
            return t.to(DEV)
        big = torch.full((m, width + 3), fill, dtype=t.dtype, device=DEV)
        big[:, 1:1 + width] = t.to(DEV)
        return big[:, 1:1 + width]

    dx, dr = rows(x), rows(r)
    out, ro = rows(torch.full((m, width), math.nan, dtype=dtype)), rows(torch.full((m, width), math.nan, dtype=res))
    dg = None if gt is None else gt.to(DEV) if gt.dim() == 1 else rows(gt)
    block.norm_run(dx, dr, out, weight_pre=w.to(DEV), weight_post=None if wp is None else wp.to(DEV), gate=dg, alpha=alpha,
                   eps=eps, residual_out=ro)
    torch.cuda.synchronize()
    rr, o, br, bo = ref.norm(x, r, w, wp, gt, alpha, eps)
    ref.assert_within("residual", ro, rr, br)
    ref.assert_within("out", out, o, bo)
    # in place: the residual updated where it is, out over x
    block.norm_run(dx, dr, dx, weight_pre=w.to(DEV), weight_post=None if wp is None else wp.to(DEV), gate=dg, alpha=alpha, eps=eps)
    torch.cuda.synchronize()
    assert torch.equal(dx, out) and torch.equal(dr, ro)


@pytest.mark.parametrize("width,res", [(4096, BF), (333, F32)])
def test_norm_before_the_first_block(block, width, res):
    say("norm first", width)
    _, r, w, _, _ = norm_inputs(6, width, BF, res, False, "none", 1)
    r[2] = 0                                # a row of zeros stays zero
    out = torch.empty(6, width, dtype=BF, device=DEV)
    block.norm_run(None, r.to(DEV), out, weight_pre=w.to(DEV))
    torch.cuda.synchronize()
    _, o, _, bo = ref.norm(None, r, w, None, None, 1.0, 1e-6)
    ref.assert_within("out", out, o, bo)
    assert bool((out[2] == 0).all())


# ------------------------------------------------------------------ refusals

def test_refusals(block):
    from gemv_decode_projections_amd.binding import ProjError

    cache, table, q_start, kv_len, gen = make_batch(block, [2], [10], 8, 2, 64, BF)
    ws = block.AttnWorkspace(64)
    q = torch.zeros(2, 4, 64, dtype=BF, device=DEV)
    out = torch.zeros_like(q)
    kv = torch.zeros(2, 2, 64, dtype=BF, device=DEV)

    def attn(q=q, out=out, table=table, q_start=q_start, kv_len=kv_len, ws=ws, **kw):
        block.attn_run(q, cache, table, q_start, kv_len, out, ws, **kw)

    for what, bad in [
        ("q has shape", dict(q=q.half())), ("q has 3 heads", dict(q=q[:, :3])), ("q has shape", dict(q=q[:, :, :32], out=out[:, :, :32])),
        ("contiguous", dict(q=torch.zeros(2, 64, 4, dtype=BF, device=DEV).transpose(1, 2))), ("out has shape", dict(out=out[:1])),
        ("not a GPU", dict(out=out.cpu())), ("gate has shape", dict(gate=q[:, :2])), ("lse", dict(lse=torch.zeros(2, 4, device=DEV).half())),
        ("int32", dict(table=table.long())), ("q_start", dict(q_start=q_start[:1])), ("int32", dict(kv_len=kv_len.float())),
        ("max_q", dict(max_q="x")), ("scale", dict(scale="x")), ("workspace", dict(ws=type("W", (), {"head_dim": 32, "index": 0})())),
    ]:
        with pytest.raises(ValueError, match=what):
            attn(**bad)
    for bad in (dict(scale=0.0), dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan), dict(window=-1), dict(max_q=0)):
        with pytest.raises(ProjError):
            attn(**bad)
    odd = torch.zeros(2 * 4 * 64 + 8, dtype=BF, device=DEV)
    with pytest.raises(ProjError, match="ALIGN"):
        attn(q=odd[1:1 + 512].view(2, 4, 64))
    with pytest.raises(ProjError, match="ARG"):
        attn(q=torch.zeros(2, 4, 65, dtype=BF, device=DEV)[:, :, :64])       # rows 130 bytes apart
    for what, bad in [("k has shape", (kv[:, :1], kv[:, :1])), ("v has shape", (kv, kv[:1])),
                      ("strides", (kv, torch.zeros(2, 3, 64, dtype=BF, device=DEV)[:, :2])), ("not a GPU", (kv.cpu(), kv))]:
        with pytest.raises(ValueError, match=what):
            block.kv_append(*bad, cache, table, q_start, kv_len)
    n = cache.n_pages
    for src, dst in [([0], [n]), ([n], [0]), ([0, 1], [2, 2]), ([0, 1], [1, 2]), ([3], [3])]:
        with pytest.raises(ProjError, match="ARG"):
            block.kv_copy_pages(cache, src, dst)
    for src, dst in [([0], [1, 2]), ([-1], [0]), (["a"], [0]), (5, [0]), ([2 ** 31], [0])]:
        with pytest.raises(ValueError):
            block.kv_copy_pages(cache, src, dst)
    gaps = torch.zeros(2, 4, 8, 2, 128, dtype=BF, device=DEV)[..., :64]        # pages with holes
    with pytest.raises(ProjError, match="ARG"):
        block.kv_copy_pages(block.KvCache(gaps[0], gaps[1]), [0], [1])
    w = block.w4_prepare(torch.zeros(8, 32, dtype=torch.uint8, device=DEV), torch.zeros(8, 2, dtype=BF, device=DEV), group=32)
    x = torch.zeros(3, 64, dtype=BF, device=DEV)
    for what, a in [("x has shape", (x[:, :32], torch.zeros(3, 8, dtype=BF, device=DEV))), ("out has shape", (x, x)),
                    ("out has shape", (x, torch.zeros(2, 8, dtype=BF, device=DEV))), ("x has shape", (x.half(), x)), ("not a GPU", (x.cpu(), x))]:
        with pytest.raises(ValueError, match=what):
            block.w4_run(w, *a)
    with pytest.raises(ProjError, match="ALIGN"):
        block.w4_run(w, torch.zeros(3, 72, dtype=BF, device=DEV)[:, 1:65], torch.zeros(3, 8, dtype=BF, device=DEV))
    r, v = torch.zeros(3, 64, device=DEV), torch.zeros(64, dtype=BF, device=DEV)
    for what, a, kw in [("weight_pre", (x, r, x), dict(weight_pre=None)), ("residual has", (x, r[:2], x), dict(weight_pre=v)),
                        ("residual must", (x, r.half(), x), dict(weight_pre=v)), ("gate has", (x, r, x), dict(weight_pre=v, gate=v[:3])),
                        ("need x", (None, r, x), dict(weight_pre=v, weight_post=v)), ("weight_post has", (x, r, x), dict(weight_pre=v, weight_post=r[0])),
                        ("x has", (x[:1], r, x), dict(weight_pre=v)), ("not a GPU", (x.cpu(), r, x), dict(weight_pre=v))]:
        with pytest.raises(ValueError, match=what):
            block.norm_run(*a, **kw)
    big = torch.zeros(1, 32769, dtype=BF, device=DEV)
    with pytest.raises(ProjError, match="ARG"):
        block.norm_run(big, big.clone(), big.clone(), weight_pre=big[0])
    torch.cuda.synchronize()


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("w4", [False, True])
def test_the_example_matches_a_plain_block(block, w4):
    # The served block (chunks, fork, compaction) against the whole sequence at once in 64 bits. The
    # stages round to BF16 six times (2^-9 of a value each at most, 2^-10 on average), through two
    # norms and a product each: a few parts in a thousand of the logits' norm; 2e-2 is held. A token
    # lost, misplaced or seen too many changes them by more than a tenth.
    from examples import decode_block as ex

    say("example", w4)
    out, fed, model = ex.main(w4=w4, prompts=(140, 37, 1), steps=6)
    weights = {name: w.double() for name, w in model.w.items()}
    if w4:
        for name in model.w4:
            q, s = ex.four_bits(model.w[name])
            n, k = model.w[name].shape
            nib = torch.stack((q & 15, q >> 4), -1).view(n, k).double() - 8
            weights[name] = nib * torch.repeat_interleave(s.double(), 128, 1)

    def rms(x, w):
        return x / torch.sqrt(x.square().mean(-1, keepdim=True) + ex.EPS) * w.double()

    assert set(out) == {"s0", "s2", "fork"}
    for name, logits in out.items():
        h = fed[name].double()
        q, k, v, gate = (rms(h, model.pre) @ weights["qkv_gate"].t().contiguous()).split([1024, 128, 128, 1024], 1)
        score = torch.softmax(q[-1].view(8, 128) @ k.t().contiguous() * 128 ** -0.5, -1)
        mixed = (score @ v) * torch.sigmoid(gate[-1].view(8, 128))
        o = mixed.view(1, 1024) @ weights["o"].t().contiguous()
        want = rms(h[-1:] + ex.ALPHA * rms(o, model.post), model.router_pre) @ weights["router"].t().contiguous()
        err = float((logits.double() - want).norm() / want.norm())
        say(name, "relative error", err)
        assert err < 2e-2
    model.release()
