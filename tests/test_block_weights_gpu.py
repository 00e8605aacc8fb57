"""GPU tests of how many bits the softmax weights keep: far below the largest, and at it."""

import math

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


def scored(block, scores, values, new, heads, dim, dtype):
    """Attention over one sequence whose position j scores scores[j] for every row."""
    total, page = len(scores), 16
    pages = -(-total // page)
    k, v = (torch.zeros(pages, page, 1, dim, dtype=dtype, device=DEV) for _ in range(2))
    k.view(-1, dim)[:total, 0] = scores.to(dtype).to(DEV)
    v.view(-1, dim)[:total] = values.to(dtype).to(DEV)
    q = torch.zeros(new, heads, dim, dtype=dtype, device=DEV)
    q[:, :, 0] = 1
    out, lse = torch.empty_like(q), torch.empty(new, heads, device=DEV)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    block.attn_run(q, block.KvCache(k, v), ints([list(range(pages))]), ints([0, new]), ints([total]), out,
                   block.AttnWorkspace(dim), max_q=new, scale=1.0, lse=lse)
    torch.cuda.synchronize()
    want, logs = [], []
    for i in range(new):
        s = scores[:total - new + i + 1].double()
        logs.append(torch.logsumexp(s, 0))
        want.append(torch.exp(s - logs[-1]) @ values[:len(s)].double())
    shape = (new, heads, dim)
    return out, lse, torch.stack(want)[:, None].expand(shape), torch.stack(logs)[:, None].expand(new, heads)


@pytest.mark.parametrize("new,heads", [(1, 8), (3, 8), (8, 8), (100, 4)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_flat_tail_below_a_sink_keeps_its_bits_in_fp16(block, new, heads, dim):
    # 4096 weights of e^-14.5 = 2^-20.9 under one of 1. In FP16 that is 8.46 of its smallest steps;
    # held as a normal number it is rounded by 2^-11 at most, as the output is.
    say("fp16 tail", new, heads, dim)
    scores, values = torch.zeros(4097), torch.full((4097, dim), 1024.0)
    scores[0], values[0] = 14.5, 0.0
    out, lse, want, logs = scored(block, scores, values, new, heads, dim, FH)
    ref.assert_within("out", out, want, (2.0 ** -10 + 2.0 ** -18) * want.abs())
    # (as in block_ref: scores and lse of 14.5 in FP32, a sum of 4097 terms)
    ref.assert_within("lse", lse, logs, 2.0 ** -18 + 4097 * 2.0 ** -23 + 2.0 ** -20 * logs.abs())


@pytest.mark.parametrize("dtype", [BF, FH])
@pytest.mark.parametrize("new,heads", [(1, 8), (3, 8), (8, 8), (100, 4)])
@pytest.mark.parametrize("gap", [3.3, 5.0, 5.4])
def test_a_dominant_key_in_a_later_tile_keeps_its_weight(block, dtype, new, heads, gap):
    # One key, and `gap` above it another some tiles later; the rest weigh nothing. The later one's
    # value comes back as the formula gives it: its weight is not rounded against the sum's, the earlier
    # one's is, by u of its share e^-gap; an output is rounded by half a step of its type.
    say("dominant", dtype, new, heads, gap)
    dim, total = 128, 400
    scores, values = torch.zeros(total), torch.zeros(total, dim)
    scores[0], scores[200] = 30.0, torch.tensor(30.0 + gap).to(dtype).float()
    values[200] = (1 + torch.arange(dim) / dim).to(dtype).float()
    out, _, want, _ = scored(block, scores, values, new, heads, dim, dtype)
    u = ref.U[dtype]
    want = want.contiguous()
    more = want.abs() * (u * math.exp(-gap) + 2.0 ** -18)
    half_step = u * 2.0 ** torch.floor(torch.log2(want.abs() + more))
    ref.assert_within("out", out, want, half_step + more)


@pytest.mark.parametrize("dtype", [BF, FH])
@pytest.mark.parametrize("dim,heads,kv_heads", [(64, 4, 2), (128, 8, 1), (256, 5, 1)])
@pytest.mark.parametrize("cached", [0, 31, 700, 5000])
def test_single_tokens_weigh_with_more_than_their_types_bits(block, dtype, dim, heads, kv_heads, cached):
    # The bound of block_ref but for the weights' rounding: in two parts of 16 bits u^2 is left of it.
    say("two parts", dtype, dim, cached)
    from tests.test_block_gpu import make_batch, run_attn

    cache, table, q_start, kv_len, gen = make_batch(block, [1, 1], [cached, cached // 2], 16, kv_heads, dim, dtype, 4)
    q = torch.randn(2, heads, dim, generator=gen).to(dtype).to(DEV)
    out, lse = run_attn(block, cache, table, q_start, kv_len, q, max_q=1)
    args = (table, q_start, kv_len, dim ** -0.5)
    want, logs, bound, log_bound = ref.attention(q, cache.k, cache.v, *args)
    size = ref.attention(q, cache.k, cache.v.abs(), *args)[0]
    u = ref.U[dtype]
    ref.assert_within("out", out, want, bound - (1 + u) * (u - u * u) * size)
    ref.assert_within("lse", lse, logs, log_bound)
