"""GPU tests of the tensors that a caller may hand to the block operators: views whose strides say
something unusual, or nothing."""

import math

import pytest
import torch

from gemv_decode_projections_amd.binding import ProjError

pytestmark = pytest.mark.gpu

BF, FH = torch.bfloat16, torch.float16
DEV = "cuda"


@pytest.fixture(scope="module")
def block():
    from gemv_decode_projections_amd import block as b

    return b


def say(*a):
    print(*a, flush=True)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def filled(block, pages, page, kv_heads, dim, seed=0):
    gen = torch.Generator(DEV).manual_seed(seed)
    shape = (pages, page, kv_heads, dim)
    return block.KvCache(*(torch.randn(shape, generator=gen, device=DEV).to(BF) for _ in range(2))), gen


@pytest.mark.parametrize("max_q", [1, 40])
def test_one_table_row_for_several_sequences(block, max_q):
    # An expanded row has a stride of 0; what lies behind its storage are valid page numbers, of others.
    say("expanded table", max_q)
    cache, gen = filled(block, 32, 16, 2, 64)
    store = ints(list(range(31, 0, -1)) * 4)
    row, seqs = store[:6][None], 4
    q_start, kv_len = ints([0, 1, 2, 5, 6]), ints([90, 17, 96, 50])
    q = torch.randn(6, 4, 64, generator=gen, device=DEV).to(BF)
    outs = []
    for table in (row.expand(seqs, -1), row.repeat(seqs, 1)):
        out = torch.full_like(q, math.nan)
        block.attn_run(q, cache, table, q_start, kv_len, out, block.AttnWorkspace(64), max_q=max_q)
        torch.cuda.synchronize()
        outs.append(out)
    assert torch.equal(*outs)
    kv = torch.randn(2, 3, 2, 64, generator=gen, device=DEV).to(BF)
    caches = []
    for table in (row.expand(2, -1), row.repeat(2, 1)):         # one appends to the first page, one to the fifth
        c = block.KvCache(cache.k.clone(), cache.v.clone())
        block.kv_append(kv[0], kv[1], c, table, ints([0, 2, 3]), ints([9, 70]))
        torch.cuda.synchronize()
        caches.append(c)
    assert torch.equal(caches[0].k, caches[1].k) and torch.equal(caches[0].v, caches[1].v)
    assert torch.equal(caches[0].k[31, 7], kv[0, 0]) and torch.equal(caches[0].v[27, 5], kv[1, 2])
    overlapping = store.as_strided((seqs, 6), (3, 1))
    with pytest.raises(ProjError, match="ARG"):
        block.attn_run(q, cache, overlapping, q_start, kv_len, out, block.AttnWorkspace(64), max_q=max_q)
    with pytest.raises(ProjError, match="ARG"):
        block.kv_append(kv[0], kv[1], cache, overlapping[:2], ints([0, 2, 3]), ints([9, 70]))


@pytest.mark.parametrize("max_q", [1, 40])
def test_a_single_table_row_of_any_stride(block, max_q):
    say("single table row", max_q)
    cache, gen = filled(block, 16, 16, 1, 64)
    q = torch.randn(2, 4, 64, generator=gen, device=DEV).to(BF)
    row = [5, 3, 9, 1]
    outs = []
    for table in (ints([row]), ints(row)[:, None].t(), ints([row]).as_strided((1, 4), (0, 1))):
        out = torch.full_like(q, math.nan)
        block.attn_run(q, cache, table, ints([0, 2]), ints([60]), out, block.AttnWorkspace(64), max_q=max_q)
        torch.cuda.synchronize()
        outs.append(out)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_another_gpu_than_the_cache_or_the_weight(block):
    # A cache and a weight that say they are on the next GPU: tensors of this one are refused, and so is
    # a call without tensors while this one is current.
    say("devices")
    here = torch.cuda.current_device()
    cache, _ = filled(block, 4, 16, 1, 64)
    w = block.w4_prepare(torch.zeros(8, 32, dtype=torch.uint8, device=DEV), torch.zeros(8, 2, dtype=BF, device=DEV), group=32)
    q = torch.zeros(1, 2, 64, dtype=BF, device=DEV)
    x, out = torch.zeros(1, 64, dtype=BF, device=DEV), torch.zeros(1, 8, dtype=BF, device=DEV)
    table, q_start, kv_len, ws = ints([[0]]), ints([0, 1]), ints([1]), block.AttnWorkspace(64)
    cache._c.device = w._shape.device = here + 1
    with pytest.raises(ValueError, match="device"):
        block.attn_run(q, cache, table, q_start, kv_len, torch.zeros_like(q), ws, max_q=1)
    with pytest.raises(ValueError, match="device"):
        block.kv_append(q[:, :1], q[:, :1], cache, table, q_start, kv_len)
    with pytest.raises(ProjError, match="DEVICE"):
        block.kv_copy_pages(cache, [0], [1])
    with pytest.raises(ValueError, match="cuda:%d" % (here + 1)):
        block.w4_run(w, x, out)
    cache._c.device = w._shape.device = here
    block.attn_run(q, cache, table, q_start, kv_len, torch.zeros_like(q), ws, max_q=1)
    block.kv_append(q[:, :1], q[:, :1], cache, table, q_start, kv_len)
    block.kv_copy_pages(cache, [0], [1])
    block.w4_run(w, x, out)

    class Stream:
        device_index, cuda_stream = here + 1, 0

    with pytest.raises(ValueError, match="stream"):
        block.w4_run(w, x, out, stream=Stream())
    torch.cuda.synchronize()


@pytest.mark.parametrize("max_q", [1, 40])
def test_one_token_and_one_head_of_any_stride(block, max_q):
    # Single rows cut from tensors whose rows are no multiple of 16 bytes apart: the stride is never used.
    say("single rows", max_q)
    cache, gen = filled(block, 8, 16, 1, 64)
    table, q_start, kv_len, ws = ints([[3, 1, 7]]), ints([0, 1]), ints([40]), block.AttnWorkspace(64)

    def odd(shape, offset):
        # one entry of the first dimension, whose stride is odd
        inner = math.prod(shape[1:])
        store = torch.randn(inner * 2 + 19, generator=gen, device=DEV).to(BF)
        size = [inner * 2 + 3]
        for n in shape[1:]:
            size.append(inner // n if len(size) == 1 else 1)
        return store[offset:].as_strided(shape, size)

    q, gate = odd((1, 4, 64), 0), odd((1, 4, 64), 8)
    out, plain = odd((1, 4, 64), 16), torch.empty(1, 4, 64, dtype=BF, device=DEV)
    block.attn_run(q, cache, table, q_start, kv_len, out, ws, max_q=max_q, gate=gate)
    block.attn_run(q.contiguous(), cache, table, q_start, kv_len, plain, ws, max_q=max_q, gate=gate.contiguous())
    torch.cuda.synchronize()
    assert torch.equal(out, plain) and bool(torch.isfinite(plain).all())
    k, v = odd((1, 1, 64), 0), odd((1, 1, 64), 8).as_strided((1, 1, 64), (5, 3, 1))
    block.kv_append(k, v, cache, table, q_start, kv_len)
    torch.cuda.synchronize()
    assert torch.equal(cache.k[7, 7], k[0]) and torch.equal(cache.v[7, 7], v[0])
    w = block.w4_prepare(torch.randint(0, 256, (24, 32), device=DEV, dtype=torch.uint8), torch.rand(24, 2, device=DEV).to(BF), group=32)
    x, o, want = odd((1, 64), 0), odd((1, 24), 3), torch.empty(1, 24, dtype=BF, device=DEV)
    block.w4_run(w, x, o)
    block.w4_run(w, x.contiguous(), want)
    r, res, pre = odd((1, 64), 8), odd((1, 64), 0), torch.rand(64, generator=gen, device=DEV).to(BF)
    y, z = torch.empty(1, 64, dtype=BF, device=DEV), torch.empty(1, 64, dtype=BF, device=DEV)
    block.norm_run(x, r, y, weight_pre=pre, residual_out=res)
    block.norm_run(x.contiguous(), r.contiguous(), z, weight_pre=pre, residual_out=torch.empty_like(z))
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(y, z)
    one = block.KvCache(cache.k[:1].as_strided((1, 16, 1, 64), (77, 64, 3, 1)), cache.v[:1].as_strided((1, 16, 1, 64), (77, 64, 3, 1)))
    block.attn_run(q, one, ints([[0]]), q_start, ints([9]), out, ws, max_q=max_q)
    block.attn_run(q, cache, ints([[0]]), q_start, ints([9]), plain, ws, max_q=max_q)
    torch.cuda.synchronize()
    assert torch.equal(out, plain)


FIRST_CALLS = """
import torch
from gemv_decode_projections_amd import block

BF, DEV = torch.bfloat16, "cuda"
g = torch.Generator(DEV).manual_seed(0)
rand = lambda *s: torch.randn(*s, generator=g, device=DEV).to(BF)
ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
ws, cache, parts = block.AttnWorkspace(128), block.KvCache(rand(240, 16, 1, 128), rand(240, 16, 1, 128)), []
for i, new in enumerate((1, 3, 8, 40)):         # every kind of kernel, with parts to be joined; each its own pages
    parts.append((rand(new, 8, 128), rand(new, 1, 128), ints([0, new]), ints([900]), torch.zeros(new, 8, 128, dtype=BF, device=DEV),
                  ints([list(range(57 * i, 57 * i + 57))])))
w = block.w4_prepare(torch.randint(0, 256, (320, 512), generator=g, device=DEV, dtype=torch.uint8), torch.rand(320, 8, generator=g, device=DEV).to(BF) / 64)
x, o, r, y = rand(4, 1024), torch.zeros(4, 320, dtype=BF, device=DEV), torch.randn(4, 320, generator=g, device=DEV), rand(4, 320)
out, pre, ro = torch.zeros_like(y), rand(320), torch.zeros_like(r)


def step():
    for q, k, start, length, dst, table in parts:
        block.kv_append(k, k, cache, table, start, length)
        block.attn_run(q, cache, table, start, length, dst, ws, max_q=q.shape[0])
    block.kv_copy_pages(cache, [1, 2], [238, 239])
    block.w4_run(w, x, o)
    block.norm_run(y, r, out, weight_pre=pre, residual_out=ro)


graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    step()
results = [p[4] for p in parts] + [o, out, ro, cache.k]
for i in range(3):
    for t in [x, y] + [p[1] for p in parts]:
        t.copy_(rand(*t.shape))
    graph.replay()
    torch.cuda.synchronize()
    replayed = [t.clone() for t in results]
    step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) and bool(a.float().abs().sum() > 0) for a, b in zip(replayed, results)), i
print("replays match")
"""


def test_the_first_calls_of_a_process_may_be_captured():
    # No launch of any of the kernels before the capture.
    import os
    import subprocess
    import sys

    say("first calls captured")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=100)
    assert r.returncode == 0 and "replays match" in r.stdout, r.stdout + r.stderr
