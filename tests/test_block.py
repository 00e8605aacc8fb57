"""The block operators' host side (CPU only): exports, refusals of the C ABI and of the compiled
tensor checks, the page pool against a plain model, and the references against one another."""

import ctypes
import math
import os
import random
import re

import pytest
import torch

from gemv_decode_projections_amd import binding
from tests import block_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

OK, NULL, ALIGN, ARG, SCRATCH = 0, -3, -4, -10, -9


@pytest.fixture(scope="module")
def block():
    if not os.path.exists(os.path.join(os.path.dirname(binding.LIB_PATH), "_block.so")):
        from gemv_decode_projections_amd import build

        build.build()
    from gemv_decode_projections_amd import block as b

    b._ext()
    return b


@pytest.fixture(scope="module")
def lib(block):
    return block._lib()


def test_every_declared_function_is_exported(lib):
    with open(os.path.join(ROOT, "include", "block.h")) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(blk_\w+)\s*\(", text, flags=re.M))
    assert len(names) >= 15, names
    for n in names:
        assert hasattr(lib, n), n


def test_zeroed_bytes_match_the_header(block):
    with open(os.path.join(ROOT, "include", "block.h")) as f:
        assert int(re.search(r"#define BLK_ATTN_ZEROED (\d+)", f.read()).group(1)) == block.ATTN_ZEROED


def test_new_statuses_have_texts(lib):
    for s in (-10, -11):
        assert binding.proj_strerror(s) != "unknown status" and s in binding.STATUS


class Batch(ctypes.Structure):
    _fields_ = [("q_start", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64), ("table_width", ctypes.c_int), ("seqs", ctypes.c_int), ("tokens", ctypes.c_int)]


class Attn(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64), ("gate_stride", ctypes.c_int64),
                ("gate_head_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64), ("out_head_stride", ctypes.c_int64),
                ("heads", ctypes.c_int), ("max_q", ctypes.c_int), ("window", ctypes.c_int), ("scale", ctypes.c_float)]


class Norm(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("x", "residual", "gate", "weight_post", "weight_pre", "residual_out", "out")] + \
               [(n, ctypes.c_int64) for n in ("xs", "rs", "gs", "ys", "os")] + \
               [("width", ctypes.c_int), ("dtype", ctypes.c_int), ("residual_dtype", ctypes.c_int), ("alpha", ctypes.c_float),
                ("eps", ctypes.c_float)]


def changed(base, **kw):
    s = type(base).from_buffer_copy(base)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def test_c_entries_refuse_before_any_launch(block, lib):
    # No GPU here: a call that passes its checks would fail in the launch, so every status below is
    # the checks' own; tokens = 0 and m = 0 return without a launch.
    vp, p = ctypes.c_void_p, 4096
    cache = block._Cache(p, p, 16 * 2 * 64, 2 * 64, 64, 8, 16, 2, 64, 0)
    batch = Batch(p, p, p, 4, 4, 2, 0)
    busy = changed(batch, tokens=3)
    ref_ = ctypes.byref
    append = lambda c, b, k=p, v=p, s=128, h=64: lib.blk_kv_append(ref_(c) if c else None, ref_(b) if b else None,  # noqa: E731
                                                                   vp(k), vp(v), ctypes.c_int64(s), ctypes.c_int64(h), vp(0))
    assert append(cache, batch) == OK
    assert append(None, batch) == NULL and append(cache, None) == NULL
    assert append(cache, busy, k=0) == NULL and append(cache, busy, v=p + 2) == ALIGN
    assert append(cache, batch, s=12) == ARG and append(cache, batch, h=-8) == ARG
    for kw, want in [(dict(k=0), NULL), (dict(v=p + 8), ALIGN), (dict(page_size=4), ARG), (dict(page_size=24), ARG),
                     (dict(head_dim=96), ARG), (dict(dtype=2), ARG), (dict(n_pages=0), ARG), (dict(kv_heads=0), ARG),
                     (dict(token_stride=100), ARG), (dict(page_stride=-8), ARG), (dict(page_stride=1 << 31), ARG),
                     (dict(page_size=1 << 20, token_stride=1 << 20), ARG)]:
        assert append(changed(cache, **kw), batch) == want, kw
    for kw, want in [(dict(seqs=-1), ARG), (dict(tokens=-1), ARG), (dict(table_width=0), ARG), (dict(table_stride=3), ARG),
                     (dict(tokens=2, table=0), NULL), (dict(kv_len=p + 2), ALIGN)]:
        assert append(cache, changed(batch, **kw)) == want, kw

    args = Attn(p, 0, p, 0, 256, 64, 0, 0, 256, 64, 4, 1, 0, 0.125)
    size = lib.blk_attn_workspace_bytes(64)
    assert size > 0 and lib.blk_attn_workspace_bytes(0) == 0 and lib.blk_attn_workspace_bytes(512) == 0
    attn = lambda a=args, b=batch, c=cache, ws=p, n=size: lib.blk_attn_run(ref_(c), ref_(b), ref_(a) if a else None,  # noqa: E731
                                                                         vp(ws), ctypes.c_size_t(n), vp(0))
    assert attn() == OK and attn(a=None) == NULL
    for kw in (dict(heads=3), dict(heads=0), dict(max_q=0), dict(window=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.inf),
               dict(scale=math.nan), dict(q_stride=4), dict(out_head_stride=-8), dict(gate_stride=1 << 41)):
        assert attn(changed(args, **kw)) == ARG, kw
    assert attn(b=busy, ws=0) == NULL and attn(changed(args, q=0), busy) == NULL and attn(changed(args, out=0), busy) == NULL
    assert attn(b=busy, ws=p + 128) == ALIGN and attn(changed(args, gate=p + 4), busy) == ALIGN
    assert attn(changed(args, lse=p + 2), busy) == ALIGN and attn(b=busy, n=size - 1) == SCRATCH
    assert attn(b=changed(busy, table_width=1 << 27, table_stride=1 << 27)) == ARG

    pages = (ctypes.c_int32 * 4)
    copy = lambda s, d, n, c=cache: lib.blk_kv_copy_pages(ref_(c), s, d, n, vp(0))  # noqa: E731
    lib.blk_kv_copy_pages.argtypes = [ctypes.c_void_p] * 3 + [ctypes.c_int, vp]
    assert copy(None, None, 0) == OK and copy(None, None, 1) == NULL and copy(pages(), pages(), -1) == ARG
    for s, d in [((0, 8), (1, 2)), ((0, 1), (2, 8)), ((0, 1), (2, 2)), ((0, 1), (1, 2)), ((0, -1), (2, 3))]:
        assert copy(pages(*s), pages(*d), 2) == ARG
    assert copy(pages(0), pages(1), 1, changed(cache, token_stride=256)) == ARG      # holes between tokens
    assert copy(pages(0), pages(1), 1, changed(cache, page_stride=64)) == ARG        # pages that overlap

    w = block._W4(64, 256, 128, 0, 0)
    assert lib.blk_w4_packed_bytes(w) == 4 * 2 * 1024 + 4 * 2 * 32 and lib.blk_w4_packed_bytes(changed(w, has_zeros=1)) > 0
    lib.blk_w4_run.argtypes = [vp, vp, vp, ctypes.c_int64, ctypes.c_int, vp, ctypes.c_int64, vp]
    run = lambda w=w, packed=p, x=p, xs=256, m=0, out=p, os=64: lib.blk_w4_run(ref_(w), packed, x, xs, m, out, os, None)  # noqa: E731
    assert run() == OK
    for kw in (dict(n=0), dict(k=0), dict(group=16), dict(k=192), dict(dtype=2), dict(n=1 << 25)):
        assert run(changed(w, **kw)) == ARG and lib.blk_w4_packed_bytes(changed(w, **kw)) == 0
    assert run(xs=12) == ARG and run(m=-1) == ARG and run(m=(1 << 20) + 1) == ARG and run(os=-1) == ARG
    assert run(m=1, x=0) == NULL and run(m=1, packed=p + 8) == ALIGN and run(m=1, x=p + 8) == ALIGN and run(m=1, out=p + 1) == ALIGN
    assert lib.blk_w4_pack(w, vp(p), vp(p), vp(p), vp(p), vp(0)) == NULL              # zeros given, none announced

    n = Norm(p, p, 0, 0, p, p, p, 64, 64, 0, 64, 64, 64, 0, 2, 1.0, 1e-6)
    lib.blk_norm_run.argtypes = [vp, ctypes.c_int, vp]
    norm = lambda m=0, **kw: lib.blk_norm_run(ref_(changed(n, **kw)), m, None)  # noqa: E731
    assert norm() == OK and lib.blk_norm_run(None, 1, None) == NULL
    for kw in (dict(width=0), dict(width=32769), dict(dtype=2), dict(residual_dtype=1), dict(xs=-1), dict(m=-1)):
        assert norm(**kw) == ARG, kw
    for kw in (dict(residual=0), dict(weight_pre=0), dict(out=0), dict(residual_out=0), dict(x=0, gate=p)):
        assert norm(1, **kw) == NULL, kw
    assert norm(1, x=p + 1) == ALIGN and norm(1, residual=p + 2) == ALIGN


def test_tensors_on_the_cpu_are_refused(block):
    bf = torch.bfloat16
    with pytest.raises(ValueError, match="not a GPU"):
        block.KvCache.empty(2, 16, 1, 64, device="cpu")
    v = torch.zeros(8, dtype=bf)
    with pytest.raises(ValueError, match="not a GPU"):
        block.norm_run(v[None], v[None], v[None], weight_pre=v)
    with pytest.raises(ValueError, match="device tensor"):
        block.w4_prepare(torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 1, dtype=bf))
    with pytest.raises(ValueError, match="head_dim"):
        block.AttnWorkspace(96)
    with pytest.raises(TypeError):
        block._ext().kv_append(1, 2)
    cache = block._Cache(4096, 4096, 1, 1, 64, 8, 16, 2, 64, 0)
    with pytest.raises(ValueError, match="tensor"):
        block._ext().kv_append(ctypes.addressof(cache), 1, 2, 3, 4, 5, 0)
    with pytest.raises(ValueError, match="address"):
        block._ext().kv_copy_pages(0, [1], [2], 0)


def test_page_pool_against_a_plain_model(block):
    rng = random.Random(3)
    for size in (1, 7, 64, 65, 200):
        pool, users, held = block.PagePool(size), [0] * size, []
        for _ in range(400):
            free = [p for p in range(size) if not users[p]]
            assert pool.free_pages == len(free)
            act = rng.random()
            if act < 0.4:
                n = rng.randint(0, max(1, size // 6))
                if n <= len(free):
                    got = pool.alloc(n)
                    assert got == free[:n]
                    for p in got:
                        users[p] = 1
                    held.append(got)
                else:
                    with pytest.raises(binding.ProjError, match="PAGES"):
                        pool.alloc(n)
            elif act < 0.55 and held:
                copy = pool.fork(rng.choice(held))
                for p in copy:
                    users[p] += 1
                held.append(copy)
            elif act < 0.65 and held:
                seq = rng.choice(held)
                if seq and (free or users[seq[-1]] == 1):
                    move = pool.writable(seq, len(seq) - 1)
                    if move:
                        assert users[move[0]] > 1 and move[1] == free[0] == seq[-1]
                        users[move[0]] -= 1
                        users[move[1]] = 1
            elif act < 0.92 and held:
                seq = held.pop(rng.randrange(len(held)))
                pool.free(seq)
                for p in seq:
                    users[p] -= 1
            else:
                src, dst = pool.compact(rng.choice([None, 1, 3]))
                assert len(set(src)) == len(src) and len(set(dst)) == len(dst) and not set(src) & set(dst)
                for s, d in zip(src, dst):
                    assert users[s] and not users[d] and d < s
                    users[d], users[s] = users[s], 0
                held = [pool.remap(h, src, dst) for h in held]
            assert [pool.users(p) for p in range(size)] == users
        moved = pool.compact()
        assert len(moved[0]) == len(moved[1])
        used = sorted(p for p in range(size) if pool.users(p))
        assert used == list(range(len(used)))
        assert pool.compact() == ([], [])


def test_page_pool_refuses_and_changes_nothing(block):
    pool = block.PagePool(6)
    a = pool.alloc(3)
    for bad in ([a[0], 5], [a[0], a[0]], [6], [-1], [a[1], a[2], a[1]]):
        with pytest.raises(binding.ProjError, match="ARG"):
            pool.free(bad)
        assert [pool.users(p) for p in range(6)] == [1, 1, 1, 0, 0, 0]
    with pytest.raises(binding.ProjError):
        pool.fork([a[0], 4])
    assert pool.users(a[0]) == 1 and pool.free_pages == 3
    b = pool.fork(a)
    pool.free([a[0], b[0]])                  # both users at once
    assert pool.free_pages == 4 and pool.alloc(1) == [0]
    with pytest.raises(binding.ProjError):
        pool.users(6)
    with pytest.raises(ValueError, match="not in use"):
        pool.writable([5], 0)
    with pytest.raises(binding.ProjError):
        block.PagePool(0)
    with pytest.raises(binding.ProjError):
        pool.alloc(-1)


# ------------------------------------------------------------------ the references themselves

def test_attention_reference_on_cases_known_by_hand():
    # One head, page size 8: equal keys give the mean of the values seen; a dominant key its value.
    k = torch.zeros(2, 8, 1, 64)
    v = torch.arange(16.0).repeat_interleave(64).view(2, 8, 1, 64)
    q = torch.ones(3, 1, 64)
    start, length = torch.tensor([0, 3]), torch.tensor([11])
    table = torch.tensor([[1, 0]])
    o, l, ob, lb = ref.attention(q, k, v, table, start, length, 1.0)
    seen = [8, 9, 10, 11, 12, 13, 14, 15, 0, 1, 2]
    for i in range(3):
        s = seen[:9 + i]
        assert torch.allclose(o[i], torch.full((1, 64), sum(s) / len(s), dtype=torch.float64))
        assert abs(float(l[i]) - math.log(len(s))) < 1e-12
    o, l, _, _ = ref.attention(q, k, v, table, start, length, 1.0, window=2)
    assert torch.allclose(o[:, 0, 0], torch.tensor([7.5, 0.5, 1.5], dtype=torch.float64))
    o, l, _, _ = ref.attention(q, k, v, torch.tensor([[-1, 0]]), start, length, 1.0, gate=torch.zeros(3, 1, 64))
    assert torch.allclose(o[:, 0, 0], torch.tensor([0.0, 0.25, 0.5], dtype=torch.float64))
    o, l, _, _ = ref.attention(q, k, v, table, start, torch.tensor([1]), 1.0)
    assert bool((o[:2] == 0).all()) and bool((l[:2] == -math.inf).all()) and float(o[2, 0, 0]) == 8
    k[0, 1, 0] = 10.0
    o, _, _, _ = ref.attention(q, k, v, table, start, length, 1.0)
    assert abs(float(o[1, 0, 0]) - 1.0) < 1e-9 and bool((ob > 0).all()) and bool((lb > 0).all())


def test_w4_and_norm_references_on_cases_known_by_hand():
    q = torch.tensor([[0x10] * 8 + [0x98] * 8], dtype=torch.uint8)       # 0, 1, 0, 1, .. then 8, 9, 8, 9, ..
    s = torch.tensor([[2.0]])
    x = torch.ones(1, 32)
    out, _ = ref.w4(q, s, None, 32, x)
    assert float(out) == 2 * ((0 - 8 + 1 - 8) * 8 + (8 - 8 + 9 - 8) * 8)
    out, _ = ref.w4(q, s, torch.tensor([[3]], dtype=torch.uint8), 32, x)
    assert float(out) == 2 * ((0 - 3 + 1 - 3) * 8 + (8 - 3 + 9 - 3) * 8)
    one = torch.ones(2)
    r, o, rb, ob = ref.norm(torch.tensor([[3.0, -3.0]]), torch.tensor([[1.0, 1.0]]), one, one, None, 2.0, 0.0)
    assert torch.allclose(r, torch.tensor([[3.0, -1.0]], dtype=torch.float64))
    assert torch.allclose(o, r / math.sqrt(5)) and bool((rb > 0).all()) and bool((ob > 0).all())


def test_bounds_hold_for_fp32_and_catch_wrong_results():
    g = torch.Generator().manual_seed(0)
    k, v = torch.randn(4, 8, 1, 64, generator=g).bfloat16(), torch.randn(4, 8, 1, 64, generator=g).bfloat16()
    q = torch.randn(1, 2, 64, generator=g).bfloat16()
    table, start, length = torch.tensor([[2, 0, 3]]), torch.tensor([0, 1]), torch.tensor([21])
    o, l, ob, lb = ref.attention(q, k, v, table, start, length, 0.125)
    keys = torch.cat([k[2], k[0], k[3]])[:21, 0].float()
    vals = torch.cat([v[2], v[0], v[3]])[:21, 0].float()
    for h in range(2):
        p = torch.softmax(keys @ q[0, h].float() * 0.125, 0)
        got = (p.bfloat16().float() @ vals).bfloat16()
        ref.assert_within("fp32 with rounded weights", got, o[0, h], ob[0, h])
        wrong = (torch.softmax(keys[:20] @ q[0, h].float() * 0.125, 0) @ vals[:20]).bfloat16()
        with pytest.raises(AssertionError):
            ref.assert_within("a key left out", wrong, o[0, h], ob[0, h])
    with pytest.raises(AssertionError):
        ref.assert_within("lse", l + 1e-3, l, lb)
