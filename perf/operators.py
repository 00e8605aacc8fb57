"""Measured cases of the decode-block operators: attention over a paged cache, the cache's
pages, 4-bit projections and the norms around a block.

Every case names one operator ("op") with its sizes. prepare() makes what a serving program
has in hand before the call, run() makes one pass: with `own` false in elementary torch
operations in 32 bits, with `own` true through gemv_decode_projections_amd.block. exact()
gives the same outputs from the definitions in 64 bits.
"""

import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases

def _attn(seqs, new, context, heads, kv_heads, dim, page, dtype="bf16", gate=False, window=0, ragged=True):
    return {"op": "attn", "seqs": seqs, "new": new, "context": context, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "page": page, "dtype": dtype, "gate": gate, "window": window, "ragged": ragged}


def _append(seqs, new, context, kv_heads, dim, page, dtype="bf16"):
    return {"op": "append", "seqs": seqs, "new": new, "context": context, "kv_heads": kv_heads, "dim": dim,
            "page": page, "dtype": dtype, "ragged": True}


def _copy(moves, pages, kv_heads, dim, page, dtype="bf16"):
    return {"op": "copy", "moves": moves, "pages": pages, "kv_heads": kv_heads, "dim": dim, "page": page,
            "dtype": dtype}


def _w4(m, n, k, group, zeros, dtype="bf16"):
    return {"op": "w4", "m": m, "n": n, "k": k, "group": group, "zeros": zeros, "dtype": dtype}


def _norm(m, width, residual, post, gate, dtype="bf16"):
    return {"op": "norm", "m": m, "width": width, "residual": residual, "post": post, "gate": gate, "dtype": dtype}


def listed():
    return [
        # One user's next token: 8 query heads on one key head, the width of the o projection's
        # input, with the gate that comes out of qkv_gate. Latency is all that counts.
        dict(_attn(1, 1, 1000, 8, 1, 128, 16, gate=True), name="attn_decode_1"),
        # A batch of 32 users' next tokens, contexts of all lengths up to 8192.
        dict(_attn(32, 1, 8192, 32, 8, 128, 64), name="attn_decode_32"),
        # 16 users with 8 drafted tokens each to verify, over long contexts.
        dict(_attn(16, 8, 32768, 8, 1, 128, 16, gate=True), name="attn_verify_16"),
        # A prompt's chunk: two prompts share a step of 2000 new tokens on 8192 cached ones.
        dict(_attn(2, 1000, 8192, 32, 8, 128, 16), name="attn_chunk_2000"),
        # Keys and values of a decode step, and of a prompt's chunk, put into their pages.
        dict(_append(16, 1, 4096, 1, 128, 16), name="append_decode_16"),
        dict(_append(3, 1365, 8192, 8, 128, 64), name="append_chunk_4095"),
        # The last pages of eight sequences forked, and a cache compacted by 1500 moves.
        dict(_copy(8, 4096, 1, 128, 16), name="copy_fork_8"),
        dict(_copy(1500, 8192, 8, 128, 16), name="copy_compact_1500"),
        # The qkv_gate and unpooler sizes with 4-bit weights, for one token and for 32.
        dict(_w4(1, 2304, 8192, 128, False), name="w4_qkv_gate_1"),
        dict(_w4(32, 8192, 4096, 64, True), name="w4_unpooler_32"),
        # The norms between two blocks of the hidden width 8192, for one token and for 1000.
        dict(_norm(1, 8192, "bf16", True, "row"), name="norm_1"),
        dict(_norm(1000, 8192, "f32", True, "token"), name="norm_1000"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("attn", "attn", "attn", "append", "copy", "w4", "w4", "norm"))
    dtype = rng.choice(("bf16", "bf16", "f16"))
    dim = rng.choice((64, 128, 128, 256))
    page = rng.choice((8, 16, 32, 64, 128))
    kv_heads = rng.choice((1, 2, 3, 4, 8))
    if op == "attn":
        heads = kv_heads * rng.choice((1, 2, 4, 5, 8))
        new = rng.choice((1, 1, _log(rng, 2, 17), _log(rng, 18, 1100)))
        context = _log(rng, 60, 32768 if new < 18 else 8192)
        # no more than the listed chunk computes, nor than the listed batches read
        room = min(2000 * 32 * 128 * 9000 / (new * heads * dim * (context + new)), 32 * 8 * 128 * 8192 / (kv_heads * dim * context))
        seqs = max(1, min(40, int(room), _log(rng, 1, 40)))
        window = rng.choice((0, 0, 0, _log(rng, 30, 2000)))
        return _attn(seqs, new, context, heads, kv_heads, dim, page, dtype, rng.random() < 0.4, window, rng.random() < 0.7)
    if op == "append":
        new = rng.choice((1, _log(rng, 2, 1300)))
        return _append(max(1, min(_log(rng, 1, 64), 4000 // new)), new, _log(rng, 60, 8192), kv_heads, dim, page, dtype)
    if op == "copy":
        pages = max(8, min(8192, int(8192 * 8 * 128 * 16 / (kv_heads * dim * page))))
        moves = _log(rng, 1, max(2, pages // 6))
        return _copy(moves, pages, kv_heads, dim, page, dtype)
    if op == "w4":
        group = rng.choice((32, 64, 128))
        n, k = _log(rng, 200, 8192), group * max(1, _log(rng, 500, 8192) // group)
        return _w4(_log(rng, 1, 64), n, k, group, rng.random() < 0.5, dtype)
    width = 8 * _log(rng, 64, 1024)
    return _norm(_log(rng, 1, 1000), width, rng.choice((dtype, "f32")), rng.random() < 0.7,
                 rng.choice(("none", "row", "token")), dtype)


# ------------------------------------------------------------------ sizes that follow from a case

def _lengths(case):
    """New tokens and cached-plus-new tokens of each sequence; the same for every seed."""
    rng = random.Random(case["seqs"] * 1000003 + case["new"] * 1009 + case["context"])
    new, total = [], []
    for b in range(case["seqs"]):
        full = not case["ragged"] or b == 0
        n = case["new"] if full else max(1, rng.randint(case["new"] // 2, case["new"]))
        c = case["context"] if full else rng.randint(case["context"] // 16, case["context"])
        new.append(n)
        total.append(n + c)
    return new, total


def _seen(case):
    """Pairs of a new token and a position that it sees, summed over the sequences."""
    pairs = 0
    for n, t in zip(*_lengths(case)):
        for i in range(n):
            pos = t - n + i
            pairs += min(pos + 1, case["window"]) if case["window"] else pos + 1
    return pairs


def _reach(case):
    """Cached positions that some new token sees, summed over the sequences."""
    if not case["window"]:
        return sum(_lengths(case)[1])
    return sum(min(t, n - 1 + case["window"]) for n, t in zip(*_lengths(case)))


def work(case):
    op, size = case["op"], DTYPES[case["dtype"]].itemsize
    if op == "attn":
        tokens = sum(_lengths(case)[0])
        rows = tokens * case["heads"] * case["dim"] * size
        kv = 2 * _reach(case) * case["kv_heads"] * case["dim"] * size
        return {"bytes": kv + rows * (3 if case["gate"] else 2) + tokens * case["heads"] * 4,
                "flops": 4 * _seen(case) * case["heads"] * case["dim"]}
    if op == "append":
        return {"bytes": 4 * sum(_lengths(case)[0]) * case["kv_heads"] * case["dim"] * size, "flops": 0}
    if op == "copy":
        return {"bytes": 4 * case["moves"] * case["page"] * case["kv_heads"] * case["dim"] * size, "flops": 0}
    if op == "w4":
        m, n, k, groups = case["m"], case["n"], case["k"], case["k"] // case["group"]
        return {"bytes": n * k // 2 + n * groups * (size + (1 if case["zeros"] else 0)) + (m * k + m * n) * size,
                "flops": 2 * m * n * k}
    m, h = case["m"], case["width"]
    res = DTYPES[case["residual"]].itemsize
    gate = {"none": 0, "row": h, "token": m * h}[case["gate"]]
    return {"bytes": m * h * (2 * size + 2 * res) + (gate + (2 if case["post"] else 1) * h) * size, "flops": 12 * m * h}


# ------------------------------------------------------------------ inputs

def _block():
    from gemv_decode_projections_amd import block

    return block


def _normal(shape, dtype, gen, scale=1.0):
    return (torch.randn(shape, generator=gen, device=DEV) * scale).to(dtype)


def _paged(case, seed):
    """A filled cache, the page table of every sequence and the lengths, as a scheduler keeps them."""
    gen = torch.Generator(DEV).manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    new, total = _lengths(case)
    page, need = case["page"], [-(-t // case["page"]) for t in total]
    n_pages = sum(need) + 7
    order = torch.randperm(n_pages, generator=gen, device=DEV, dtype=torch.int32)
    width = max(need)
    table = torch.zeros((len(need), width), dtype=torch.int32, device=DEV)
    at = 0
    for b, p in enumerate(need):
        table[b, :p] = order[at:at + p]
        at += p
    shape = (n_pages, page, case["kv_heads"], case["dim"])
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    s = {"gen": gen, "dtype": dtype, "tokens": start[-1], "max_new": max(new), "table": table,
         "k": _normal(shape, dtype, gen), "v": _normal(shape, dtype, gen),
         "q_start": torch.tensor(start, dtype=torch.int32, device=DEV),
         "kv_len": torch.tensor(total, dtype=torch.int32, device=DEV)}
    if own:
        s["cache"] = _block().KvCache(s["k"], s["v"])
    return s


def prepare(case, seed):
    op = case["op"]
    s = {}
    if op == "attn":
        s = _paged(case, seed)
        shape = (s["tokens"], case["heads"], case["dim"])
        # Sharper than even weights: the logits' spread is two
        s["q"] = _normal(shape, s["dtype"], s["gen"], 2.0)
        s["gate"] = _normal(shape, s["dtype"], s["gen"]) if case["gate"] else None
        s["scale"] = case["dim"] ** -0.5
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(shape[:2], dtype=torch.float32, device=DEV)
        if own:
            s["ws"] = _block().AttnWorkspace(case["dim"])
    elif op == "append":
        s = _paged(case, seed)
        shape = (s["tokens"], 2, case["kv_heads"], case["dim"])
        s["new"] = _normal(shape, s["dtype"], s["gen"])     # keys and values as one projection gives them
    elif op == "copy":
        gen = torch.Generator(DEV).manual_seed(seed)
        dtype = DTYPES[case["dtype"]]
        shape = (case["pages"], case["page"], case["kv_heads"], case["dim"])
        s = {"k": _normal(shape, dtype, gen), "v": _normal(shape, dtype, gen)}
        order = random.Random(seed).sample(range(case["pages"]), 2 * case["moves"])
        s["src"], s["dst"] = order[:case["moves"]], order[case["moves"]:]
        if own:
            s["cache"] = _block().KvCache(s["k"], s["v"])
    elif op == "w4":
        gen = torch.Generator(DEV).manual_seed(seed)
        dtype = DTYPES[case["dtype"]]
        m, n, k, groups = case["m"], case["n"], case["k"], case["k"] // case["group"]
        s = {"x": _normal((m, k), dtype, gen),
             "q": torch.randint(0, 256, (n, k // 2), generator=gen, device=DEV, dtype=torch.uint8),
             "scale": ((0.5 + torch.rand((n, groups), generator=gen, device=DEV)) * (k ** -0.5 / 4)).to(dtype),
             "zero": torch.randint(4, 12, (n, groups), generator=gen, device=DEV, dtype=torch.uint8) if case["zeros"] else None,
             "out": torch.empty((m, n), dtype=dtype, device=DEV)}
        if own:
            s["w"] = _block().w4_prepare(s["q"], s["scale"], s["zero"], case["group"])
    else:
        gen = torch.Generator(DEV).manual_seed(seed)
        dtype, res = DTYPES[case["dtype"]], DTYPES[case["residual"]]
        m, h = case["m"], case["width"]
        s = {"x": _normal((m, h), dtype, gen), "residual": _normal((m, h), res, gen, 3.0),
             "post": (1 + 0.1 * torch.randn(h, generator=gen, device=DEV)).to(dtype) if case["post"] else None,
             "pre": (1 + 0.1 * torch.randn(h, generator=gen, device=DEV)).to(dtype),
             "gate": {"none": None, "row": _normal((h,), dtype, gen), "token": _normal((m, h), dtype, gen)}[case["gate"]],
             "alpha": 0.7, "eps": 1e-6, "out": torch.empty((m, h), dtype=dtype, device=DEV),
             "new_residual": torch.empty((m, h), dtype=res, device=DEV)}
    s["case"] = case
    return s


# ------------------------------------------------------------------ one pass

def _positions(s, page, width):
    """Sequence, place among the new tokens, and position of every new token."""
    t = torch.arange(s["tokens"], device=DEV, dtype=torch.int32)
    b = torch.searchsorted(s["q_start"], t, right=True).long() - 1
    i = (t - s["q_start"][b]).long()
    n = (s["q_start"][1:] - s["q_start"][:-1]).long()
    return b, i, s["kv_len"].long()[b] - n[b] + i


def _plain_attn(s, case):
    hq, hk, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    seqs, width = s["table"].shape
    long = width * page
    table = s["table"].long()
    k = s["k"][table].float().reshape(seqs, long, hk, d).permute(0, 2, 3, 1).contiguous()
    v = s["v"][table].float().reshape(seqs, long, hk, d).permute(0, 2, 1, 3).contiguous()
    b, i, pos = _positions(s, page, width)
    q = torch.zeros((seqs, s["max_new"], hq, d), device=DEV)
    q[b, i] = s["q"].float()
    at = torch.full((seqs, s["max_new"]), -1, dtype=torch.long, device=DEV)
    at[b, i] = pos
    q = q.reshape(seqs, s["max_new"], hk, hq // hk, d).permute(0, 2, 1, 3, 4).reshape(seqs, hk, -1, d).contiguous()
    logits = torch.matmul(q, k).reshape(seqs, hk, s["max_new"], hq // hk, long) * s["scale"]
    j = torch.arange(long, device=DEV)
    sees = j <= at[:, :, None]
    if case["window"]:
        sees &= j > at[:, :, None] - case["window"]
    logits.masked_fill_(~sees[:, None, :, None, :], -math.inf)
    top = logits.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    p = torch.exp(logits.sub_(top))
    total = p.sum(-1, keepdim=True)
    lse = (torch.log(total) + top)[..., 0]
    o = torch.matmul(p.reshape(seqs, hk, -1, long), v).reshape(seqs, hk, s["max_new"], hq // hk, d)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    o = o.permute(0, 2, 1, 3, 4).reshape(seqs, s["max_new"], hq, d)[b, i]
    if s["gate"] is not None:
        o = o * torch.sigmoid(s["gate"].float())
    return {"out": o.to(s["dtype"]), "lse": lse.permute(0, 2, 1, 3).reshape(seqs, s["max_new"], hq)[b, i]}


def _plain_append(s, case):
    page = case["page"]
    b, i, pos = _positions(s, page, s["table"].shape[1])
    slot = s["table"].long()[b, pos // page]
    s["k"][slot, pos % page] = s["new"][:, 0]
    s["v"][slot, pos % page] = s["new"][:, 1]
    return {"k": s["k"], "v": s["v"]}


def _plain_copy(s, case):
    src, dst = torch.tensor(s["src"], device=DEV), torch.tensor(s["dst"], device=DEV)
    s["k"][dst] = s["k"][src]
    s["v"][dst] = s["v"][src]
    return {"k": s["k"], "v": s["v"]}


def _plain_w4(s, case):
    n, k, group = case["n"], case["k"], case["group"]
    q = torch.stack((s["q"] & 15, s["q"] >> 4), -1).reshape(n, k // group, group).float()
    zero = s["zero"].float()[:, :, None] if s["zero"] is not None else 8.0
    w = ((q - zero) * s["scale"].float()[:, :, None]).reshape(n, k)
    return torch.matmul(s["x"].float(), w.t()).to(s["x"].dtype)


def _plain_norm(s, case):
    x = s["x"].float()
    if s["post"] is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * s["post"].float()
    if s["gate"] is not None:
        x = x * s["gate"].float()
    y = s["residual"].float() + s["alpha"] * x
    out = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + s["eps"]) * s["pre"].float()
    return {"residual": y.to(s["residual"].dtype), "out": out.to(s["x"].dtype)}


PLAIN = {"attn": _plain_attn, "append": _plain_append, "copy": _plain_copy, "w4": _plain_w4, "norm": _plain_norm}


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return PLAIN[op](s, case)
    block = _block()
    if op == "attn":
        block.attn_run(s["q"], s["cache"], s["table"], s["q_start"], s["kv_len"], s["out"], s["ws"], max_q=s["max_new"],
                       scale=s["scale"], window=case["window"], gate=s["gate"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "append":
        block.kv_append(s["new"][:, 0], s["new"][:, 1], s["cache"], s["table"], s["q_start"], s["kv_len"])
        return {"k": s["k"], "v": s["v"]}
    if op == "copy":
        block.kv_copy_pages(s["cache"], s["src"], s["dst"])
        return {"k": s["k"], "v": s["v"]}
    if op == "w4":
        block.w4_run(s["w"], s["x"], s["out"])
        return s["out"]
    block.norm_run(s["x"], s["residual"], s["out"], weight_pre=s["pre"], weight_post=s["post"], gate=s["gate"],
                   alpha=s["alpha"], eps=s["eps"], residual_out=s["new_residual"])
    return {"residual": s["new_residual"], "out": s["out"]}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    op = case["op"]
    if op == "attn":
        outs, lses = [], []
        group = case["heads"] // case["kv_heads"]
        q_all = s["q"].double()
        start = s["q_start"].tolist()
        for b, total in enumerate(s["kv_len"].tolist()):
            rows = torch.arange(total, device=DEV)
            pages = s["table"][b].long()[rows // case["page"]]
            q = q_all[start[b]:start[b + 1]]
            at = total - len(q) + torch.arange(len(q), device=DEV)
            hide = rows[None, :] > at[:, None]
            if case["window"]:
                hide |= at[:, None] - rows[None, :] >= case["window"]
            heads_o, heads_l = [], []
            for h in range(case["kv_heads"]):
                k = s["k"][pages, rows % case["page"], h].double()
                v = s["v"][pages, rows % case["page"], h].double()
                for g in range(group):
                    logit = (q[:, h * group + g] @ k.t().contiguous()) * s["scale"]
                    logit[hide] = -math.inf
                    lse = torch.logsumexp(logit, -1)
                    heads_o.append(torch.exp(logit - lse[:, None]) @ v)
                    heads_l.append(lse)
            outs.append(torch.stack(heads_o, 1))
            lses.append(torch.stack(heads_l, 1))
        out = torch.cat(outs)
        if s["gate"] is not None:
            out = out / (1 + torch.exp(-s["gate"].double()))
        return {"out": out, "lse": torch.cat(lses)}
    if op == "append":
        start, k, v = s["q_start"].tolist(), s["k"].double(), s["v"].double()
        for b, total in enumerate(s["kv_len"].tolist()):
            n = start[b + 1] - start[b]
            at = torch.arange(total - n, total, device=DEV)
            page, place = s["table"][b].long()[at // case["page"]], at % case["page"]
            k[page, place] = s["new"][start[b]:start[b + 1], 0].double()
            v[page, place] = s["new"][start[b]:start[b + 1], 1].double()
        return {"k": k, "v": v}
    if op == "copy":
        k, v = s["k"].double(), s["v"].double()
        for a, b in zip(s["src"], s["dst"]):
            k[b], v[b] = k[a].clone(), v[a].clone()
        return {"k": k, "v": v}
    if op == "w4":
        n, k = case["n"], case["k"]
        w = torch.empty((n, k), dtype=torch.float64, device=DEV)
        w[:, 0::2] = (s["q"] % 16).double()
        w[:, 1::2] = (s["q"] // 16).double()
        each = torch.arange(k, device=DEV) // case["group"]
        w -= s["zero"].double()[:, each] if s["zero"] is not None else 8
        w *= s["scale"].double()[:, each]
        return s["x"].double() @ w.t().contiguous()
    x, r = s["x"].double(), s["residual"].double()
    if s["post"] is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / case["width"] + s["eps"]) * s["post"].double()
    if s["gate"] is not None:
        x = x * s["gate"].double()
    r = r + s["alpha"] * x
    return {"residual": r, "out": r / torch.sqrt((r * r).sum(-1, keepdim=True) / case["width"] + s["eps"]) * s["pre"].double()}
