"""Plain 64-bit implementations of the decode-block operators (CPU, one sequence, row or group at
a time), and the error bounds their FP32 kernels are held to."""

import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# Smallest step of the type near zero: FP16 loses relative precision below 2^-14.
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}


def gather(cache, table_row, length):
    """The first `length` positions of one sequence (float64; NaN where the page is unmapped) and which are mapped."""
    pages, size, heads, dim = cache.shape
    at = torch.arange(length)
    page = table_row.long()[at // size]
    held = (page >= 0) & (page < pages)
    device = cache.device
    out = cache[page.clamp(0, pages - 1).to(device), (at % size).to(device)].cpu().double()
    out[~held] = math.nan
    return out, held


def attention(q, k, v, table, q_start, kv_len, scale, window=0, gate=None):
    """out, lse and their bounds. A masked position contributes nothing, whatever it holds.

    The bound of an output: with w the exact weights, A = sum w |v|,
      - scores: dim exact products summed in FP32 (any order) err by at most dim * 2^-23 * sum |q k|,
        which with the scaling and the exponential's own error moves every weight by a factor within
        1 +- (2 d + 2^-18), d = scale * max over j of that + 2^-21 * max |score|;
      - each weight is rounded to the type of v for the matrix product: u, plus half a step of the
        subnormals (weights are at most 1 before the division by their sum, which is at least 1);
      - sums of n products in FP32: n 2^-23;
      - the output is rounded once: u."""
    q, table = q.cpu(), table.cpu()
    tokens, heads, dim = q.shape
    hk = k.shape[2]
    group = heads // hk
    dtype = q.dtype
    out = torch.zeros(tokens, heads, dim, dtype=torch.float64)
    lse = torch.full((tokens, heads), -math.inf, dtype=torch.float64)
    ob, lb = torch.zeros_like(out), torch.zeros_like(lse)
    starts, lens = q_start.tolist(), kv_len.tolist()
    cap = table.shape[1] * k.shape[1]
    for b in range(len(lens)):
        s, e = starts[b], starts[b + 1]
        n, length = e - s, min(max(lens[b], 0), cap)
        if n <= 0:
            continue
        ks, held = gather(k, table[b], length)
        vs, _ = gather(v, table[b], length)
        for i in range(n):
            pos = length - n + i
            j = torch.arange(length)
            see = held & (j <= pos)
            if window:
                see &= j > pos - window
            if not bool(see.any()):
                continue
            for h in range(heads):
                kk, vv = ks[see][:, h // group], vs[see][:, h // group]
                qq = q[s + i, h].double()
                logit = kk @ qq * scale
                lse[s + i, h] = torch.logsumexp(logit, 0)
                w = torch.exp(logit - lse[s + i, h])
                out[s + i, h] = w @ vv
                d = scale * dim * 2.0 ** -23 * (kk.abs() @ qq.abs()).max() + 2.0 ** -21 * logit.abs().max()
                a = w @ vv.abs()
                part = (U[dtype] + 2 * d + 2.0 ** -18 + len(w) * 2.0 ** -23) * a
                if dtype == torch.float16:
                    part = part + TINY[dtype] * vv.abs().sum(0)
                ob[s + i, h] = part
                lb[s + i, h] = d + 2.0 ** -18 + len(w) * 2.0 ** -23 + 2.0 ** -21 * lse[s + i, h].abs()
    if gate is not None:
        g = torch.sigmoid(gate.cpu().double())
        out = out * g
        ob = ob * g + 2.0 ** -18 * out.abs()
    ob = U[dtype] * out.abs() + (1 + U[dtype]) * ob + TINY[dtype]
    return out, lse, ob, lb


def w4(q, scales, zeros, group, x):
    """out and its bound. The kernel may take the offset off after the product, so its sums hold
    terms of up to (1024 or 128 + 15 + z) |x|: FP32 sums of k + 2 k / group of those, any order."""
    n, k = q.shape[0], 2 * q.shape[1]
    w = torch.empty(n, k, dtype=torch.float64)
    w[:, 0::2] = (q.cpu() % 16).double()
    w[:, 1::2] = (q.cpu() // 16).double()
    z = zeros.cpu().double() if zeros is not None else torch.full(scales.shape, 8.0, dtype=torch.float64)
    s = scales.cpu().double()
    spread = torch.repeat_interleave
    w = (w - spread(z, group, 1)) * spread(s, group, 1)
    xd = x.cpu().double()
    out = xd @ w.t()
    offset = 2 * 143.0 if x.dtype == torch.bfloat16 else 15.0
    mag = xd.abs() @ spread(s.abs() * offset, group, 1).t()
    terms = k + 2 * k // group + 16
    u = U[x.dtype]
    return out, u * out.abs() + (1 + u) * terms * 2.0 ** -23 * mag + TINY[x.dtype]


def norm(x, residual, weight_pre, weight_post, gate, alpha, eps):
    """residual_out, out and their bounds. FP32 sums of `width` squares (relative width * 2^-23 at
    most, half of it after the root) and a few roundings of each factor: each of the two terms of
    residual_out is within c = width * 2^-24 + 2^-19 of itself; out = y * f * w with |dy| as bounded
    there and f moved by the relative error of y's norm."""
    r = residual.cpu().double()
    width = r.shape[1]
    c = width * 2.0 ** -24 + 2.0 ** -19
    dy = torch.zeros_like(r)
    if x is not None:
        t = x.cpu().double()
        if weight_post is not None:
            t = t / torch.sqrt(t.square().mean(1, keepdim=True) + eps) * weight_post.cpu().double()
        if gate is not None:
            t = t * gate.cpu().double()
        t = alpha * t
        dy = c * (t.abs() + r.abs())
        r = r + t
    f = 1 / torch.sqrt(r.square().mean(1, keepdim=True) + eps)
    w = weight_pre.cpu().double()
    out = r * f * w
    # d f / f <= sqrt(mean dy^2) * f
    df = torch.sqrt(dy.square().mean(1, keepdim=True)) * f
    dout = (dy * f * w.abs()) + out.abs() * (df + c)
    u, ur = U[weight_pre.dtype], U[residual.dtype]
    ry = ur * r.abs() + (1 + ur) * dy + TINY[residual.dtype]
    return r, out, ry, u * out.abs() + (1 + u) * 1.01 * dout + TINY[weight_pre.dtype]


def assert_within(what, got, ref, bound):
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, what
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), "%s: NaN in other places" % what
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), "%s: infinities differ" % what
    fine = torch.isfinite(ref)
    assert bool(torch.isfinite(got[fine]).all()), "%s: not finite where the reference is" % what
    over = (got[fine] - ref[fine]).abs() / bound[fine]
    assert over.numel() == 0 or float(over.max()) <= 1.0, "%s: %.3g times its bound" % (what, float(over.max()))
