"""Python binding of the C ABI in include/block.h: the operators between the
projections of a decode block.

    cache = KvCache.empty(n_pages, 16, kv_heads, head_dim)
    kv_append(k, v, cache, table, q_start, kv_len)
    attn_run(q, cache, table, q_start, kv_len, out, AttnWorkspace(head_dim), max_q=1)

Argument marshalling and checks only, as in `binding`: the work runs in the HIP
library, on the stream given or torch's current one. Calls launch and return;
nothing is allocated, synchronized or copied to the host.
"""

import ctypes

import torch

from . import binding as _b

_i, _i64, _vp, _f = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
HEAD_DIMS = (64, 128, 256)


class _Cache(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("page_stride", _i64), ("token_stride", _i64), ("head_stride", _i64),
                ("n_pages", _i), ("page_size", _i), ("kv_heads", _i), ("head_dim", _i), ("dtype", _i)]


class _Batch(ctypes.Structure):
    _fields_ = [("q_start", _vp), ("kv_len", _vp), ("table", _vp), ("table_stride", _i64), ("table_width", _i),
                ("seqs", _i), ("tokens", _i)]


class _Attn(ctypes.Structure):
    _fields_ = [("q", _vp), ("gate", _vp), ("out", _vp), ("lse", _vp), ("q_stride", _i64), ("q_head_stride", _i64),
                ("gate_stride", _i64), ("gate_head_stride", _i64), ("out_stride", _i64), ("out_head_stride", _i64),
                ("heads", _i), ("max_q", _i), ("window", _i), ("scale", _f)]


class _W4(ctypes.Structure):
    _fields_ = [("n", _i), ("k", _i), ("group", _i), ("dtype", _i), ("has_zeros", _i)]


class _Norm(ctypes.Structure):
    _fields_ = [("x", _vp), ("residual", _vp), ("gate", _vp), ("weight_post", _vp), ("weight_pre", _vp),
                ("residual_out", _vp), ("out", _vp), ("x_stride", _i64), ("residual_stride", _i64),
                ("gate_stride", _i64), ("residual_out_stride", _i64), ("out_stride", _i64), ("width", _i),
                ("dtype", _i), ("residual_dtype", _i), ("alpha", _f), ("eps", _f)]


_FUNCS = None


def _lib():
    """The library with block.h's signatures set."""
    global _FUNCS
    if _FUNCS is None:
        lib = _b._lib()
        cache, batch = ctypes.POINTER(_Cache), ctypes.POINTER(_Batch)
        sig = {
            "blk_kv_append": ([cache, batch, _vp, _vp, _i64, _i64, _vp], _i),
            "blk_kv_copy_pages": ([cache, _vp, _vp, _i, _vp], _i),
            "blk_attn_run": ([cache, batch, ctypes.POINTER(_Attn), _vp, ctypes.c_size_t, _vp], _i),
            "blk_attn_workspace_bytes": ([_i], ctypes.c_size_t),
            "blk_w4_packed_bytes": ([ctypes.POINTER(_W4)], ctypes.c_size_t),
            "blk_w4_pack": ([ctypes.POINTER(_W4), _vp, _vp, _vp, _vp, _vp], _i),
            "blk_w4_run": ([ctypes.POINTER(_W4), _vp, _vp, _i64, _i, _vp, _i64, _vp], _i),
            "blk_norm_run": ([ctypes.POINTER(_Norm), _i, _vp], _i),
        }
        for name, (args, res) in sig.items():
            f = getattr(lib, name)
            f.argtypes = args
            f.restype = res
        _FUNCS = lib
    return _FUNCS


def _raw_stream(stream, device):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _fail(rc, what):
    if rc != _b.PROJ_OK:
        raise _b.ProjError(rc, what)


def _need(ok, what):
    if not ok:
        raise ValueError(what)


class KvCache:
    """A paged cache over the tensors k and v, pages x page_size x kv_heads x head_dim
    (BF16 or FP16; any strides with the last one 1, so permuted views of head-major
    pages and slices of an interleaved tensor are fine). The tensors stay the caller's."""

    def __init__(self, k, v):
        for what, t in (("k", k), ("v", v)):
            _need(t.dim() == 4, "%s has shape %s, expected pages x page_size x kv_heads x head_dim" % (what, tuple(t.shape)))
            _need(t.is_cuda, "%s is on %s, not a GPU" % (what, t.device))
            _need(t.dtype in (torch.bfloat16, torch.float16), "%s has dtype %s, expected bfloat16 or float16" % (what, t.dtype))
            _need(t.stride(3) == 1, "%s: the elements of a head must be contiguous" % what)
        _need(k.shape == v.shape and k.stride() == v.stride() and k.dtype == v.dtype and k.device == v.device,
              "k and v differ in shape, strides, dtype or device")
        pages, size, heads, dim = k.shape
        _need(dim in HEAD_DIMS, "head_dim %d, expected one of %s" % (dim, HEAD_DIMS))
        _need(size >= 8 and size & (size - 1) == 0, "page_size %d, expected a power of two, at least 8" % size)
        self.k, self.v = k, v
        self.n_pages, self.page_size, self.kv_heads, self.head_dim = pages, size, heads, dim
        self.dtype, self.device = k.dtype, k.device
        s = k.stride()
        self._c = _Cache(k.data_ptr(), v.data_ptr(), s[0], s[1], s[2], pages, size, heads, dim, DTYPES[k.dtype])
        self._ref = ctypes.byref(self._c)

    @classmethod
    def empty(cls, n_pages, page_size, kv_heads, head_dim, dtype=torch.bfloat16, device="cuda"):
        """A cache of uninitialised pages (what no token was written to is never used)."""
        shape = (n_pages, page_size, kv_heads, head_dim)
        return cls(torch.empty(shape, dtype=dtype, device=device), torch.empty(shape, dtype=dtype, device=device))


def _batch(cache, table, q_start, kv_len, tokens):
    for what, t, dims in (("table", table, 2), ("q_start", q_start, 1), ("kv_len", kv_len, 1)):
        if t.dtype != torch.int32 or t.dim() != dims or t.device != cache.device:
            raise ValueError("%s must be an int32 tensor of %d dimension(s) on %s" % (what, dims, cache.device))
    seqs, width = table.shape
    if q_start.shape[0] != seqs + 1 or kv_len.shape[0] != seqs:
        raise ValueError("%d table rows need %d q_start and %d kv_len entries, got %d and %d"
                         % (seqs, seqs + 1, seqs, q_start.shape[0], kv_len.shape[0]))
    if (width > 1 and table.stride(1) != 1) or not q_start.is_contiguous() or not kv_len.is_contiguous():
        raise ValueError("q_start, kv_len and the rows of table must be contiguous")
    _need(width >= 1, "table has no columns")
    return _Batch(q_start.data_ptr(), kv_len.data_ptr(), table.data_ptr(),
                  max(table.stride(0), width), width, seqs, tokens)


def _heads(what, t, cache, heads, dim, tokens=None):
    """A token-major tensor tokens x heads x dim of the cache's type and device."""
    if t.dtype != cache.dtype or t.device != cache.device:
        raise ValueError("%s has dtype %s on %s, the cache %s on %s" % (what, t.dtype, t.device, cache.dtype, cache.device))
    shape = t.shape
    if len(shape) != 3 or shape[2] != dim or (heads is not None and shape[1] != heads) or (tokens is not None and shape[0] != tokens):
        raise ValueError("%s has shape %s, expected %s x %s x %d" % (what, tuple(shape), tokens or "tokens", heads or "heads", dim))
    s = t.stride()
    if s[2] != 1:
        raise ValueError("%s: the elements of a head must be contiguous" % what)
    return s


def kv_append(k, v, cache, table, q_start, kv_len, stream=None):
    """Write the new tokens' keys and values (tokens x kv_heads x head_dim) into their pages.

    table (seqs x pages), q_start (seqs + 1) and kv_len (seqs, the new tokens included) are int32 on
    the device; a token at a negative position or on an unmapped page is not written."""
    ks = _heads("k", k, cache, cache.kv_heads, cache.head_dim)
    vs = _heads("v", v, cache, cache.kv_heads, cache.head_dim, k.shape[0])
    _need(ks == vs, "k and v have different strides %s and %s" % (ks, vs))
    batch = _batch(cache, table, q_start, kv_len, k.shape[0])
    _fail(_lib().blk_kv_append(cache._ref, batch, k.data_ptr(), v.data_ptr(), ks[0], ks[1],
                               _raw_stream(stream, cache.device)), "kv_append")


def kv_copy_pages(cache, src, dst, stream=None):
    """Copy page src[i] to page dst[i], keys and values (lists of page numbers; no page twice in dst,
    none in both)."""
    n = len(src)
    _need(len(dst) == n, "%d source pages, %d destinations" % (n, len(dst)))
    pages = ctypes.c_int32 * n
    _fail(_lib().blk_kv_copy_pages(cache._ref, pages(*src), pages(*dst), n, _raw_stream(stream, cache.device)),
          "kv_copy_pages")


class AttnWorkspace:
    """Scratch of attn_run for one head_dim, ready for any batch. Calls that can overlap (other
    streams) need workspaces of their own."""

    def __init__(self, head_dim, device="cuda"):
        _need(head_dim in HEAD_DIMS, "head_dim %d, expected one of %s" % (head_dim, HEAD_DIMS))
        self.head_dim = head_dim
        self.bytes = _lib().blk_attn_workspace_bytes(head_dim)
        self.buffer = torch.zeros(self.bytes, dtype=torch.uint8, device=device)
        # Any stream may use it from here on.
        torch.cuda.current_stream(self.buffer.device).synchronize()
        self._ptr = self.buffer.data_ptr()


def attn_run(q, cache, table, q_start, kv_len, out, ws, *, max_q=None, scale=None, window=0, gate=None, lse=None,
             stream=None):
    """out = attention of the new tokens' queries q (tokens x heads x head_dim) over the cache,
    times sigmoid(gate) if given.

    A token sees the positions up to its own (the last `window` of them if window > 0); heads share
    key heads in groups. lse (float32, tokens x heads) receives the log of the sums of exponentials.
    max_q is the largest number of new tokens of a sequence (default: all of them): it picks the
    kernel, not the result."""
    tokens, heads, dim = q.shape
    _need(dim == cache.head_dim and heads % cache.kv_heads == 0,
          "q has %d heads of %d, the cache %d of %d" % (heads, dim, cache.kv_heads, cache.head_dim))
    qs = _heads("q", q, cache, heads, dim)
    os = _heads("out", out, cache, heads, dim, tokens)
    gs = _heads("gate", gate, cache, heads, dim, tokens) if gate is not None else (0, 0)
    if lse is not None:
        _need(lse.dtype == torch.float32 and lse.shape == (tokens, heads) and lse.is_contiguous() and lse.device == cache.device,
              "lse must be a contiguous float32 tensor %d x %d on %s" % (tokens, heads, cache.device))
    _need(ws.buffer.device == cache.device and ws.head_dim >= dim, "the workspace is for head_dim %d on %s" % (ws.head_dim, ws.buffer.device))
    args = _Attn(q.data_ptr(), gate.data_ptr() if gate is not None else None, out.data_ptr(),
                 lse.data_ptr() if lse is not None else None, qs[0], qs[1], gs[0], gs[1], os[0], os[1], heads,
                 max(tokens, 1) if max_q is None else max_q, window, dim ** -0.5 if scale is None else scale)
    batch = _batch(cache, table, q_start, kv_len, tokens)
    _fail(_lib().blk_attn_run(cache._ref, batch, args, ws._ptr, ws.bytes, _raw_stream(stream, cache.device)), "attn_run")


# ------------------------------------------------------------- 4-bit projections

class W4Weight:
    """A 4-bit weight matrix laid out for w4_run; made by w4_prepare."""

    def __init__(self, shape, packed, dtype):
        self.n, self.k, self.group = shape.n, shape.k, shape.group
        self.packed, self.dtype, self.device = packed, dtype, packed.device
        self._ref, self._ptr = ctypes.byref(shape), packed.data_ptr()
        self._shape = shape


def w4_prepare(q, scales, zeros=None, group=128):
    """Lay out n x k 4-bit weights: q uint8 n x k/2 (element 2j in the low nibble of byte j), scales
    n x k/group (BF16 or FP16, the type of the activations), zeros uint8 n x k/group of 0..15
    (None: 8). Runs once and waits; the tensors may be freed afterwards."""
    _need(q.dim() == 2 and q.dtype == torch.uint8 and q.is_contiguous() and q.is_cuda,
          "q must be a contiguous uint8 device tensor n x k/2")
    n, k = q.shape[0], 2 * q.shape[1]
    _need(group in (32, 64, 128) and k % group == 0 and n >= 1 and k >= 1,
          "group %s of k = %d: expected 32, 64 or 128, dividing k" % (group, k))
    _need(scales.dtype in (torch.bfloat16, torch.float16) and scales.shape == (n, k // group) and scales.is_contiguous()
          and scales.device == q.device, "scales must be a contiguous bfloat16 or float16 tensor %d x %d" % (n, k // group))
    _need(zeros is None or (zeros.dtype == torch.uint8 and zeros.shape == scales.shape and zeros.is_contiguous()
                            and zeros.device == q.device), "zeros must be a contiguous uint8 tensor %d x %d" % (n, k // group))
    shape = _W4(n, k, group, DTYPES[scales.dtype], int(zeros is not None))
    packed = torch.empty(_lib().blk_w4_packed_bytes(shape), dtype=torch.uint8, device=q.device)
    stream = torch.cuda.current_stream(q.device)
    _fail(_lib().blk_w4_pack(shape, q.data_ptr(), scales.data_ptr(), zeros.data_ptr() if zeros is not None else None,
                             packed.data_ptr(), stream.cuda_stream), "w4_prepare")
    stream.synchronize()
    return W4Weight(shape, packed, scales.dtype)


def w4_run(w, x, out, stream=None):
    """out (m x n) = x (m x k) @ W^T with 4-bit weights; rows of x and out may be strided."""
    if x.dtype != w.dtype or out.dtype != w.dtype or x.device != w.device or out.device != w.device:
        raise ValueError("x is %s on %s, out %s on %s, the weights %s on %s"
                         % (x.dtype, x.device, out.dtype, out.device, w.dtype, w.device))
    m = x.shape[0]
    if x.dim() != 2 or out.dim() != 2 or x.shape[1] != w.k or out.shape[0] != m or out.shape[1] != w.n:
        raise ValueError("x has shape %s, out %s, expected m x %d and m x %d" % (tuple(x.shape), tuple(out.shape), w.k, w.n))
    xs, os = x.stride(), out.stride()
    if xs[1] != 1 or (os[1] != 1 and w.n > 1):
        raise ValueError("the rows of x and out must be contiguous")
    _fail(_lib().blk_w4_run(w._ref, w._ptr, x.data_ptr(), xs[0], m, out.data_ptr(), os[0],
                            _raw_stream(stream, w.device)), "w4_run")


# ------------------------------------------------------------- norms around a block

def norm_run(x, residual, out, *, weight_pre, weight_post=None, gate=None, alpha=1.0, eps=1e-6, residual_out=None,
             stream=None):
    """residual_out = residual + alpha * gate * rms_norm(x, weight_post); out = rms_norm(residual_out, weight_pre).

    x: a block's output (m x width), or None for the norm before the first block; residual: m x width
    of x's type or float32; gate: width, or m x width; without weight_post x is added as it is.
    residual_out defaults to residual, updated in place."""
    _need(out.dim() == 2 and out.dtype in (torch.bfloat16, torch.float16) and out.is_cuda,
          "out must be a bfloat16 or float16 device tensor m x width")
    m, width = out.shape
    dtype, device = out.dtype, out.device
    _need(residual.dtype in (dtype, torch.float32), "residual has dtype %s, expected %s or float32" % (residual.dtype, dtype))
    if x is None:
        _need(weight_post is None and gate is None and residual_out is None, "weight_post, gate and residual_out need x")
    elif residual_out is None:
        residual_out = residual

    def rows(what, t, kind):
        if t is None:
            return None, 0
        if t.dtype != kind or t.device != device or t.shape != (m, width) or (t.stride(1) != 1 and width > 1):
            raise ValueError("%s must be %s on %s, %d x %d, with contiguous rows" % (what, kind, device, m, width))
        return t.data_ptr(), t.stride(0)

    def vector(what, t):
        if t is None:
            return None
        if t.dtype != dtype or t.device != device or t.shape != (width,) or (t.stride(0) != 1 and width > 1):
            raise ValueError("%s must be a contiguous %s vector of %d on %s" % (what, dtype, width, device))
        return t.data_ptr()

    _need(weight_pre is not None, "weight_pre is needed")
    xp, xs = rows("x", x, dtype)
    rp, rs = rows("residual", residual, residual.dtype)
    yp, ys = rows("residual_out", residual_out, residual.dtype)
    op, os = rows("out", out, dtype)
    if gate is not None and gate.dim() == 1:
        gp, gs = vector("gate", gate), 0
    else:
        gp, gs = rows("gate", gate, dtype)
    args = _Norm(xp, rp, gp, vector("weight_post", weight_post), vector("weight_pre", weight_pre), yp, op,
                 xs, rs, gs, ys, os, width, DTYPES[dtype], DTYPES[residual.dtype], alpha, eps)
    _fail(_lib().blk_norm_run(args, m, _raw_stream(stream, device)), "norm_run")
