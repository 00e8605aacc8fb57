"""Python binding of the C ABI in include/block.h: the operators between the
projections of a decode block.

    cache = KvCache.empty(n_pages, 16, kv_heads, head_dim)
    kv_append(k, v, cache, table, q_start, kv_len)
    attn_run(q, cache, table, q_start, kv_len, out, AttnWorkspace(head_dim), max_q=1)

Argument marshalling and checks only, as in `binding`: the work runs in the HIP
library, on the stream given or torch's current one. Calls launch and return;
nothing is allocated, synchronized or copied to the host. The run functions'
checks are compiled (csrc/block_py.cpp): a tensor of the wrong shape, type,
device or layout raises ValueError before anything is launched, what the
library itself refuses raises ProjError (PROJ_ERR_DEVICE: the tensors are on
one GPU, and another is current).
"""

import array
import ctypes
import importlib.machinery
import importlib.util
import os

import torch

from . import binding as _b

_i, _i64, _vp = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p
_pages = ctypes.POINTER(ctypes.c_int32)

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
HEAD_DIMS = (64, 128, 256)
ATTN_ZEROED = 32768        # BLK_ATTN_ZEROED
EXT_PATH = os.path.join(os.path.dirname(_b.LIB_PATH), "_block.so")


class _Cache(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("page_stride", _i64), ("token_stride", _i64), ("head_stride", _i64),
                ("n_pages", _i), ("page_size", _i), ("kv_heads", _i), ("head_dim", _i), ("dtype", _i),
                ("_end", _i), ("device", _i)]        # (behind blk_cache: the GPU, for the compiled checks)


class _W4(ctypes.Structure):
    _fields_ = [("n", _i), ("k", _i), ("group", _i), ("dtype", _i), ("has_zeros", _i),
                ("device", _i)]                      # (behind blk_w4)


_LIB = None
_EXT = None


def _lib():
    """The library with the signatures of block.h's other functions set."""
    global _LIB
    if _LIB is None:
        lib = _b._lib()
        shape = ctypes.POINTER(_W4)
        sig = {
            "blk_attn_workspace_bytes": ([_i], ctypes.c_size_t),
            "blk_pool_create": ([_i, ctypes.POINTER(_vp)], _i),
            "blk_pool_destroy": ([_vp], None),
            "blk_pool_free_pages": ([_vp], _i),
            "blk_pool_users": ([_vp, ctypes.c_int32], _i),
            "blk_pool_alloc": ([_vp, _i, _pages], _i),
            "blk_pool_share": ([_vp, _pages, _i], _i),
            "blk_pool_release": ([_vp, _pages, _i], _i),
            "blk_pool_compact": ([_vp, _i, _pages, _pages], _i),
            "blk_w4_packed_bytes": ([shape], ctypes.c_size_t),
            "blk_w4_pack": ([shape, _vp, _vp, _vp, _vp, _vp], _i),
        }
        for name, (args, res) in sig.items():
            f = getattr(lib, name)
            f.argtypes = args
            f.restype = res
        _LIB = lib
    return _LIB


def _ext():
    """The compiled run functions."""
    global _EXT
    if _EXT is None:
        _lib()
        if not os.path.exists(EXT_PATH):
            raise RuntimeError("%s is not built; run `python -m gemv_decode_projections_amd.build` first" % EXT_PATH)
        loader = importlib.machinery.ExtensionFileLoader("_block", EXT_PATH)
        _EXT = importlib.util.module_from_spec(importlib.util.spec_from_loader("_block", loader))
        loader.exec_module(_EXT)
    return _EXT


def _raw_stream(stream, index):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    if isinstance(stream, int):
        return stream
    _need(stream.device_index == index, "the stream is of GPU %d, the tensors are on GPU %d" % (stream.device_index, index))
    return stream.cuda_stream


def _fail(rc, what):
    if rc != _b.PROJ_OK:
        raise _b.ProjError(rc, what)


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _int32(what, n):
    """n as the library takes it (a C conversion would drop the upper bits)."""
    _need(hasattr(n, "__index__") and -2 ** 31 <= n < 2 ** 31, "%s must be an integer of 32 bits, not %r" % (what, n))
    return int(n)


def _page_list(pages):
    try:
        a = array.array("i", pages)
    except (OverflowError, TypeError) as e:
        raise ValueError("page numbers must be integers of 32 bits: %s" % e) from None
    return (ctypes.c_int32 * len(a)).from_buffer(a) if len(a) else (ctypes.c_int32 * 0)()


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
        self._c = _Cache(k.data_ptr(), v.data_ptr(), s[0], s[1], s[2], pages, size, heads, dim, DTYPES[k.dtype],
                         0, k.device.index)
        self._addr, self._index = ctypes.addressof(self._c), k.device.index

    @classmethod
    def empty(cls, n_pages, page_size, kv_heads, head_dim, dtype=torch.bfloat16, device="cuda"):
        """A cache of uninitialised pages (what no token was written to is never used)."""
        shape = (n_pages, page_size, kv_heads, head_dim)
        return cls(torch.empty(shape, dtype=dtype, device=device), torch.empty(shape, dtype=dtype, device=device))


def kv_append(k, v, cache, table, q_start, kv_len, stream=None):
    """Write the new tokens' keys and values (tokens x kv_heads x head_dim) into their pages.

    k and v may be views of a projection's output, with the same strides.
    table (seqs x pages), q_start (seqs + 1) and kv_len (seqs, the new tokens included) are int32 on
    the device; a token at a negative position or on an unmapped page is not written."""
    rc = _ext().kv_append(cache._addr, k, v, table, q_start, kv_len, _raw_stream(stream, cache._index))
    if rc:
        _fail(rc, "kv_append")


def kv_copy_pages(cache, src, dst, stream=None):
    """Copy page src[i] to page dst[i], keys and values (sequences of page numbers; no page twice in
    dst, none in both)."""
    rc = _ext().kv_copy_pages(cache._addr, src, dst, _raw_stream(stream, cache._index))
    if rc:
        _fail(rc, "kv_copy_pages")


class PagePool:
    """Which pages of a cache are in use, and by how many sequences (host memory only).

    A sequence is the caller's list of pages. fork shares them; a page to be written that other
    sequences use too is first replaced by writable(), which says what to copy."""

    def __init__(self, n_pages):
        self.n_pages = _int32("n_pages", int(n_pages))
        handle = _vp()
        _fail(_lib().blk_pool_create(self.n_pages, ctypes.byref(handle)), "PagePool(%d)" % self.n_pages)
        self._handle = handle

    def __del__(self):
        handle, self._handle = getattr(self, "_handle", None), None
        if handle and _LIB is not None:
            _LIB.blk_pool_destroy(handle)

    @property
    def free_pages(self):
        return _lib().blk_pool_free_pages(self._handle)

    def users(self, page):
        n = _lib().blk_pool_users(self._handle, _int32("page", page))
        _fail(min(n, 0), "users(%d)" % page)
        return n

    def alloc(self, n):
        """The n lowest free pages; ProjError (PROJ_ERR_PAGES), and none taken, if there are fewer."""
        pages = (ctypes.c_int32 * max(_int32("n", n), 0))()
        _fail(_lib().blk_pool_alloc(self._handle, n, pages), "alloc(%d)" % n)
        return list(pages)

    def fork(self, pages):
        """Another sequence's list of the same pages: each gets one more user."""
        _fail(_lib().blk_pool_share(self._handle, _page_list(pages), len(pages)), "fork")
        return list(pages)

    def free(self, pages):
        """Takes one user from each page; pages without users are free again."""
        _fail(_lib().blk_pool_release(self._handle, _page_list(pages), len(pages)), "free")

    def writable(self, pages, index):
        """Makes pages[index] this sequence's own before a write: (old, new) to be copied if others
        use it too (the list then names new), None if they do not."""
        old = pages[index]
        users = self.users(old)
        _need(users > 0, "page %d is not in use" % old)
        if users == 1:
            return None
        new = self.alloc(1)[0]
        self.free([old])
        pages[index] = new
        return old, new

    def compact(self, max_moves=None):
        """Moves of pages down into free ones: (src, dst), as kv_copy_pages takes them. Replace src[i]
        by dst[i] in every page list (remap) and table."""
        n = self.n_pages if max_moves is None else _int32("max_moves", max_moves)
        src, dst = (ctypes.c_int32 * max(n, 0))(), (ctypes.c_int32 * max(n, 0))()
        moves = _lib().blk_pool_compact(self._handle, n, src, dst)
        _fail(min(moves, 0), "compact(%s)" % max_moves)
        return src[:moves], dst[:moves]

    @staticmethod
    def remap(pages, src, dst):
        """The page list after the moves."""
        to = dict(zip(src, dst))
        return [to.get(p, p) for p in pages]


class AttnWorkspace:
    """Scratch of attn_run for one head_dim, ready for any batch. Calls that can overlap (other
    streams) need workspaces of their own."""

    def __init__(self, head_dim, device="cuda"):
        _need(head_dim in HEAD_DIMS, "head_dim %d, expected one of %s" % (head_dim, HEAD_DIMS))
        self.head_dim = head_dim
        self.bytes = _lib().blk_attn_workspace_bytes(head_dim)
        self.buffer = torch.empty(self.bytes, dtype=torch.uint8, device=device)
        self.buffer[:ATTN_ZEROED].zero_()
        # Any stream may use it from here on.
        torch.cuda.current_stream(self.buffer.device).synchronize()
        self._ptr, self.index = self.buffer.data_ptr(), self.buffer.device.index


def attn_run(q, cache, table, q_start, kv_len, out, ws, *, max_q=None, scale=None, window=0, gate=None, lse=None,
             stream=None):
    """out = attention of the new tokens' queries q (tokens x heads x head_dim) over the cache,
    times sigmoid(gate) if given.

    A token sees the positions up to its own (the last `window` of them if window > 0); heads share
    key heads in groups. Tokens of no sequence (from q_start[-1] on) are left as they are. lse (float32,
    tokens x heads) receives the log of the sums of exponentials.
    max_q is the largest number of new tokens of a sequence (default: all of them): it picks the
    kernel, not the result."""
    if ws.head_dim < cache.head_dim or ws.index != cache._index:
        raise ValueError("the workspace is for head_dim %d on GPU %d" % (ws.head_dim, ws.index))
    rc = _ext().attn_run(cache._addr, ws._ptr, ws.bytes, q, table, q_start, kv_len, out, gate, lse, max_q, scale, window,
                         _raw_stream(stream, cache._index))
    if rc:
        _fail(rc, "attn_run")


# ------------------------------------------------------------- 4-bit projections

class W4Weight:
    """A 4-bit weight matrix laid out for w4_run; made by w4_prepare."""

    def __init__(self, shape, packed, dtype):
        self.n, self.k, self.group = shape.n, shape.k, shape.group
        self.packed, self.dtype, self.device = packed, dtype, packed.device
        self._addr, self._ptr, self._index = ctypes.addressof(shape), packed.data_ptr(), packed.device.index
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
    shape = _W4(n, k, group, DTYPES[scales.dtype], int(zeros is not None), q.device.index)
    packed = torch.empty(_lib().blk_w4_packed_bytes(shape), dtype=torch.uint8, device=q.device)
    stream = torch.cuda.current_stream(q.device)
    with torch.cuda.device(q.device):
        _fail(_lib().blk_w4_pack(shape, q.data_ptr(), scales.data_ptr(), zeros.data_ptr() if zeros is not None else None,
                                 packed.data_ptr(), stream.cuda_stream), "w4_prepare")
    stream.synchronize()
    return W4Weight(shape, packed, scales.dtype)


def w4_run(w, x, out, stream=None):
    """out (m x n) = x (m x k) @ W^T with 4-bit weights; rows of x and out may be strided."""
    rc = _ext().w4_run(w._addr, w._ptr, x, out, _raw_stream(stream, w._index))
    if rc:
        _fail(rc, "w4_run")


# ------------------------------------------------------------- norms around a block

def norm_run(x, residual, out, *, weight_pre, weight_post=None, gate=None, alpha=1.0, eps=1e-6, residual_out=None,
             stream=None):
    """residual_out = residual + alpha * gate * rms_norm(x, weight_post); out = rms_norm(residual_out, weight_pre).

    x: a block's output (m x width), or None for the norm before the first block; residual: m x width
    of x's type or float32; gate: width, or m x width; without weight_post x is added as it is.
    residual_out defaults to residual, updated in place."""
    rc = _ext().norm_run(x, residual, out, weight_pre, weight_post, gate, alpha, eps, residual_out,
                         _raw_stream(stream, out.device.index) if out.is_cuda else 0)
    if rc:
        _fail(rc, "norm_run")
