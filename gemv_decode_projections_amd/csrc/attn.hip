// C ABI of the paged cache and the attention over it (include/block.h):
// checks, the choice of the kernel, launches; and the two cache kernels.
#include <math.h>

#include <algorithm>
#include <new>
#include <vector>

#include "attn.h"

namespace gdp {
namespace {

// One 16-byte piece of a new token's key or value per thread: a pure copy,
// bound by the launch at decode sizes (16 tokens: 2.2 us on the GPU) and by HBM
// at a prompt's (3488 tokens of 8 heads, 28.6 MB: 6.7 us a call, 4.3 TB/s).
struct AppendArgs {
    AttnArgs a;
    const char *k, *v;
    int64_t in_stride, in_head;        // bytes
    int64_t total;                     // 16-byte pieces of k
    int per_head;                      // of them in a head
    Divisor by_token, by_head;         // of the pieces of a token, of a head
};

__global__ __launch_bounds__(256) void kv_append_kernel(AppendArgs x)
{
    const AttnArgs &a = x.a;
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= x.total)
        return;
    const int per_head = x.per_head, per_token = per_head * a.kv_heads;
    const int tok = x.by_token((int)id);
    const int piece = (int)id - tok * per_token;
    const int head = x.by_head(piece);
    const int at = (piece - head * per_head) * 16;
    // The token's sequence: the last whose first row is not past it.
    int lo = 0, hi = a.seqs;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (a.q_start[mid] <= tok)
            lo = mid;
        else
            hi = mid - 1;
    }
    if (lo >= a.seqs)
        return;
    int tok0, n, len;
    seq_bounds(a, lo, tok0, n, len);
    const int pos = len - n + tok - tok0;
    if (tok < tok0 || tok >= tok0 + n || pos < 0)
        return;
    int64_t off;
    if (!kv_offset(a, a.table[lo * a.table_stride + (pos >> a.page_shift)], pos, (int64_t)head * a.head_stride, off))
        return;
    const int64_t from = tok * x.in_stride + head * x.in_head + at;
    const u32x4 k = *reinterpret_cast<const u32x4 *>(x.k + from);
    const u32x4 v = *reinterpret_cast<const u32x4 *>(x.v + from);
    *reinterpret_cast<u32x4 *>(const_cast<char *>(a.k) + off + at) = k;
    *reinterpret_cast<u32x4 *>(const_cast<char *>(a.v) + off + at) = v;
}

// Page pairs travel in the kernel's arguments: no device list to allocate,
// copy or keep alive, and a graph keeps its own. Page numbers of 16 bits fit
// twice as many in the 4 KB that a launch takes (1500 moves of 64 KB pages: two
// launches instead of four: 50 us a call, 4 TB/s).
template <class I>
struct CopyArgs {
    static constexpr int kPairs = 1792 / sizeof(I);
    char *k, *v;
    int64_t page_stride;       // bytes
    int page_bytes;
    I src[kPairs], dst[kPairs];
};

constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;         // 16-byte pieces per thread, all loads in flight

template <class I>
__global__ __launch_bounds__(kCopyThreads) void kv_copy_kernel(CopyArgs<I> a)
{
    char *base = blockIdx.z ? a.v : a.k;
    const char *src = base + a.src[blockIdx.y] * a.page_stride;
    char *dst = base + a.dst[blockIdx.y] * a.page_stride;
    const int at = (blockIdx.x * kCopyThreads * kCopyUnroll + threadIdx.x) * 16;
    u32x4 x[kCopyUnroll];
#pragma unroll
    for (int i = 0; i < kCopyUnroll; ++i)
        if (at + i * kCopyThreads * 16 < a.page_bytes)
            x[i] = *reinterpret_cast<const u32x4 *>(src + at + i * kCopyThreads * 16);
#pragma unroll
    for (int i = 0; i < kCopyUnroll; ++i)
        if (at + i * kCopyThreads * 16 < a.page_bytes)
            *reinterpret_cast<u32x4 *>(dst + at + i * kCopyThreads * 16) = x[i];
}

constexpr int kJoinGrid = 2048;        // workgroups of the join kernel, which loop over the rows

constexpr int64_t kMaxOffset = (int64_t)1 << 31;

bool stride_ok(int64_t s) { return s >= 0 && s % 8 == 0 && s < ((int64_t)1 << 40); }

int check_cache(const blk_cache *c)
{
    if (!c || !c->k || !c->v)
        return PROJ_ERR_NULL;
    if (!aligned_to(c->k, 16) || !aligned_to(c->v, 16))
        return PROJ_ERR_ALIGN;
    if (c->dtype != BLK_BF16 && c->dtype != BLK_F16)
        return PROJ_ERR_ARG;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
        return PROJ_ERR_ARG;
    if (c->n_pages < 1 || c->kv_heads < 1 || c->kv_heads > 65535 || c->page_size < 8 ||
        (c->page_size & (c->page_size - 1)))
        return PROJ_ERR_ARG;
    const int64_t page = stride_of(c->page_stride, c->n_pages), head = stride_of(c->head_stride, c->kv_heads);
    if (!stride_ok(page) || !stride_ok(c->token_stride) || !stride_ok(head) || page >= kMaxOffset ||
        c->token_stride >= kMaxOffset / 2 || head >= kMaxOffset / 2 ||
        (c->page_size - 1) * c->token_stride + (c->kv_heads - 1) * head + c->head_dim > kMaxOffset)
        return PROJ_ERR_ARG;
    return PROJ_OK;
}

int check_batch(const blk_batch *b)
{
    if (!b)
        return PROJ_ERR_NULL;
    if (b->seqs < 0 || b->tokens < 0 || b->table_width < 1 || (b->table_stride && b->table_stride < b->table_width))
        return PROJ_ERR_ARG;
    if (b->seqs && b->tokens && (!b->q_start || !b->kv_len || !b->table))
        return PROJ_ERR_NULL;
    if (!aligned_to(b->q_start, 4) || !aligned_to(b->kv_len, 4) || !aligned_to(b->table, 4))
        return PROJ_ERR_ALIGN;
    return PROJ_OK;
}

AttnArgs base_args(const blk_cache *c, const blk_batch *b)
{
    AttnArgs a{};
    a.k = static_cast<const char *>(c->k);
    a.v = static_cast<const char *>(c->v);
    a.page_stride = (uint32_t)(stride_of(c->page_stride, c->n_pages) * 2);
    a.token_stride = (int)(c->token_stride * 2);
    a.head_stride = (int)(stride_of(c->head_stride, c->kv_heads) * 2);
    a.n_pages = c->n_pages;
    a.page_shift = __builtin_ctz((unsigned)c->page_size);
    a.page_mask = c->page_size - 1;
    a.kv_heads = c->kv_heads;
    a.q_start = b->q_start;
    a.kv_len = b->kv_len;
    a.table = b->table;
    a.table_stride = b->table_stride;
    a.table_width = b->table_width;
    a.seqs = b->seqs;
    a.tokens = b->tokens;
    return a;
}

int launch(const void *fn, dim3 grid, dim3 block, void *arg, void *stream)
{
    void *params[1] = {arg};
    const hipError_t e = hipLaunchKernel(fn, grid, block, params, 0, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? PROJ_OK : hip_fail(e);
}

// Up to n page numbers, in a table of their own number, not the cache's: a fork
// of one page costs the same in a cache of any size.
class PageSet {
    std::vector<uint32_t> slots;       // page + 1, or 0
    int shift;

    size_t find(uint32_t key) const    // the key's slot, or the free one for it
    {
        size_t i = (key * 2654435769u) >> shift;
        while (slots[i] && slots[i] != key)
            i = (i + 1) & (slots.size() - 1);
        return i;
    }

public:
    explicit PageSet(int n)
    {
        int bits = 2;
        while (((int64_t)1 << bits) < 2 * (int64_t)n)
            ++bits;
        slots.assign((size_t)1 << bits, 0);
        shift = 32 - bits;
    }
    bool has(int32_t page) const { return slots[find((uint32_t)page + 1)] != 0; }
    bool add(int32_t page)             // false if it was there
    {
        uint32_t &slot = slots[find((uint32_t)page + 1)];
        const bool fresh = !slot;
        slot = (uint32_t)page + 1;
        return fresh;
    }
};

template <class I>
int copy_pages(const blk_cache *cache, const int32_t *src, const int32_t *dst, int n, int64_t elems, void *stream)
{
    typedef CopyArgs<I> Args;
    Args a{};
    a.k = static_cast<char *>(cache->k);
    a.v = static_cast<char *>(cache->v);
    a.page_stride = cache->page_stride * 2;
    a.page_bytes = (int)(elems * 2);
    const int per_wg = kCopyThreads * kCopyUnroll * 16;
    for (int i = 0; i < n; i += Args::kPairs) {
        const int c = std::min(Args::kPairs, n - i);
        std::copy(src + i, src + i + c, a.src);
        std::copy(dst + i, dst + i + c, a.dst);
        const int rc = launch(reinterpret_cast<const void *>(kv_copy_kernel<I>),
                              dim3((unsigned)((a.page_bytes + per_wg - 1) / per_wg), c, 2), dim3(kCopyThreads), &a, stream);
        if (rc)
            return rc;
    }
    return PROJ_OK;
}

}  // namespace
}  // namespace gdp

using namespace gdp;

extern "C" {

int blk_kv_append(const blk_cache *cache, const blk_batch *batch, const void *k, const void *v, int64_t in_stride,
                  int64_t in_head_stride, void *stream)
{
    int rc = check_cache(cache);
    if (rc == PROJ_OK)
        rc = check_batch(batch);
    if (rc)
        return rc;
    in_stride = stride_of(in_stride, batch->tokens);
    in_head_stride = stride_of(in_head_stride, cache->kv_heads);
    if (!stride_ok(in_stride) || !stride_ok(in_head_stride) ||
        !rows_apart<3>(cache->head_dim, {cache->page_stride, cache->token_stride, cache->head_stride},
                       {cache->n_pages, cache->page_size, cache->kv_heads}))
        return PROJ_ERR_ARG;
    if (!batch->seqs || !batch->tokens)
        return PROJ_OK;
    if (!k || !v)
        return PROJ_ERR_NULL;
    if (!aligned_to(k, 16) || !aligned_to(v, 16))
        return PROJ_ERR_ALIGN;
    AppendArgs x{};
    x.a = base_args(cache, batch);
    x.per_head = cache->head_dim / 8;
    const int64_t per_token = (int64_t)x.per_head * cache->kv_heads;
    x.total = batch->tokens * per_token;
    if (x.total > 0x7fffffff)
        return PROJ_ERR_ARG;
    x.by_token = Divisor::of((uint32_t)per_token);
    x.by_head = Divisor::of((uint32_t)x.per_head);
    x.k = static_cast<const char *>(k);
    x.v = static_cast<const char *>(v);
    x.in_stride = in_stride * 2;
    x.in_head = in_head_stride * 2;
    return launch(reinterpret_cast<const void *>(kv_append_kernel), dim3((unsigned)((x.total + 255) / 256)), dim3(256), &x,
                  stream);
}

int blk_kv_copy_pages(const blk_cache *cache, const int32_t *src, const int32_t *dst, int n, void *stream)
{
    const int rc = check_cache(cache);
    if (rc)
        return rc;
    if (n < 0)
        return PROJ_ERR_ARG;
    if (n == 0)
        return PROJ_OK;
    if (!src || !dst)
        return PROJ_ERR_NULL;
    // One dense block per page: the two inner strides are the two ways to
    // order tokens and heads.
    const int64_t elems = (int64_t)cache->page_size * cache->kv_heads * cache->head_dim;
    const bool token_major = (cache->head_stride == cache->head_dim || cache->kv_heads == 1) &&
                             cache->token_stride == (int64_t)cache->kv_heads * cache->head_dim;
    const bool head_major = cache->token_stride == cache->head_dim &&
                            (cache->head_stride == (int64_t)cache->page_size * cache->head_dim || cache->kv_heads == 1);
    if (!(token_major || head_major) || elems * 2 > (1 << 30) || (cache->n_pages > 1 && cache->page_stride < elems))
        return PROJ_ERR_ARG;
    try {
        // A page is written once at most, and none both read and written.
        PageSet written(n);
        for (int i = 0; i < n; ++i)
            if (src[i] < 0 || src[i] >= cache->n_pages || dst[i] < 0 || dst[i] >= cache->n_pages || !written.add(dst[i]))
                return PROJ_ERR_ARG;
        for (int i = 0; i < n; ++i)
            if (written.has(src[i]))
                return PROJ_ERR_ARG;
    } catch (const std::bad_alloc &) {
        return PROJ_ERR_HIP;
    }
    return cache->n_pages <= 65536 ? copy_pages<uint16_t>(cache, src, dst, n, elems, stream)
                                   : copy_pages<int32_t>(cache, src, dst, n, elems, stream);
}

size_t blk_attn_workspace_bytes(int head_dim) { return head_dim > 0 && head_dim <= 256 ? attn_ws_bytes(head_dim) : 0; }

int blk_attn_run(const blk_cache *cache, const blk_batch *batch, const blk_attn_args *args, void *ws, size_t ws_bytes,
                 void *stream)
{
    int rc = check_cache(cache);
    if (rc == PROJ_OK)
        rc = check_batch(batch);
    if (rc)
        return rc;
    if (!args)
        return PROJ_ERR_NULL;
    if (args->heads < 1 || args->heads % cache->kv_heads || args->max_q < 1 || args->window < 0 ||
        !(args->scale > 0.f) || !isfinite(args->scale))
        return PROJ_ERR_ARG;
    auto token_stride = [&](int64_t s) { return stride_of(s, batch->tokens); };
    auto head_stride = [&](int64_t s) { return stride_of(s, args->heads); };
    for (int64_t s : {token_stride(args->q_stride), token_stride(args->gate_stride), token_stride(args->out_stride),
                      head_stride(args->q_head_stride), head_stride(args->gate_head_stride), head_stride(args->out_head_stride)})
        if (!stride_ok(s))
            return PROJ_ERR_ARG;
    if (!rows_apart<2>(cache->head_dim, {args->out_stride, args->out_head_stride}, {batch->tokens, args->heads}))
        return PROJ_ERR_ARG;
    if (!batch->seqs || !batch->tokens)
        return PROJ_OK;
    if (!args->q || !args->out || !ws)
        return PROJ_ERR_NULL;
    if (!aligned_to(args->q, 16) || !aligned_to(args->out, 16) || !aligned_to(args->gate, 16) ||
        !aligned_to(args->lse, 4) || !aligned_to(ws, 256))
        return PROJ_ERR_ALIGN;
    if (ws_bytes < attn_ws_bytes(cache->head_dim))
        return PROJ_ERR_SCRATCH;
    // Row counts, positions and tile counts are kept in 32 bits.
    const int64_t rows = (int64_t)batch->tokens * (args->heads / cache->kv_heads);
    if (rows > 0x3fffffff || ((int64_t)batch->table_width << __builtin_ctz((unsigned)cache->page_size)) > 0x3fffffff)
        return PROJ_ERR_ARG;

    AttnArgs a = base_args(cache, batch);
    a.q = static_cast<const char *>(args->q);
    a.gate = static_cast<const char *>(args->gate);
    a.out = static_cast<char *>(args->out);
    a.lse = args->lse;
    a.q_stride = token_stride(args->q_stride) * 2;
    a.q_head = head_stride(args->q_head_stride) * 2;
    a.gate_stride = token_stride(args->gate_stride) * 2;
    a.gate_head = head_stride(args->gate_head_stride) * 2;
    a.out_stride = token_stride(args->out_stride) * 2;
    a.out_head = head_stride(args->out_head_stride) * 2;
    a.heads = args->heads;
    a.group = args->heads / cache->kv_heads;
    a.by_group = Divisor::of(a.group);
    a.by_heads = Divisor::of(a.kv_heads);
    a.window = std::min(args->window, 0x3fffffff);
    a.scale_log2 = args->scale * 1.44269504f;
    a.counters = static_cast<uint32_t *>(ws);
    a.slots = static_cast<char *>(ws) + kAttnCounterBytes;

    const int64_t seq_rows = (int64_t)std::min(args->max_q, batch->tokens) * a.group;
    // Up to 32 rows per sequence and key head take the row kernel, which holds
    // keys and values in registers; more take the tile kernel.
    // The row kernel counts the joins of its tiles of 16 rows itself; the
    // others' are a second launch.
    const void *fn, *join = nullptr;
    int tile, threads;
    a.rounds = 1;
    if (seq_rows <= 32) {
        const int nb = seq_rows <= 16 ? 1 : 2;
        tile = 16 * nb;
        threads = 256;
        a.kv_step = 128;
        a.min_split = 128;
        // Two workgroups per compute unit; one where a head's 256 elements
        // take all registers, four of 64 elements.
        a.target = cache->head_dim == 64 ? 1024 : cache->head_dim == 128 ? 512 : 256;
        a.rounds = 4 / nb;
        fn = reinterpret_cast<const void *>(attn_rows_kernel(cache->dtype, cache->head_dim, nb));
    } else {
        tile = seq_rows <= 64 ? 64 : 128;
        threads = 2 * tile;
        a.kv_step = 64;
        a.min_split = 256;
        // Two workgroups per compute unit; one where a head's 256 elements
        // take all registers.
        a.target = cache->head_dim == 256 ? 256 : 512;
        fn = reinterpret_cast<const void *>(attn_tile_kernel(cache->dtype, cache->head_dim, tile));
    }
    if (tile > 16)
        join = reinterpret_cast<const void *>(attn_join_kernel(cache->dtype, cache->head_dim, tile));
    a.per_target = 1.0f / (float)a.target;
    // Units: one per row tile and key head, and at most `target` more, times
    // the rounds if the most work there can be asks for them (2047: the kernels
    // compare with 2048 in FP32, rounded up).
    const int64_t tiles = (rows / tile + batch->seqs) * a.kv_heads;
    const int64_t positions = (int64_t)batch->table_width * cache->page_size;
    const int64_t more =
        tiles * positions >= (int64_t)2047 * a.target || tiles > a.target / 2 ? a.target * a.rounds : a.target;
    const int64_t grid = (std::min(tiles + more, tiles * ((positions + a.min_split - 1) / a.min_split)) + 7) / 8 * 8;
    if (grid > 0x7fffffff)
        return PROJ_ERR_ARG;
    rc = launch(fn, dim3((unsigned)grid), dim3(threads), &a, stream);
    // No range can be split if the longest one is not longer than a part.
    if (rc || !join || positions <= a.min_split)
        return rc;
    return launch(join, dim3((unsigned)std::min<int64_t>(rows * a.kv_heads, kJoinGrid)), dim3(kJoinThreads), &a, stream);
}

}  // extern "C"
