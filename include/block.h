/*
 * block.h - C ABI of the operators that sit between the projections of a
 * decode block (proj.h): keys and values into a paged cache, attention over
 * that cache, the cache's pages, projections with 4-bit weights, and the
 * norms around a block.
 *
 * Conventions are those of proj.h: device pointers of the current device,
 * streams as void * (NULL = the null stream), PROJ_OK (0) or a negative
 * proj_status returned, no function aborts the process. Every run function
 * only launches: no allocation, no synchronization, no host read of device
 * memory, safe to capture in a HIP graph. Arguments that the host can see are
 * checked before the launch (PROJ_ERR_NULL, PROJ_ERR_ALIGN, PROJ_ERR_ARG);
 * lengths, page tables and offsets live on the device and are bounded by the
 * kernels themselves, so no value in them makes a kernel leave its buffers.
 * Strides are in elements; the stride of a dimension with one entry is not
 * looked at. Rows that a call writes must not overlap (PROJ_ERR_ARG); those
 * that it only reads may. The library keeps no state between calls: what a
 * call needs beyond its tensors is a buffer of the caller.
 */
#ifndef BLOCK_H
#define BLOCK_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
enum blk_dtype { BLK_BF16 = 0, BLK_F16 = 1, BLK_F32 = 2 };

/*
 * A paged cache: n_pages pages of page_size tokens of kv_heads heads of
 * head_dim elements, keys and values in two tensors of one layout. Element
 * (page, token, head, d) of either lies at
 *     page * page_stride + token * token_stride + head * head_stride + d
 * elements past its pointer, so token-major and head-major pages, and keys
 * and values interleaved in one tensor, are all described.
 *   page_size  a power of two, at least 8
 *   head_dim   64, 128 or 256
 *   dtype      BLK_BF16 or BLK_F16
 *   strides    multiples of 8 elements, non-negative; page_stride below 2^31,
 *              offsets inside a page below 2^31 (the cache itself may be of
 *              any size: offsets are computed in 64 bits)
 *   pointers   16-byte aligned
 */
typedef struct {
    void *k;
    void *v;
    int64_t page_stride, token_stride, head_stride;
    int n_pages, page_size, kv_heads, head_dim, dtype;
} blk_cache;

/*
 * The new tokens of a step and where they stand: seqs sequences, whose new
 * tokens are rows q_start[b] .. q_start[b + 1] - 1 of the token-major
 * tensors (tokens rows in all). kv_len[b] counts sequence b's cached tokens,
 * the new ones included, so new token i of n stands at position
 * kv_len[b] - n + i. Position p is in page table[b * table_stride + p /
 * page_size]; a table entry outside 0 .. n_pages - 1 holds no tokens (a page
 * already given back, say, outside an attention window). A table_stride of 0
 * gives all sequences one row; otherwise rows do not overlap (PROJ_ERR_ARG).
 * All three arrays are int32 on the device. Values are bounded where they
 * are read: kv_len to 0 .. table_width * page_size, q_start to 0 .. tokens.
 * q_start does not descend; if it does, it is unspecified whose new tokens
 * are whose, but not that they are within the tensors. Rows of no sequence
 * (before q_start[0], from q_start[seqs] on) are neither read nor written.
 */
typedef struct {
    const int32_t *q_start;     /* seqs + 1 */
    const int32_t *kv_len;      /* seqs */
    const int32_t *table;       /* seqs x table_width, rows table_stride apart */
    int64_t table_stride;
    int table_width, seqs, tokens;
} blk_batch;

/*
 * blk_kv_append - write the new tokens' keys and values into their pages.
 * k, v: tokens x kv_heads x head_dim of the cache's type, rows in_stride
 * (tokens) and in_head_stride (heads) elements apart, multiples of 8, 16-byte
 * aligned pointers; views into a projection's output are fine. Tokens whose
 * position is negative or whose page is not in the cache are not written.
 * Two sequences must not append to one page.
 */
int blk_kv_append(const blk_cache *cache, const blk_batch *batch, const void *k, const void *v, int64_t in_stride,
                  int64_t in_head_stride, void *stream);

/*
 * blk_kv_copy_pages - copy whole pages of keys and values, dst[i] = src[i]
 * for n pairs (host arrays, read during the call). For forking a sequence
 * (its last, partly filled page) and for compacting a cache. A page must be
 * one dense block of page_size * kv_heads * head_dim elements, in any order
 * inside (PROJ_ERR_ARG otherwise); page numbers must be in range, no page
 * may be written twice and none both read and written (PROJ_ERR_ARG): the
 * copies of one call run at once.
 */
int blk_kv_copy_pages(const blk_cache *cache, const int32_t *src, const int32_t *dst, int n, void *stream);

/*
 * Page pool: which pages of a cache are in use, on the host. A page has a
 * number of users: alloc gives it one, share (a fork: the sequences share the
 * page) adds one, release takes one away, and without users it is free. alloc
 * takes the lowest free pages. share and release do all or nothing:
 * PROJ_ERR_ARG if a page is not in use (or released more often than used).
 * PROJ_ERR_PAGES if fewer than n pages are free (none is taken then).
 *
 * blk_pool_compact moves pages from the top of the cache to free pages below:
 * up to max_moves pairs into src and dst, returns their number (0: nothing to
 * move, every page in use lies below every free one). The pool counts the
 * pages as moved; the caller copies them (blk_kv_copy_pages takes the pairs as
 * they are) and replaces src[i] by dst[i] in its page tables.
 *
 * Calls on one pool must not race each other.
 */
typedef struct blk_pool blk_pool;

int blk_pool_create(int n_pages, blk_pool **pool);
void blk_pool_destroy(blk_pool *pool);
int blk_pool_free_pages(const blk_pool *pool);
int blk_pool_users(const blk_pool *pool, int32_t page);
int blk_pool_alloc(blk_pool *pool, int n, int32_t *pages);
int blk_pool_share(blk_pool *pool, const int32_t *pages, int n);
int blk_pool_release(blk_pool *pool, const int32_t *pages, int n);
int blk_pool_compact(blk_pool *pool, int max_moves, int32_t *src, int32_t *dst);

/*
 * blk_attn_run - attention of the new tokens over the cache:
 *     out[t, h] = sum_j softmax_j(scale * q[t, h] . K[j]) V[j]   [* sigmoid(gate[t, h])]
 * over the positions j that token t sees: j <= its own position, and with
 * window > 0 only the last `window` positions, its own included. Query head
 * h reads key head h / (heads / kv_heads). A token that sees nothing gives 0.
 *   q, gate, out: tokens x heads x head_dim of the cache's type; token and
 *       head strides in elements, multiples of 8; pointers 16-byte aligned.
 *       gate may be NULL.
 *   lse: NULL, or float32 tokens x heads (contiguous): ln sum_j exp(scale *
 *       q . K[j]), -inf for a token that sees nothing.
 *   A value of infinity under a weight too small for the cache's type (2^-32
 *   of the row's largest in FP16, 2^-126 in BF16) gives NaN.
 *   max_q: the largest number of new tokens of one sequence, which picks the
 *       kernel (any value >= 1 gives right results; the true one is fastest).
 *   ws: blk_attn_workspace_bytes(head_dim) bytes, 256-byte aligned, its first
 *       BLK_ATTN_ZEROED bytes zero before the first use; the kernels leave
 *       them so. One workspace serves batches of any size and head_dim up to
 *       its own; calls that can overlap need workspaces of their own.
 * One launch, or two (none if seqs or tokens is 0).
 */
typedef struct {
    const void *q;
    const void *gate;
    void *out;
    float *lse;
    int64_t q_stride, q_head_stride;
    int64_t gate_stride, gate_head_stride;
    int64_t out_stride, out_head_stride;
    int heads;
    int max_q;
    int window;     /* 0: none */
    float scale;    /* > 0 */
} blk_attn_args;

#define BLK_ATTN_ZEROED 32768

int blk_attn_run(const blk_cache *cache, const blk_batch *batch, const blk_attn_args *args, void *ws, size_t ws_bytes,
                 void *stream);
size_t blk_attn_workspace_bytes(int head_dim);

/*
 * Projections with 4-bit weights:
 *     out[i, n] = sum over groups g of s[n, g] * sum over k in g of (q[n, k] - z[n, g]) * x[i, k]
 * with n x k weights in groups of `group` consecutive k (32, 64 or 128; k a
 * multiple of it). q: n x k / 2 bytes, element 2j in the low nibble of byte j.
 * scales: n x k / group of dtype (BLK_BF16 or BLK_F16, the type of x and out
 * too). zeros: n x k / group bytes of 0..15, or none (has_zeros 0): z = 8.
 * n and k up to 2^24.
 *
 * blk_w4_pack lays them out once in `packed` (blk_w4_packed_bytes bytes,
 * 16-byte aligned, of the caller); the sources may be freed when the stream
 * has passed it. blk_w4_run: x is m x k, rows x_stride elements apart (a
 * multiple of 8), 16-byte aligned; out m x n, rows out_stride apart. Made for
 * small m (a decode step's tokens); any m up to 2^20 is right. One launch
 * (none at m = 0).
 */
typedef struct {
    int n, k, group, dtype, has_zeros;
} blk_w4;

size_t blk_w4_packed_bytes(const blk_w4 *w);     /* 0: not a shape of the operator */
int blk_w4_pack(const blk_w4 *w, const void *q, const void *scales, const void *zeros, void *packed, void *stream);
int blk_w4_run(const blk_w4 *w, const void *packed, const void *x, int64_t x_stride, int m, void *out,
               int64_t out_stride, void *stream);

/*
 * blk_norm_run - the norms around a block, for m rows of `width` elements (1
 * to 32768):
 *     t = x * rsqrt(mean(x^2) + eps) * weight_post      (t = x without weight_post)
 *     residual_out = residual + alpha * gate * t        (no gate: 1)
 *     out = r * rsqrt(mean(r^2) + eps) * weight_pre     with r = residual_out before rounding
 * x NULL (then no weight_post, gate and residual_out either): only the last
 * line, of residual. x, gate, the weights and out are of dtype (BLK_BF16 or
 * BLK_F16), residual and residual_out of residual_dtype (dtype or BLK_F32).
 * residual_out may be residual, and out may be x. Row strides in elements; a
 * gate_stride of 0 shares one gate row. Rows whose strides, pointers and
 * width are multiples of 8 elements (16 bytes) are read 16 bytes at a time,
 * others element by element. One launch (none at m = 0).
 */
typedef struct {
    const void *x, *residual, *gate, *weight_post, *weight_pre;
    void *residual_out, *out;
    int64_t x_stride, residual_stride, gate_stride, residual_out_stride, out_stride;
    int width, dtype, residual_dtype;
    float alpha, eps;
} blk_norm_args;

int blk_norm_run(const blk_norm_args *args, int m, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* BLOCK_H */
