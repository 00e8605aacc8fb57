// Attention over a paged cache: kernel arguments, the partition of a batch
// into work units, and the joining of a row tile's splits, shared by the
// row kernel (attn_rows.h: few rows, cache straight into registers) and the
// tile kernel (attn_tile.h: many rows, cache through LDS).
//
// A row is one (new token, query head) pair of a key head's group; the rows of
// a sequence are ordered token first, r = token * G + head % G with G = heads
// / kv_heads, so one row tile of consecutive rows reads each key once for the
// whole group.
#pragma once

#include "block_common.h"

namespace gdp {

struct AttnArgs {
    const char *k, *v;                 // cache
    uint32_t page_stride;              // bytes
    int token_stride, head_stride;     // bytes
    int n_pages, page_shift, page_mask;
    const int32_t *q_start, *kv_len, *table;
    int64_t table_stride;
    int table_width, seqs, tokens;
    const char *q, *gate;
    char *out;
    float *lse;
    int64_t q_stride, gate_stride, out_stride;     // bytes
    int64_t q_head, gate_head, out_head;           // bytes
    int heads, kv_heads, group;
    int window;
    float scale_log2;                  // scale * log2(e): softmax in base 2
    int kv_step;                       // split lengths are multiples of this
    int min_split;                     // smallest split length
    int target;                        // units aimed at when rows alone are too few
    char *slots;                       // partials
    uint32_t *counters;                // one per slot, zero between launches
};

// A split's partial result takes a slot: its rows' FP32 outputs, maxima and
// sums. Splits that share row tiles number at most two per unit aimed at (a
// tile's range r is cut in ceil(r / C) parts; where that is more than one it
// is less than 2 r / C, and the ranges sum to at most target * C), so the
// kernels aim at units in inverse proportion to their tile's rows and one
// workspace serves all of them.
constexpr int kAttnSlotRows = 65536;               // rows of all slots together
constexpr int kAttnMaxTarget = 512;
__host__ __device__ constexpr int attn_target(int rows)
{
    return kAttnSlotRows / 2 / rows < kAttnMaxTarget ? kAttnSlotRows / 2 / rows : kAttnMaxTarget;
}
constexpr size_t kAttnCounterBytes = 2 * kAttnMaxTarget * sizeof(uint32_t);
constexpr size_t attn_ws_bytes(int dim) { return kAttnCounterBytes + (size_t)kAttnSlotRows * (dim + 2) * 4; }

// One workgroup's share: rows row0 .. row0 + nrows - 1 of sequence `seq`
// (first new token tok0, n new tokens) of key head kvh, against positions
// lo .. hi - 1; split `split` of `splits`, slots slot0 .. slot0 + splits - 1.
struct AttnUnit {
    int seq, tok0, n, len, kvh;
    int row0, nrows;
    int lo, hi;
    int split, splits, slot0;
};

__device__ __forceinline__ int wave_scan(int x, int lane)
{
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
        const int y = __shfl_up(x, d);
        if (lane >= d)
            x += y;
    }
    return x;
}

// New tokens and cached positions of sequence b, bounded to the tensors.
__device__ __forceinline__ void seq_bounds(const AttnArgs &a, int b, int &tok0, int &n, int &len)
{
    const int s = min(max(a.q_start[b], 0), a.tokens);
    const int e = min(max(a.q_start[b + 1], s), a.tokens);
    const int64_t cap = (int64_t)a.table_width << a.page_shift;
    tok0 = s;
    n = e - s;
    len = (int)min((int64_t)max(a.kv_len[b], 0), cap);
}

// Partition: with W = the row tiles' ranges summed over sequences and heads,
// every tile's range is cut in parts of C = max(min_split, W / target)
// positions, so a batch of any mix of lengths gives about `target` equal
// units, or one per tile where there are many tiles. Every workgroup computes
// the same partition from the device's lengths and finds its own unit.
// Returns false for workgroups past the last unit.
template <int ROWS>
__device__ bool find_unit(const AttnArgs &a, int id, AttnUnit &u)
{
    const int lane = threadIdx.x % kWave;
    const int kvh = id % a.kv_heads;
    const int want = id / a.kv_heads;
    auto shape = [&](int b, int &tok0, int &n, int &len, int &tiles, int &first) {
        tok0 = n = len = tiles = first = 0;
        if (b < a.seqs) {
            seq_bounds(a, b, tok0, n, len);
            tiles = (n * a.group + ROWS - 1) / ROWS;
            if (a.window > 0)
                first = max(0, len - n - a.window + 1) / a.kv_step * a.kv_step;
        }
        return len - first;
    };
    int tok0, n, len, tiles, first;
    int range = 0;
    unsigned long long w = 0;
    for (int b0 = 0; b0 < a.seqs; b0 += kWave) {
        range = shape(b0 + lane, tok0, n, len, tiles, first);
        w += (unsigned long long)tiles * (unsigned)range;
    }
#pragma unroll
    for (int d = 1; d < kWave; d *= 2)
        w += __shfl_xor(w, d);
    w *= (unsigned)a.kv_heads;
    const unsigned long long per = (w + a.target - 1) / a.target;
    const int c = (int)min((unsigned long long)0x40000000,
                           max((unsigned long long)a.min_split, (per + a.kv_step - 1) / a.kv_step * a.kv_step));
    int units_before = 0, slots_before = 0;
    for (int b0 = 0; b0 < a.seqs; b0 += kWave) {
        if (a.seqs > kWave)
            range = shape(b0 + lane, tok0, n, len, tiles, first);
        const int splits = max(1, (range + c - 1) / c);
        const int units = tiles * splits;
        const int slots = splits > 1 ? units : 0;
        const int usum = units_before + wave_scan(units, lane);
        const int ssum = slots_before + wave_scan(slots, lane);
        const unsigned long long mine = __ballot(usum > want);
        if (mine) {
            const int l = __ffsll(mine) - 1;
            const int local = want - __shfl(usum - units, l);
            u.seq = b0 + l;
            u.tok0 = __shfl(tok0, l);
            u.n = __shfl(n, l);
            u.len = __shfl(len, l);
            u.splits = __shfl(splits, l);
            const int lo0 = __shfl(first, l);
            const int tile = local / u.splits;
            u.split = local - tile * u.splits;
            u.slot0 = (__shfl(ssum - slots, l) + tile * u.splits) * a.kv_heads + kvh;
            u.kvh = kvh;
            u.row0 = tile * ROWS;
            u.nrows = min(ROWS, u.n * a.group - u.row0);
            u.lo = lo0 + u.split * c;
            // The tile's last token sees no further than its own position.
            const int last = u.len - u.n + (u.row0 + u.nrows - 1) / a.group;
            u.hi = min(u.split + 1 < u.splits ? u.lo + c : u.len, max(last + 1, 0));
            return true;
        }
        units_before = __shfl(usum, kWave - 1);
        slots_before = __shfl(ssum, kWave - 1);
    }
    return false;
}

// Byte offset of position p's key (or value) of the unit's head, and whether
// its page is in the cache; an unmapped page reads page 0 (its values are
// replaced by zeros and its scores masked).
__device__ __forceinline__ bool kv_offset(const AttnArgs &a, int page, int p, int64_t head_off, int64_t &off)
{
    const bool ok = (unsigned)page < (unsigned)a.n_pages;
    off = (int64_t)((uint64_t)(uint32_t)(ok ? page : 0) * a.page_stride) + (int64_t)(p & a.page_mask) * a.token_stride +
          head_off;
    return ok;
}

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + exp2_fast(-1.44269504f * x)); }

// Writes four consecutive outputs of a row: divided, gated, rounded once.
template <class T>
__device__ __forceinline__ void write_out(const AttnArgs &a, const AttnUnit &u, int row, int d, f32x4 o, float inv)
{
    const int tok = u.tok0 + row / a.group;
    const int head = u.kvh * a.group + row % a.group;
    o *= inv;
    if (a.gate) {
        const u32x2 g = *reinterpret_cast<const u32x2 *>(a.gate + tok * a.gate_stride + head * a.gate_head + d * 2);
        o.x *= sigmoid(T::lo(g.x));
        o.y *= sigmoid(T::hi(g.x));
        o.z *= sigmoid(T::lo(g.y));
        o.w *= sigmoid(T::hi(g.y));
    }
    *reinterpret_cast<u32x2 *>(a.out + tok * a.out_stride + head * a.out_head + d * 2) =
        u32x2{T::pack(o.x, o.y), T::pack(o.z, o.w)};
}

__device__ __forceinline__ void write_lse(const AttnArgs &a, const AttnUnit &u, int row, float m, float l)
{
    if (a.lse)
        a.lse[(int64_t)(u.tok0 + row / a.group) * a.heads + u.kvh * a.group + row % a.group] =
            l > 0.f || l != l ? (m + __builtin_amdgcn_logf(l)) * 0.693147181f : -INFINITY;
}

// The workgroup's rows, unnormalised in LDS (o: rows x pitch floats, maxima m
// in base-2 scaled scores, sums l), leave the unit: straight to the output if
// the tile has one split. Otherwise they are published in the unit's slot
// with stores that pass the XCD-local L2, the arrival is counted, and the
// tile's last workgroup joins the splits in split order (so the result does
// not depend on which came last).
template <class T, int DIM, int ROWS, int THREADS>
__device__ __forceinline__ void leave_unit(const AttnArgs &a, const AttnUnit &u, const float *o, int pitch,
                                           const float *m, const float *l, int *flag)
{
    const int tid = threadIdx.x;
    constexpr int PER = DIM / 4;               // threads per row
    constexpr int STEP = THREADS / PER;        // rows per pass
    const int d = 4 * (tid % PER);
    if (u.splits == 1) {
        for (int r = tid / PER; r < u.nrows; r += STEP) {
            const float sum = l[r];
            const f32x4 v = *reinterpret_cast<const f32x4 *>(o + r * pitch + d);
            write_out<T>(a, u, u.row0 + r, d, v, sum == 0.f ? 0.f : 1.0f / sum);
            if (d == 0)
                write_lse(a, u, u.row0 + r, m[r], sum);
        }
        return;
    }
    constexpr uint32_t SLOT = ROWS * (DIM + 2) * 4u;
    constexpr uint32_t stats = ROWS * DIM * 4u;
    const __amdgpu_buffer_rsrc_t ws =
        __builtin_amdgcn_make_buffer_rsrc(a.slots, 0, (int)(kAttnSlotRows * (DIM + 2) * 4u), 0x00020000);
    // Consecutive slots of a tile are kv_heads apart.
    auto slot = [&](int s) { return (uint32_t)(u.slot0 + s * a.kv_heads) * SLOT; };
    const uint32_t mine = slot(u.split);
    for (int r = tid / PER; r < u.nrows; r += STEP) {
        const f32x4 v = *reinterpret_cast<const f32x4 *>(o + r * pitch + d);
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), ws, mine + (uint32_t)(r * DIM + d) * 4u, 0,
                                               kDeviceScope);
        if (d == 0)
            __builtin_amdgcn_raw_buffer_store_b64(u32x2{__builtin_bit_cast(uint32_t, m[r]),
                                                        __builtin_bit_cast(uint32_t, l[r])},
                                                  ws, mine + stats + (uint32_t)r * 8u, 0, kDeviceScope);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (tid == 0) {
        uint32_t *c = a.counters + u.slot0;
        const uint32_t before = __hip_atomic_fetch_add(c, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        const bool last = before == (uint32_t)(u.splits - 1);
        if (last)
            __hip_atomic_store(c, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        *flag = last;
    }
    __syncthreads();
    if (!*flag)
        return;
    for (int r = tid / PER; r < u.nrows; r += STEP) {
        float top = -INFINITY, sum = 0.f;
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
        constexpr int CH = 4;                  // splits in flight
        for (int s0 = 0; s0 < u.splits; s0 += CH) {
            u32x2 st[CH];
            u32x4 v[CH];
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const uint32_t at = slot(min(s0 + i, u.splits - 1));
                st[i] = __builtin_amdgcn_raw_buffer_load_b64(ws, at + stats + (uint32_t)r * 8u, 0, kDeviceScope);
                v[i] = __builtin_amdgcn_raw_buffer_load_b128(ws, at + (uint32_t)(r * DIM + d) * 4u, 0, kDeviceScope);
            }
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                if (s0 + i >= u.splits)
                    break;
                // (by value: a bit cast of a vector's element takes element 0)
                const uint32_t mbits = st[i].x, lbits = st[i].y;
                const float ms = __builtin_bit_cast(float, mbits);
                const float big = fmaxf(top, ms);
                const float safe = big == -INFINITY ? 0.f : big;
                const float f = exp2_fast(top - safe), g = exp2_fast(ms - safe);
                acc = acc * f + __builtin_bit_cast(f32x4, v[i]) * g;
                sum = sum * f + __builtin_bit_cast(float, lbits) * g;
                top = big;
            }
        }
        write_out<T>(a, u, u.row0 + r, d, acc, sum == 0.f ? 0.f : 1.0f / sum);
        if (d == 0)
            write_lse(a, u, u.row0 + r, top, sum);
    }
}

using AttnKernel = void (*)(AttnArgs);
// Row kernels for tiles of 16 * nb rows (nb 1, 2, 4); nullptr if not built.
AttnKernel attn_rows_kernel(int dtype, int dim, int nb);

}  // namespace gdp
