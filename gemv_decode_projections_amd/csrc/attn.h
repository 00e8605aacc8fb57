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
constexpr int kAttnSlotRows = 131072;              // rows of all slots together
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
// Workgroups are dealt to the 8 XCDs round-robin; the units, ordered so that
// the row tiles that read the same keys follow each other, are given to the
// XCDs in contiguous eighths, so those tiles share an L2.
// Returns false for workgroups past the last unit.
template <int ROWS>
__device__ bool find_unit(const AttnArgs &a, int id, AttnUnit &u)
{
    const int lane = threadIdx.x % kWave;
    struct Shape {
        int tok0, n, len, tiles, first, range;
    };
    auto shape = [&](int b) {
        Shape s = {0, 0, 0, 0, 0, 0};
        if (b < a.seqs) {
            seq_bounds(a, b, s.tok0, s.n, s.len);
            s.tiles = (s.n * a.group + ROWS - 1) / ROWS;
            if (a.window > 0)
                s.first = max(0, s.len - s.n - a.window + 1) / a.kv_step * a.kv_step;
            s.range = s.len - s.first;
        }
        return s;
    };
    Shape s;
    unsigned long long w = 0;
    for (int b0 = 0; b0 < a.seqs; b0 += kWave) {
        s = shape(b0 + lane);
        w += (unsigned long long)s.tiles * (unsigned)s.range;
    }
#pragma unroll
    for (int d = 1; d < kWave; d *= 2)
        w += __shfl_xor(w, d);
    w *= (unsigned)a.kv_heads;
    const unsigned long long per = (w + a.target - 1) / a.target;
    // (read from the first lane, so that what follows stays in scalar registers)
    const int c = __builtin_amdgcn_readfirstlane(
        (int)min((unsigned long long)0x40000000,
                 max((unsigned long long)a.min_split, (per + a.kv_step - 1) / a.kv_step * a.kv_step)));
    auto units_of = [&](const Shape &x, int &splits) {
        splits = max(1, (x.range + c - 1) / c);
        return x.tiles * splits * a.kv_heads;
    };
    int splits;
    int total = 0;
    for (int b0 = 0; b0 < a.seqs; b0 += kWave) {
        if (a.seqs > kWave)
            s = shape(b0 + lane);
        total += units_of(s, splits);
    }
#pragma unroll
    for (int d = 1; d < kWave; d *= 2)
        total += __shfl_xor(total, d);
    total = __builtin_amdgcn_readfirstlane(total);
    const int per_xcd = (total + 7) / 8;
    const int want = id % 8 * per_xcd + id / 8;
    if (id / 8 >= per_xcd || want >= total)
        return false;
    int units_before = 0, slots_before = 0;
    for (int b0 = 0; b0 < a.seqs; b0 += kWave) {
        if (a.seqs > kWave)
            s = shape(b0 + lane);
        const int units = units_of(s, splits);
        const int slots = splits > 1 ? units : 0;
        const int usum = units_before + wave_scan(units, lane);
        const int ssum = slots_before + wave_scan(slots, lane);
        const unsigned long long mine = __ballot(usum > want);
        if (mine) {
            const int l = __ffsll(mine) - 1;
            auto of = [&](int x) { return __builtin_amdgcn_readlane(x, l); };
            const int local = want - of(usum - units);
            const int tiles = of(s.tiles);
            u.seq = b0 + l;
            u.tok0 = of(s.tok0);
            u.n = of(s.n);
            u.len = of(s.len);
            u.splits = of(splits);
            const int tile = local % tiles;
            u.split = local / tiles % u.splits;
            u.kvh = local / tiles / u.splits;
            u.slot0 = of(ssum - slots) + (u.kvh * tiles + tile) * u.splits;
            u.row0 = tile * ROWS;
            u.nrows = min(ROWS, u.n * a.group - u.row0);
            u.lo = of(s.first) + u.split * c;
            // The tile's last token sees no further than its own position.
            const int last = u.len - u.n + (u.row0 + u.nrows - 1) / a.group;
            u.hi = min(u.split + 1 < u.splits ? u.lo + c : u.len, max(last + 1, 0));
            return true;
        }
        units_before = __builtin_amdgcn_readlane(usum, kWave - 1);
        slots_before = __builtin_amdgcn_readlane(ssum, kWave - 1);
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

// The workgroup's rows, unnormalised, leave the unit: straight to the output
// if the tile has one split. Otherwise they are published in the unit's slot
// with stores that pass the XCD-local L2 and the arrival is counted; the last
// of every kJoin consecutive splits joins those, and where there are more
// splits the joins are joined the same way, each result in the slot of its
// first split. A join thus reads at most kJoin slots, all loads in flight, and
// always in split order: the result does not depend on who came last.
// Measured: one workgroup joining all splits took 290 us of a 340 us call (16
// tiles of 64 rows in 30 splits each); the joins of kJoin take about 2 us a
// level.
// pieces(f) calls f(row, d, value, m, l) for the four elements d.. of each of
// the calling thread's pieces, m and l the row's maximum (in base-2 scaled
// scores) and sum.
constexpr int kJoin = 16;

template <class T, int DIM, int ROWS, int THREADS, class Pieces>
__device__ __forceinline__ void leave_unit(const AttnArgs &a, const AttnUnit &u, Pieces pieces, int *flag)
{
    const int tid = threadIdx.x;
    if (u.splits == 1) {
        pieces([&](int r, int d, f32x4 v, float m, float l) {
            write_out<T>(a, u, u.row0 + r, d, v, l == 0.f ? 0.f : 1.0f / l);
            if (d == 0)
                write_lse(a, u, u.row0 + r, m, l);
        });
        return;
    }
    constexpr uint32_t SLOT = ROWS * (DIM + 2) * 4u;
    constexpr uint32_t stats = ROWS * DIM * 4u;
    const __amdgpu_buffer_rsrc_t ws =
        __builtin_amdgcn_make_buffer_rsrc(a.slots, 0, (int)(kAttnSlotRows * (DIM + 2) * 4u), 0x00020000);
    auto publish = [&](int split, int r, int d, f32x4 v, float m, float l) {
        const uint32_t at = (uint32_t)(u.slot0 + split) * SLOT;
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), ws, at + (uint32_t)(r * DIM + d) * 4u, 0,
                                               kDeviceScope);
        if (d == 0)
            __builtin_amdgcn_raw_buffer_store_b64(
                u32x2{__builtin_bit_cast(uint32_t, m), __builtin_bit_cast(uint32_t, l)}, ws,
                at + stats + (uint32_t)r * 8u, 0, kDeviceScope);
    };
    pieces([&](int r, int d, f32x4 v, float m, float l) { publish(u.split, r, d, v, m, l); });
    constexpr int PER = DIM / 4;               // threads per row
    const int d = 4 * (tid % PER);
    for (int stride = 1, level = 0;; stride *= kJoin, ++level) {
        const int first = u.split / (stride * kJoin) * (stride * kJoin);
        const int members = min(kJoin, (u.splits - first + stride - 1) / stride);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (tid == 0) {
            // Counters of the levels lie at slots of different remainders.
            uint32_t *c = a.counters + u.slot0 + first + level;
            const uint32_t before = __hip_atomic_fetch_add(c, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            const bool last = before == (uint32_t)(members - 1);
            if (last)
                __hip_atomic_store(c, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            *flag = last;
        }
        __syncthreads();
        if (!*flag)
            return;
        const bool done = first == 0 && stride * kJoin >= u.splits;
        for (int r = tid / PER; r < u.nrows; r += THREADS / PER) {
            u32x2 st[kJoin];
            u32x4 v[kJoin];
#pragma unroll
            for (int i = 0; i < kJoin; ++i)
                if (i < members) {
                    const uint32_t at = (uint32_t)(u.slot0 + first + i * stride) * SLOT;
                    st[i] = __builtin_amdgcn_raw_buffer_load_b64(ws, at + stats + (uint32_t)r * 8u, 0, kDeviceScope);
                    v[i] = __builtin_amdgcn_raw_buffer_load_b128(ws, at + (uint32_t)(r * DIM + d) * 4u, 0, kDeviceScope);
                }
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < kJoin; ++i)
                if (i < members) {
                    // (by value: a bit cast of a vector's element takes element 0)
                    const uint32_t bits = st[i].x;
                    top = fmaxf(top, __builtin_bit_cast(float, bits));
                }
            const float safe = top == -INFINITY ? 0.f : top;
            float sum = 0.f;
            f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < kJoin; ++i)
                if (i < members) {
                    const uint32_t mbits = st[i].x, lbits = st[i].y;
                    const float f = exp2_fast(__builtin_bit_cast(float, mbits) - safe);
                    sum += f * __builtin_bit_cast(float, lbits);
                    acc += f * __builtin_bit_cast(f32x4, v[i]);
                }
            if (done) {
                write_out<T>(a, u, u.row0 + r, d, acc, sum == 0.f ? 0.f : 1.0f / sum);
                if (d == 0)
                    write_lse(a, u, u.row0 + r, top, sum);
            } else {
                publish(first, r, d, acc, top, sum);
            }
        }
        if (done)
            return;
    }
}

constexpr int kTilePos = 64;               // positions of the tile kernel's tiles

using AttnKernel = void (*)(AttnArgs);
// Row kernels for tiles of 16 * nb rows (nb 1, 2); nullptr if not built.
AttnKernel attn_rows_kernel(int dtype, int dim, int nb);
// Tile kernels for tiles of 32 * waves rows (waves 2, 4), 64 * waves threads.
AttnKernel attn_tile_kernel(int dtype, int dim, int waves);

}  // namespace gdp
