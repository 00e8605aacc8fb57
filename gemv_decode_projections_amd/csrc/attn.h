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

// Division by a number the host knows, exact below 2^31: x * ceil(2^p / d) >>
// p with p = 31 + ceil(log2 d).
struct Divisor {
    uint32_t mul;
    int shift;

    static Divisor of(uint32_t d)
    {
        int s = 0;
        while (((uint64_t)1 << s) < d)
            ++s;
        return {(uint32_t)((((uint64_t)1 << (31 + s)) + d - 1) / d), 31 + s};
    }
    __device__ __forceinline__ int operator()(int x) const { return (int)((uint64_t)(uint32_t)x * mul >> shift); }
};

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
    Divisor by_heads, by_group;        // of kv_heads and group
    int window;
    float scale_log2;                  // scale * log2(e): softmax in base 2
    int kv_step;                       // split lengths are multiples of this (a power of two)
    int min_split;                     // smallest split length
    int target;                        // workgroups the chip holds at once
    float per_target;                  // 1 / target
    int rounds;                        // of them, where one round would not be even
    char *slots;                       // partials
    uint32_t *counters;                // one per slot, zero between launches
};

// A split's partial result takes a slot: its rows' FP32 outputs, maxima and
// sums. Splits that share row tiles number at most two per unit aimed at (a
// tile's range r is cut in ceil(r / C) parts; where that is more than one it
// is less than 2 r / C, and the ranges sum to at most target * C), so kernels
// whose tiles have more rows aim at fewer units, and one workspace serves all.
constexpr int kAttnSlotRows = 131072;              // rows of all slots together
constexpr int kAttnMaxSlots = kAttnSlotRows / 16;
constexpr size_t kAttnCounterBytes = kAttnMaxSlots * sizeof(uint32_t);
static_assert(kAttnCounterBytes == BLK_ATTN_ZEROED, "the counters are what a caller zeroes");
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

// Inclusive sums over the wave's lanes, in the vector unit: within rows of 16
// lanes, then the rows' totals passed on (row_shr 1, 2, 4, 8, row_bcast 15, 31).
template <int CTRL, int ROWMASK>
__device__ __forceinline__ int lane_moved(int x)
{
    return __builtin_amdgcn_update_dpp(0, x, CTRL, ROWMASK, 0xf, false);
}
template <int CTRL, int ROWMASK>
__device__ __forceinline__ unsigned long long lane_moved(unsigned long long x)
{
    return (unsigned long long)(unsigned)lane_moved<CTRL, ROWMASK>((int)(x >> 32)) << 32 |
           (unsigned)lane_moved<CTRL, ROWMASK>((int)x);
}
template <class I>
__device__ __forceinline__ I wave_scan(I x)
{
    x += lane_moved<0x111, 0xf>(x);
    x += lane_moved<0x112, 0xf>(x);
    x += lane_moved<0x114, 0xf>(x);
    x += lane_moved<0x118, 0xf>(x);
    x += lane_moved<0x142, 0xa>(x);
    x += lane_moved<0x143, 0xc>(x);
    return x;
}
// Inclusive maxima over the wave's lanes, no value negative.
__device__ __forceinline__ int wave_max_scan(int x)
{
    x = max(x, lane_moved<0x111, 0xf>(x));
    x = max(x, lane_moved<0x112, 0xf>(x));
    x = max(x, lane_moved<0x114, 0xf>(x));
    x = max(x, lane_moved<0x118, 0xf>(x));
    x = max(x, lane_moved<0x142, 0xa>(x));
    return max(x, lane_moved<0x143, 0xc>(x));
}
__device__ __forceinline__ int last_lane(int x) { return __builtin_amdgcn_readlane(x, kWave - 1); }

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

// Partition. Every tile's range is cut in parts of C positions. Every
// workgroup computes the same partition from the device's lengths, one lane
// per sequence. With W the row tiles' ranges summed over sequences and heads
// and `target` the workgroups the chip holds at once, C starts as W / target:
//   - the last part of a tile is short, so that gives more units than W / C: C
//     is raised until they fit one round (32 sequences of up to 8192 positions
//     x 8 heads: 640 units in 512 places took 139 us, 512 in 128);
//   - row kernels, with much work per unit or more tiles than half the places:
//     several rounds of smaller parts even out better (2048 units: 121 us);
//   - row kernels: short parts are not worth a join: up to 512 positions (640,
//     rounded up) per part as long as a tile has no more than 16 parts and half
//     the places are taken (one token over 131072 positions: 256 parts 20.5 us,
//     512 parts 24);
//   - tile kernels, with more tiles than half the places: the join of 128 rows
//     costs more than an uneven round, so C is twice that (416 tiles: 288 us,
//     cut for 512 places 446; 256 tiles cut in two: 177 us, whole 203).
// (Each pair of times is of the kernels as they were when the choice was made:
// the difference counts.) A tile's range is its sequence's, not what the tile
// sees: of a prompt with nothing cached the later tiles are the longer ones.
// (All of it inlined: called as functions, a unit's fields come back through
// memory and are no longer scalars.)
template <int ROWS>
struct Partition {
    struct Shape {
        int tok0, n, len, tiles, first, range, splits;
    };
    const AttnArgs &a;
    Shape s;             // the lane's sequence of the last 64 looked at
    int c;
    float per_c;
    int before;          // where the next 64 sequences begin at the earliest

    // The shapes of sequences b0 .. b0 + 63, in turn from 0. An offset counts as
    // the largest up to it: sequences do not overlap then, and their rows stay
    // within what the grid and the slots were made for.
    __device__ __forceinline__ void shape(int b0)
    {
        const int b = b0 + (int)(threadIdx.x % kWave);
        s = Shape{0, 0, 0, 0, 0, 0, 1};
        if (b < a.seqs)
            seq_bounds(a, b, s.tok0, s.n, s.len);
        const int end = s.tok0 + s.n, from = max(b0 ? before : 0, wave_max_scan(s.tok0));
        s.tok0 = from;
        s.n = max(end - from, 0);
        before = last_lane(from + s.n);
        s.tiles = (s.n * a.group + ROWS - 1) / ROWS;
        if (a.window > 0)
            s.first = max(0, s.len - s.n - a.window + 1) & -a.kv_step;
        s.range = s.len - s.first;
    }
    // ceil(range / c): the FP32 quotient is at most one off.
    __device__ __forceinline__ void cut()
    {
        int q = (int)((float)(s.range + c - 1) * per_c);
        q += q * c < s.range ? 1 : 0;
        q -= (q - 1) * c >= s.range ? 1 : 0;
        s.splits = max(q, 1);
    }
    __device__ __forceinline__ explicit Partition(const AttnArgs &args) : a(args)
    {
        unsigned long long w = 0;
        int t = 0, longest = 0;
        for (int b0 = 0; b0 < a.seqs; b0 += kWave) {
            shape(b0);
            w += (unsigned long long)s.tiles * (unsigned)s.range;
            t += s.tiles;
            longest = max(longest, s.range);
        }
        w = wave_scan(w);
        // Rounded up past the error of FP32: a larger c only means fewer parts.
        const float all = ((float)(unsigned)last_lane((int)(w >> 32)) * 0x1p32f + (float)(unsigned)last_lane((int)w)) *
                          (float)a.kv_heads * 1.00001f;
        const float per = all * a.per_target;
        const float tiles = (float)last_lane(wave_scan(t)) * (float)a.kv_heads;
        bool fit = tiles <= 0.5f * (float)a.target;
        if (ROWS <= 32) {
            fit = fit && per < 2048.f;
            set_part(fmaxf(fit ? per : per / (float)a.rounds,
                           fminf(512.f, fmaxf((float)last_lane(wave_max_scan(longest)) * (1.f / 16), all * a.per_target * 2.f))));
        } else {
            set_part(fit ? per : 2.f * per);
        }
        if (fit && a.seqs <= kWave)
            for (int i = 0; i < 2; ++i) {
                const int n = last_lane(wave_scan(units()));
                if (n <= a.target)
                    break;
                set_part((float)c * (float)n * a.per_target);
            }
    }
    __device__ __forceinline__ void set_part(float positions)
    {
        const int p = (int)fminf(positions + 1.0f, 0x1p29f);
        c = __builtin_amdgcn_readfirstlane(max(a.min_split, (p + a.kv_step - 1) & -a.kv_step));
        per_c = 1.0f / (float)c;
        cut();
    }
    __device__ __forceinline__ int units() const { return s.tiles * s.splits * a.kv_heads; }
    __device__ __forceinline__ int slots() const { return s.splits > 1 ? units() : 0; }
    // Blocks of rows whose splits have to be joined (join_rows each, attn_join.h).
    __device__ __forceinline__ int joins(int few, int rows) const
    {
        const int per = s.splits <= few ? rows : 1;
        return s.splits > 1 ? (s.n * a.group + per - 1) / per * a.kv_heads : 0;
    }

    template <class Count>
    __device__ __forceinline__ int total(Count count)
    {
        int t = 0;
        for (int b0 = 0; b0 < a.seqs; b0 += kWave) {
            if (a.seqs > kWave) {
                shape(b0);
                cut();
            }
            t += count(*this);
        }
        return last_lane(wave_scan(t));
    }
    // Finds item `want` (below the total) of those that `count` gives per
    // sequence: sets u's sequence and its first slot, returns the item's
    // number inside the sequence.
    template <class Count>
    __device__ __forceinline__ int find(int want, Count count, AttnUnit &u, int &tiles)
    {
        int items_before = 0, slots_before = 0;
        for (int b0 = 0;; b0 += kWave) {
            if (a.seqs > kWave) {
                shape(b0);
                cut();
            }
            const int isum = items_before + wave_scan(count(*this));
            const int ssum = slots_before + wave_scan(slots());
            const unsigned long long mine = __ballot(isum > want);
            if (mine || b0 + kWave >= a.seqs) {
                const int l = mine ? __ffsll(mine) - 1 : 0;
                auto of = [&](int x) { return __builtin_amdgcn_readlane(x, l); };
                u.seq = b0 + l;
                u.tok0 = of(s.tok0);
                u.n = of(s.n);
                u.len = of(s.len);
                u.splits = of(s.splits);
                u.lo = of(s.first);
                u.slot0 = of(ssum - slots());
                tiles = of(s.tiles);
                return want - of(isum - count(*this));
            }
            items_before = last_lane(isum);
            slots_before = last_lane(ssum);
        }
    }
};

// The workgroup's unit; false for workgroups past the last one. Workgroups are
// dealt to the 8 XCDs round-robin; the units are given to the XCDs in
// contiguous eighths. The heads of a key come first, as they lie next to each
// other in a page (32 sequences x 8 heads, when it was chosen: 131 us, with the
// heads apart in time 145), then the row tiles, which share their keys in an L2
// (chunks of 1000 and 630 tokens in pages of 16: 282 us, though the L2s fetch
// 540 MB; tiles before heads 289 and 119 MB; not measured on other contexts).
template <int ROWS>
__device__ __forceinline__ bool find_unit(const AttnArgs &a, int id, AttnUnit &u)
{
    Partition<ROWS> part(a);
    auto units = [](const Partition<ROWS> &p) { return p.units(); };
    const int total = part.total(units);
    const int per_xcd = (total + 7) / 8;
    const int want = id % 8 * per_xcd + id / 8;
    if (id / 8 >= per_xcd || want >= total)
        return false;
    int tiles;
    const int local = part.find(want, units, u, tiles);
    const int rest = a.by_heads(local);
    u.kvh = local - rest * a.kv_heads;
    int tile = 0;
    u.split = rest;
    if (tiles > 1) {
        u.split = rest / tiles;
        tile = rest - u.split * tiles;
    }
    u.slot0 += (u.kvh * tiles + tile) * u.splits;
    // (never more than there are, see kAttnSlotRows; a slot past them is no memory)
    if (u.splits > 1 && (unsigned)(u.slot0 + u.splits) > (unsigned)kAttnSlotRows / ROWS)
        return false;
    u.row0 = tile * ROWS;
    u.nrows = min(ROWS, u.n * a.group - u.row0);
    // The part, less what no row of the tile sees: its last token sees no
    // further than its own position, its first no further back than the window.
    const int lo = u.lo + u.split * part.c;
    const int hi = u.split + 1 < u.splits ? lo + part.c : u.len;
    const int before = u.len - u.n;
    u.lo = a.window > 0 ? max(lo, (before + a.by_group(u.row0) - a.window + 1) & -a.kv_step) : lo;
    u.hi = min(hi, max(before + a.by_group(u.row0 + u.nrows - 1) + 1, 0));
    return true;
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

// Token and query head of a row.
__device__ __forceinline__ void row_place(const AttnArgs &a, const AttnUnit &u, int row, int &tok, int &head)
{
    const int i = a.by_group(row);
    tok = u.tok0 + i;
    head = u.kvh * a.group + row - i * a.group;
}

// The gate's four elements for outputs d .. d + 3 of a row.
__device__ __forceinline__ u32x2 load_gate(const AttnArgs &a, int tok, int head, int d)
{
    return *reinterpret_cast<const u32x2 *>(a.gate + tok * a.gate_stride + head * a.gate_head + d * 2);
}

// Writes four consecutive outputs of a row: divided by the sum, gated, rounded once.
template <class T>
__device__ __forceinline__ void write_out(const AttnArgs &a, int tok, int head, int d, f32x4 o, float sum, u32x2 g)
{
    o *= sum == 0.f ? 0.f : 1.0f / sum;
    if (a.gate) {
        o.x *= sigmoid(T::lo(g.x));
        o.y *= sigmoid(T::hi(g.x));
        o.z *= sigmoid(T::lo(g.y));
        o.w *= sigmoid(T::hi(g.y));
    }
    *reinterpret_cast<u32x2 *>(a.out + tok * a.out_stride + head * a.out_head + d * 2) =
        u32x2{T::pack(o.x, o.y), T::pack(o.z, o.w)};
}

__device__ __forceinline__ void write_lse(const AttnArgs &a, int tok, int head, float m, float l)
{
    if (a.lse)
        a.lse[(int64_t)tok * a.heads + head] =
            l > 0.f || l != l ? (m + __builtin_amdgcn_logf(l)) * 0.693147181f : -INFINITY;
}

// Slots of the workspace. SCOPE kDeviceScope passes the XCD-local L2, for
// splits joined in the launch that made them; 0 is enough across launches.
template <int DIM, int ROWS, int SCOPE>
struct Slots {
    static constexpr uint32_t kSlot = ROWS * (DIM + 2) * 4u;
    static constexpr uint32_t kStats = ROWS * DIM * 4u;
    static constexpr uint32_t kEnd = kAttnSlotRows * (DIM + 2) * 4u;
    const __amdgpu_buffer_rsrc_t ws;

    __device__ explicit Slots(const AttnArgs &a)
        : ws(__builtin_amdgcn_make_buffer_rsrc(a.slots, 0, (int)kEnd, 0x00020000))
    {
    }
    __device__ __forceinline__ void put(int slot, int r, int d, f32x4 v, float m, float l) const
    {
        const uint32_t at = (uint32_t)slot * kSlot;
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), ws, at + (uint32_t)(r * DIM + d) * 4u, 0, SCOPE);
        if (d == 0)
            __builtin_amdgcn_raw_buffer_store_b64(
                u32x2{__builtin_bit_cast(uint32_t, m), __builtin_bit_cast(uint32_t, l)}, ws,
                at + kStats + (uint32_t)r * 8u, 0, SCOPE);
    }
    // Joins slots first, first + stride, .. of one row's elements d .. d + 3:
    // `members` of them, at most N, all loads in flight, in order.
    template <int N>
    __device__ __forceinline__ f32x4 join(int first, int stride, int members, int r, int d, float &top, float &sum) const
    {
        // The loads past the last member address the end of the workspace:
        // out of range, they return zero without a memory access.
        u32x2 st[N];
        u32x4 v[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t at = i < members ? (uint32_t)(first + i * stride) * kSlot : kEnd;
            st[i] = __builtin_amdgcn_raw_buffer_load_b64(ws, at + kStats + (uint32_t)r * 8u, 0, SCOPE);
            v[i] = __builtin_amdgcn_raw_buffer_load_b128(ws, at + (uint32_t)(r * DIM + d) * 4u, 0, SCOPE);
        }
        // (m and l by value: a bit cast of a vector's element takes element 0)
        float m[N];
        top = -INFINITY;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t bits = st[i].x;
            m[i] = i < members ? __builtin_bit_cast(float, bits) : -INFINITY;
            top = fmaxf(top, m[i]);
        }
        const float safe = top == -INFINITY ? 0.f : top;
        sum = 0.f;
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t bits = st[i].y;
            const float f = exp2_fast(m[i] - safe);
            sum += f * __builtin_bit_cast(float, bits);
            acc += f * __builtin_bit_cast(f32x4, v[i]);
        }
        return acc;
    }
};

// Positions of the tile kernel's tiles.
constexpr int attn_tile_pos(int dim) { return dim == 256 ? 32 : 64; }

using AttnKernel = void (*)(AttnArgs);
// Row kernels for tiles of 16 * nb rows (nb 1, 2); nullptr if not built.
AttnKernel attn_rows_kernel(int dtype, int dim, int nb);
// Tile kernels for tiles of 64 or 128 rows, two threads per row.
AttnKernel attn_tile_kernel(int dtype, int dim, int rows);
// Join kernels for tiles of 32, 64 or 128 rows (the row kernel joins its tiles of
// 16 itself), kJoinThreads threads.
AttnKernel attn_join_kernel(int dtype, int dim, int rows);
constexpr int kJoinThreads = 256;

}  // namespace gdp
