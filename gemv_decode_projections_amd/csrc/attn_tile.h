// Attention of many rows (drafted tokens of a large group, chunks of a
// prompt) over a paged cache: keys and values go through LDS once for all the
// rows of a workgroup.
//
// Mathematics, per wave of 32 rows and tile of 64 positions, on v_mfma
// 32x32x16 (A: lane l holds row l%32, k = 8 (l/32) + 0..7; B: column l%32, the
// same k; C: column l%32, rows 8 (i/4) + 4 (l/32) + i%4 for i = 0..15):
//   S^T (64 x 32) = K Q^T         A = keys from LDS, B = queries in registers;
//   O^T (DIM x 32) += V^T P^T     A = values, transposed as LDS is read.
// A row's scores sit in two lanes (l and l + 32), so its maximum takes one lane
// swap, and the packed probabilities are the B operand as they are if A takes
// the positions in the same order: 16 s + 4 (l/32) + {0..3, 8..11}. The
// transposing LDS read hands each lane four such positions of one element.
//
// The rows' maximum is raised only when a score passes it by more than 2^8 (in
// powers of two): the weights then stay below 2^8, exact in FP32 and in the
// types' range, and the accumulators are rescaled a few times per row instead
// of once per tile.
//
// Tiles of K and V fill a ring of LDS by DMA, one tile ahead of the products. A
// tile row's 16-byte pieces are permuted (by the address that each lane of the
// DMA reads) so that neither read meets a bank conflict.
#pragma once

#include "attn.h"

namespace gdp {

// Piece at which piece c of row r is kept. Keys: 16 lanes read 16 rows at one
// piece. Values: 32 lanes read 4 rows x 64 bytes (two pairs of pieces).
template <int DIM>
__device__ __forceinline__ int key_piece(int r, int c)
{
    return c ^ (r & (DIM == 64 ? 7 : 15));
}
template <int DIM>
__device__ __forceinline__ int value_piece(int r, int c)
{
    return DIM == 64 ? c ^ ((r & 3) << 1) : c ^ ((r & 3) << 2 | (r >> 2 & 1) << 1);
}

// 64 lanes x 16 bytes from base + lane_off to LDS, lane l at lds + 16 l. In
// assembly for the reason given at lds_dma16 in wide.h; waits are explicit.
__device__ __forceinline__ void dma_rows(const char *base, uint32_t lane_off, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %2\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(lane_off), "s"(base), "s"(lds)
                 : "memory", "m0");
}

template <int N>
__device__ __forceinline__ void wait_vm()
{
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

template <class T, int DIM, int WAVES>
__global__ __launch_bounds__(64 * WAVES, DIM == 256 || WAVES == 2 ? 1 : 2) void attn_tile(AttnArgs a)
{
    constexpr int ROWS = 32 * WAVES;
    constexpr int KS = DIM / 16;                     // k-steps of Q K^T
    constexpr int DB = DIM / 32;                     // 32-element blocks of the output
    constexpr int ROWB = DIM * 2;
    constexpr int TILEB = kTilePos * ROWB;           // bytes of one tile of K or V
    constexpr int RPI = 1024 / ROWB;                 // rows per DMA instruction (8, 4 or 2)
    constexpr int NI = kTilePos / RPI / WAVES;       // DMA instructions per wave and tile, each of K and V
    constexpr int STAGES = 2;
    constexpr float RAISE = 8.0f;
    __shared__ __align__(1024) char s_ring[STAGES][2][TILEB];

    AttnUnit u;
    if (!find_unit<ROWS>(a, blockIdx.x, u))
        return;
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int col = lane % 32, half = lane / 32;

    // Queries as B operands; rows past the last read it again and see nothing.
    u32x4 qf[KS];
    const int r = wave * 32 + col;
    int see_lo, see_hi, tok, head;
    {
        row_place(a, u, u.row0 + min(r, u.nrows - 1), tok, head);
        const char *p = a.q + tok * a.q_stride + head * a.q_head + half * 16;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
            qf[ks] = *reinterpret_cast<const u32x4 *>(p + ks * 32);
        const int pos = u.len - u.n + tok - u.tok0;
        see_hi = r < u.nrows ? pos + 1 : 0;
        see_lo = a.window > 0 ? pos - a.window + 1 : 0;
    }
    const int i0 = a.by_group(u.row0), i1 = a.by_group(u.row0 + u.nrows - 1);
    const int all_hi = u.len - u.n + i0 + 1;
    const int all_lo = a.window > 0 ? u.len - u.n + i1 - a.window + 1 : 0;

    // The unit's pages, read by scalar loads: a DMA instruction's rows are
    // aligned and share a page.
    typedef const __attribute__((address_space(4))) int32_t *ScalarPtr;
    const ScalarPtr table = (ScalarPtr)(uintptr_t)(a.table + (int64_t)u.seq * a.table_stride);
    const int64_t head_off = (int64_t)u.kvh * a.head_stride;
    auto page_of = [&](int p) { return table[min(p >> a.page_shift, a.table_width - 1)]; };
    bool gap = false;
    for (int p = (u.lo >> a.page_shift) + threadIdx.x; p < a.table_width && p << a.page_shift < u.hi; p += 64 * WAVES)
        gap |= (unsigned)a.table[(int64_t)u.seq * a.table_stride + p] >= (unsigned)a.n_pages;
    const bool holes = __syncthreads_or(gap);

    // Lane offsets of a DMA instruction: instruction n covers rows RPI n ..,
    // lane l row RPI n + l / (64 / RPI), piece l % (64 / RPI) of LDS.
    constexpr int PIECES = 64 / RPI;
    const int sub = lane / PIECES, piece = lane % PIECES;
    auto issue = [&](int base, int stage) {
        const uint32_t lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)&s_ring[stage][0][0];
#pragma unroll
        for (int n = 0; n < NI; ++n) {
            const int row = (wave * NI + n) * RPI;
            int64_t off;
            kv_offset(a, page_of(base + row), base + row, head_off, off);
            const uint32_t step = (uint32_t)sub * (uint32_t)a.token_stride;
            dma_rows(a.k + off, step + 16 * key_piece<DIM>(row + sub, piece), lds + row * ROWB);
            dma_rows(a.v + off, step + 16 * value_piece<DIM>(row + sub, piece), lds + TILEB + row * ROWB);
        }
    };

    f32x16 acc[DB];
#pragma unroll
    for (int d = 0; d < DB; ++d)
        acc[d] = f32x16{};
    float top = -INFINITY, sum = 0.f;

    // Value fragment of positions 32 pb + 16 s + 4 half + {0..3, 8..11},
    // element 32 d + col, by two transposing reads: of each 16 lanes, lane i
    // points at row i / 4, elements 4 (i % 4) .. + 3, and receives element i
    // of the four rows.
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    const int trow = 4 * half + lane % 16 / 4;
    const int tcol = 16 * (lane / 16 % 2) + 4 * (lane % 4);
    auto value_frag = [&](const char *v, int k0, int d) {
        u32x4 f;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const int row = k0 + 8 * p + trow, el = 32 * d + tcol;
            const char *at = v + row * ROWB + 16 * value_piece<DIM>(row, el / 8) + el % 8 * 2;
            const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) s16x4 *)at);
            const u32x2 y = __builtin_bit_cast(u32x2, x);
            f[2 * p] = y.x;
            f[2 * p + 1] = y.y;
        }
        return f;
    };

    if (u.lo < u.hi)
        issue(u.lo, 0);
    int stage = 0;
    for (int base = u.lo; base < u.hi; base += kTilePos, stage ^= 1) {
        wait_vm<0>();
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if (base + kTilePos < u.hi)
            issue(base + kTilePos, stage ^ 1);
        const char *kt = s_ring[stage][0], *vt = s_ring[stage][1];

        f32x16 s[2];
#pragma unroll
        for (int pb = 0; pb < 2; ++pb) {
            s[pb] = f32x16{};
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const int row = 32 * pb + col;
                const u32x4 kf =
                    *reinterpret_cast<const u32x4 *>(kt + row * ROWB + 16 * key_piece<DIM>(row, 2 * ks + half));
                s[pb] = T::mfma32(kf, qf[ks], s[pb]);
            }
        }
        const bool masked = holes || base < all_lo || base + kTilePos > all_hi || base + kTilePos > u.hi;
        uint32_t held = 0xffffffffu;       // bit 16 pb + i: position 32 pb + 8 (i / 4) + 4 half + i % 4
        if (masked) {
#pragma unroll
            for (int pb = 0; pb < 2; ++pb)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int p0 = base + 32 * pb + 8 * g + 4 * half;
                    const bool ok = !holes || (unsigned)a.table[(int64_t)u.seq * a.table_stride +
                                                                min(p0 >> a.page_shift, a.table_width - 1)] <
                                                  (unsigned)a.n_pages;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int p = p0 + e;
                        const bool in = ok && p < u.hi;
                        if (!in)
                            held &= ~(1u << (16 * pb + 4 * g + e));
                        if (!(in && p >= see_lo && p < see_hi))
                            s[pb][4 * g + e] = -INFINITY;
                    }
                }
        }
        float m = -INFINITY;
#pragma unroll
        for (int pb = 0; pb < 2; ++pb)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                m = fmaxf(m, s[pb][i]);
        m = max32(m) * a.scale_log2;
        if (__any(m > top + RAISE)) {
            const float raised = fmaxf(m, top);
            const float f = exp2_fast(top - (raised == -INFINITY ? 0.f : raised));
            top = raised;
            sum *= f;
#pragma unroll
            for (int d = 0; d < DB; ++d)
                acc[d] *= f;
        }
        const float safe = top == -INFINITY ? 0.f : top;
        // Probabilities in 16 bits for the matrix instruction: each within
        // half a unit of the type, errors that average out over a row; the sum
        // keeps the unrounded ones.
        u32x4 pf[2][2];
#pragma unroll
        for (int pb = 0; pb < 2; ++pb)
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                const float p0 = exp2_fast(__builtin_fmaf(s[pb][i], a.scale_log2, -safe));
                const float p1 = exp2_fast(__builtin_fmaf(s[pb][i + 1], a.scale_log2, -safe));
                sum += p0;
                sum += p1;
                pf[pb][i / 8][i % 8 / 2] = T::pack(p0, p1);
            }
        if (!masked) {
#pragma unroll
            for (int pb = 0; pb < 2; ++pb)
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int d = 0; d < DB; ++d)
                        acc[d] = T::mfma32(value_frag(vt, 32 * pb + 16 * t, d), pf[pb][t], acc[d]);
        } else {
            // Values past the last token or on unmapped pages are not the
            // cache's: zero. One that only some rows see may be an infinity or
            // a NaN, which a zero weight does not silence in a product: it is
            // left out of the product and added to the rows that see it.
            bool poisoned = false;
#pragma unroll
            for (int pb = 0; pb < 2; ++pb)
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    u32x4 keep;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t b = held >> (16 * pb + 8 * t + 2 * e);
                        keep[e] = (b & 1 ? 0xffffu : 0u) | (b & 2 ? 0xffff0000u : 0u);
                    }
#pragma unroll
                    for (int d = 0; d < DB; ++d) {
                        u32x4 f = value_frag(vt, 32 * pb + 16 * t, d) & keep;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            poisoned |= not_finite<T>(f[e]);
                            f[e] = finite_only<T>(f[e]);
                        }
                        acc[d] = T::mfma32(f, pf[pb][t], acc[d]);
                    }
                }
            if (__any(poisoned))
                for (int pos = 0; pos < kTilePos; ++pos) {
                    if (base + pos >= u.hi || (unsigned)page_of(base + pos) >= (unsigned)a.n_pages)
                        continue;
                    const int i = pos % 32 / 8 * 4 + pos % 4;
                    uint32_t pair = 0;
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        if (k == pos / 32 * 8 + i / 2)
                            pair = pf[k / 8][k / 4 % 2][k % 4];
                    const float w = __shfl(i % 2 ? T::hi(pair) : T::lo(pair), pos / 4 % 2 * 32 + col);
                    if (base + pos < see_lo || base + pos >= see_hi)
                        continue;
#pragma unroll
                    for (int d = 0; d < DB; ++d)
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            const int el = 32 * d + 8 * g + 4 * half;
                            const u32x2 x = *reinterpret_cast<const u32x2 *>(
                                vt + pos * ROWB + 16 * value_piece<DIM>(pos, el / 8) + el % 8 * 2);
                            const float v[4] = {T::lo(x.x), T::hi(x.x), T::lo(x.y), T::hi(x.y)};
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (!__builtin_isfinite(v[e]))
                                    acc[d][4 * g + e] += w * v[e];
                        }
                }
        }
    }
    sum = sum32(sum);
    // Out of the unit: straight to the output if the tile has one split, else
    // to the unit's slot for the join kernel.
    if (r >= u.nrows)
        return;
    const Slots<DIM, ROWS> slots(a);
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int el = 32 * d + 8 * g + 4 * half;
            const f32x4 v = {acc[d][4 * g], acc[d][4 * g + 1], acc[d][4 * g + 2], acc[d][4 * g + 3]};
            if (u.splits == 1)
                write_out<T>(a, tok, head, el, v, sum, a.gate ? load_gate(a, tok, head, el) : u32x2{0, 0});
            else
                slots.put(u.slot0 + u.split, r, el, v, top, sum);
        }
    if (u.splits == 1 && half == 0)
        write_lse(a, tok, head, top, sum);
}

}  // namespace gdp
