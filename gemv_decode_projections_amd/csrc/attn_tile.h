// Attention of many rows (drafted tokens of a large group, chunks of a
// prompt) over a paged cache: keys and values go through LDS once for all the
// rows of a workgroup.
//
// Mathematics, per block of 32 rows and tile of 64 positions (32 for heads of
// 256 elements, whose accumulators leave fewer registers), on v_mfma
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
// powers of two): the weights then stay below 2^8 (FP16: 2^15), exact in FP32
// and in the types' range, and the accumulators are rescaled a few times per row
// instead of once per tile (raised at every new maximum, which would keep the
// largest weight a power of two, chunks of 1000 and 630 tokens take 301 us
// instead of 285, of heads of 256 a fifth more). Weights are rounded to 16 bits
// (twice the products, with what rounding left: 8 % on drafted tokens of heads
// of 64 and 256).
//
// Tiles of K and V fill a ring of LDS by DMA, one tile ahead of the products. A
// tile row's 16-byte pieces are permuted (by the address that each lane of the
// DMA reads) so that neither read meets a bank conflict.
//
// Measured, BF16, heads of 128: chunks of 1000 and 630 tokens over 17 k
// positions, 32 heads on 8: 282 us, 780 TFLOP/s, half the rate of a large
// matrix product. The matrix unit is busy 43 % of the time, the vector unit's
// exponentials take about as long, and a wave's two kinds of work depend on
// each other. 16 sequences of up to 8 drafted tokens over 250 k positions, 8
// heads on 1: 39 us before the join, of which 20 at 6.5 TB/s (part of the cache
// comes from the last level of cache) and the rest the start and the ends.
#pragma once

#include <type_traits>

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
__global__ __launch_bounds__(64 * WAVES, DIM < 256 && WAVES > 2 ? 2 : 1) void attn_tile(AttnArgs a)
{
    constexpr int ROWS = 32 * WAVES;
    constexpr int KS = DIM / 16;                     // k-steps of Q K^T
    constexpr int DB = DIM / 32;                     // 32-element blocks of the output
    constexpr int ROWB = DIM * 2;
    constexpr int POS = attn_tile_pos(DIM);          // positions of a tile
    constexpr int HALVES = POS / 32;
    constexpr int TILEB = POS * ROWB;                // bytes of one tile of K or V
    constexpr int RPI = 1024 / ROWB;                 // rows per DMA instruction (8, 4 or 2)
    constexpr int NI = POS / RPI / WAVES;       // DMA instructions per wave and tile, of K as of V
    // (FP16: the largest weight is 2^7 to 2^15, and those down to 2^-21 of it are
    // normal numbers of the type)
    constexpr float RAISE = 8.0f, ABOVE = T::kId == BLK_F16 ? 15.0f - RAISE : 0.0f;
    // The ring of tiles; at the end each wave's 32 rows in FP32, 16-byte pieces
    // permuted so that neither side meets a bank conflict.
    constexpr int OUTB = ROWS * DIM * 4;
    __shared__ __align__(1024) char s_mem[4 * TILEB > OUTB ? 4 * TILEB : OUTB];
    char(&s_k)[2][TILEB] = *reinterpret_cast<char(*)[2][TILEB]>(s_mem);
    char(&s_v)[2][TILEB] = *reinterpret_cast<char(*)[2][TILEB]>(s_mem + 2 * TILEB);

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
    const uint32_t sub_off = (uint32_t)sub * (uint32_t)a.token_stride;
    auto lds_of = [](char *p) { return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)p; };
    // (the pages of a tile are read one tile before its DMA)
    int pages[NI];
    auto read_pages = [&](int base) {
#pragma unroll
        for (int n = 0; n < NI; ++n)
            pages[n] = page_of(base + (wave * NI + n) * RPI);
    };
    auto issue = [&](int base, auto stage) {
        int64_t off[NI];
#pragma unroll
        for (int n = 0; n < NI; ++n)
            kv_offset(a, pages[n], base + (wave * NI + n) * RPI, head_off, off[n]);
#pragma unroll
        for (int n = 0; n < NI; ++n) {
            const int row = (wave * NI + n) * RPI;
            dma_rows(a.k + off[n], sub_off + 16 * key_piece<DIM>(row + sub, piece), lds_of(s_k[stage.value]) + row * ROWB);
        }
#pragma unroll
        for (int n = 0; n < NI; ++n) {
            const int row = (wave * NI + n) * RPI;
            dma_rows(a.v + off[n], sub_off + 16 * value_piece<DIM>(row + sub, piece), lds_of(s_v[stage.value]) + row * ROWB);
        }
    };
    // (this wave's reads of LDS have ended: another's DMA overwrites what they read)
    auto barrier = [] { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); };

    f32x16 acc[DB];
#pragma unroll
    for (int d = 0; d < DB; ++d)
        acc[d] = f32x16{};
    float most = -INFINITY, top = -INFINITY, sum = 0.f;      // the row's largest score, what weights are relative to

    // Value fragment of positions k0 + 4 half + {0..3, 8..11}, element 32 d +
    // col, by two transposing reads: of each 16 lanes, lane i points at row
    // i / 4, elements 4 (i % 4) .. + 3, and receives element i of the four rows.
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    const int trow = 4 * half + lane % 16 / 4;
    const int tcol = 16 * (lane / 16 % 2) + 4 * (lane % 4);
    auto value_frag = [&](const char *v, int k0, int d) {
        u32x4 f;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const int row = k0 + 8 * p + trow, el = 32 * d + tcol;
            const char *at = v + row * ROWB + 16 * value_piece<DIM>(row, el / 8) + el % 8 * 2;
            const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)at);
            const u32x2 y = __builtin_bit_cast(u32x2, x);
            f[2 * p] = y.x;
            f[2 * p + 1] = y.y;
        }
        return f;
    };
    // Scores of a tile's halves, their chains of products side by side.
    auto scores = [&](const char *k, f32x16 (&s)[HALVES]) {
#pragma unroll
        for (int h = 0; h < HALVES; ++h)
            s[h] = f32x16{};
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int h = 0; h < HALVES; ++h) {
                const int row = 32 * h + col;
                s[h] = T::mfma32(
                    *reinterpret_cast<const u32x4 *>(k + row * ROWB + 16 * key_piece<DIM>(row, 2 * ks + half)), qf[ks],
                    s[h]);
            }
    };
    auto needs_mask = [&](int p) { return holes || p < all_lo || p + POS > all_hi || p + POS > u.hi; };
    // Masks the scores of positions p .. p + 31; bit i of the result: position
    // p + 8 (i / 4) + 4 half + i % 4 holds a token.
    auto mask = [&](int p, f32x16 &s) {
        uint32_t held = 0;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int p0 = p + 8 * g + 4 * half;
            const bool ok = !holes || (unsigned)a.table[(int64_t)u.seq * a.table_stride +
                                                        min(p0 >> a.page_shift, a.table_width - 1)] < (unsigned)a.n_pages;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool in = ok && p0 + e < u.hi;
                held |= in ? 1u << (4 * g + e) : 0u;
                if (!(in && p0 + e >= see_lo && p0 + e < see_hi))
                    s[4 * g + e] = -INFINITY;
            }
        }
        return held;
    };
    // Raises the rows' maxima to fit the scores, rescaling what was summed.
    auto raise = [&](const f32x16 (&s)[HALVES]) {
        // (the maximum that passes NaN on: it needs no canonical operands)
        float m = s[0][0];
#pragma unroll
        for (int i = 1; i < 16 * HALVES; ++i)
            m = __builtin_elementwise_maximum(m, s[i / 16][i % 16]);
        most = fmaxf(most, max32(m));
        m = most * a.scale_log2;
        const bool passes = m > top + (ABOVE + RAISE);
        if (__any(passes)) {
            // (this row only if it has to: `top` is then as it was when `most` was weighed)
            const float raised = passes ? m - ABOVE : top;
            const float f = exp2_fast(top - (raised == -INFINITY ? 0.f : raised));
            top = raised;
            sum *= f;
#pragma unroll
            for (int d = 0; d < DB; ++d)
                acc[d] *= f;
        }
    };
    // Probabilities in 16 bits for the matrix instruction: each within half a
    // unit of the type, errors that average out over a row; the sum keeps the
    // unrounded ones. (The largest's does not average out where it dominates:
    // see `even`.)
    auto weights = [&](const f32x16 &s, u32x4 (&pf)[2]) {
        const float safe = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            const float p0 = exp2_fast(__builtin_fmaf(s[i], a.scale_log2, -safe));
            const float p1 = exp2_fast(__builtin_fmaf(s[i + 1], a.scale_log2, -safe));
            sum += p0;
            sum += p1;
            pf[i / 8][i % 8 / 2] = T::pack(p0, p1);
        }
    };
    auto product = [&](const char *v, int h, const u32x4 (&pf)[2]) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int d = 0; d < DB; ++d)
                acc[d] = T::mfma32(value_frag(v, 32 * h + 16 * t, d), pf[t], acc[d]);
    };
    // The same for half a tile with masked positions p .. p + 31. Values past
    // the last token or on unmapped pages are not the cache's: zero. One that
    // only some rows see may be an infinity or a NaN, which a zero weight does
    // not silence in a product: it is left out of the product and added to the
    // rows that see it.
    auto masked_product = [&](const char *v, int h, int p, uint32_t held, const u32x4 (&pf)[2]) {
        FiniteCheck<T> check;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            u32x4 keep;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t bits = held >> (8 * t + 2 * e);
                keep[e] = (bits & 1 ? 0xffffu : 0u) | (bits & 2 ? 0xffff0000u : 0u);
            }
#pragma unroll
            for (int d = 0; d < DB; ++d) {
                u32x4 f = value_frag(v, 32 * h + 16 * t, d) & keep;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    check.add(f[e]);
                    f[e] = finite_only<T>(f[e]);
                }
                acc[d] = T::mfma32(f, pf[t], acc[d]);
            }
        }
        if (!__any(check.fails()))
            return;
#pragma unroll 1
        for (int j = 0; j < 32; ++j) {
            if (p + j >= u.hi || (unsigned)page_of(p + j) >= (unsigned)a.n_pages)
                continue;
            const int i = j / 8 * 4 + j % 4;
            uint32_t pair = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k == i / 2)
                    pair = pf[k / 4][k % 4];
            const float w = __shfl(i % 2 ? T::hi(pair) : T::lo(pair), j / 4 % 2 * 32 + col);
            if (p + j < see_lo || p + j >= see_hi)
                continue;
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int el = 32 * d + 8 * g + 4 * half;
                    const u32x2 x = *reinterpret_cast<const u32x2 *>(
                        v + (32 * h + j) * ROWB + 16 * value_piece<DIM>(32 * h + j, el / 8) + el % 8 * 2);
                    const float val[4] = {T::lo(x.x), T::hi(x.x), T::lo(x.y), T::hi(x.y)};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (!__builtin_isfinite(val[e]))
                            acc[d][4 * g + e] += w * val[e];
                }
        }
    };
    // The queries are here before the first DMA: a wait for them inside the loop
    // would wait for the DMA issued behind them.
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
        asm volatile("" : "+v"(qf[ks]));

    // One tile: its K and V are waited for, the next one's set off. Tiles that
    // need masks have a loop of their own, which keeps the other one lean.
    typedef std::integral_constant<int, 0> Stage0;
    typedef std::integral_constant<int, 1> Stage1;
    auto step = [&](int base, auto stage, auto other, auto masked) {
        wait_vm<0>();
        barrier();
        if (base + POS < u.hi) {
            issue(base + POS, other);
            read_pages(base + 2 * POS);
        }
        const char *k = s_k[stage.value], *v = s_v[stage.value];
        f32x16 s[HALVES];
        scores(k, s);
        uint32_t held[HALVES];
        if constexpr (masked.value)
#pragma unroll
            for (int h = 0; h < HALVES; ++h)
                held[h] = mask(base + 32 * h, s[h]);
        raise(s);
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
            u32x4 pf[2];
            weights(s[h], pf);
            if constexpr (masked.value)
                masked_product(v, h, base + 32 * h, held[h], pf);
            else
                product(v, h, pf);
        }
    };
    if (u.lo < u.hi) {
        read_pages(u.lo);
        issue(u.lo, Stage0());
        read_pages(u.lo + POS);
    }
    // (in pairs, so that a tile's place in LDS is a constant)
    for (int base = u.lo; base < u.hi;) {
#pragma unroll 1
        for (; base < u.hi && (needs_mask(base) || needs_mask(base + POS)); base += 2 * POS) {
            step(base, Stage0(), Stage1(), std::true_type());
            if (base + POS < u.hi)
                step(base + POS, Stage1(), Stage0(), std::true_type());
        }
#pragma unroll 1
        for (; base < u.hi && !(needs_mask(base) || needs_mask(base + POS)); base += 2 * POS) {
            step(base, Stage0(), Stage1(), std::false_type());
            step(base + POS, Stage1(), Stage0(), std::false_type());
        }
    }
    // Out of the unit, through LDS, so that a row is written whole: straight
    // to the output if the tile has one split, else to the unit's slot for the
    // join kernel.
    __syncthreads();
    constexpr int PIECES_O = DIM / 4;                // 16-byte pieces of a row
    char *rows = s_mem + wave * 32 * DIM * 4;
    sum = sum32(sum);
    // A row is divided by its weights' sum as they were rounded, as far as the
    // largest goes: one key alone gives its value. (1: nothing seen, or NaN)
    const float p0 = exp2_fast(__builtin_fmaf(most, a.scale_log2, -top));
    const float even = sum > 0.f ? sum / (sum + (T::lo(T::pack(p0, p0)) - p0)) : 1.f;
    auto place = [](int row, int p) { return (row * PIECES_O + (p ^ (row % 16))) * 16; };
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int g = 0; g < 4; ++g)
            *reinterpret_cast<f32x4 *>(rows + place(col, 8 * d + 2 * g + half)) =
                f32x4{acc[d][4 * g], acc[d][4 * g + 1], acc[d][4 * g + 2], acc[d][4 * g + 3]} * even;
    if (u.splits == 1 && half == 0 && r < u.nrows)
        write_lse(a, tok, head, top, sum);
    const Slots<DIM, ROWS, 0> slots(a);
    constexpr int PER_PASS = 64 / PIECES_O < 1 ? 1 : 64 / PIECES_O;
    const int p = lane % PIECES_O;
#pragma unroll 4
    for (int i = 0; i < 32; i += PER_PASS) {
        const int row = i + lane / PIECES_O;
        const float m = __shfl(top, row), l = __shfl(sum, row);
        if (wave * 32 + row >= u.nrows)
            continue;
        const f32x4 v = *reinterpret_cast<const f32x4 *>(rows + place(row, p));
        if (u.splits == 1) {
            int t, h;
            row_place(a, u, u.row0 + wave * 32 + row, t, h);
            write_out<T>(a, t, h, 4 * p, v, l, a.gate ? load_gate(a, t, h, 4 * p) : u32x2{0, 0});
        } else {
            slots.put(u.slot0 + u.split, wave * 32 + row, 4 * p, v, m, l);
        }
    }
}

}  // namespace gdp
