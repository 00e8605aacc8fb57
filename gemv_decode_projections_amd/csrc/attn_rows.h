// Attention of few rows (up to 32 per tile: single tokens, a few drafted ones)
// over a paged cache. Memory bound: every key and value is read once, as long
// as a sequence's rows fit one tile, and straight into registers.
//
// Mathematics, per tile of R = 16 NB rows and step of 32 positions, on
// v_mfma 16x16x32 (geometry in common.h):
//   S^T (32 x R) = K Q^T      A = keys (row l%16, elements 8(l/16)..+7 of each
//                             32), B = the rows' queries;
//   O^T (DIM x R) += V^T P^T  A = values transposed, B = P^T.
// The score fragment of lane l holds column (row of the tile) l%16 and
// positions 4(l/16) + i of each 16: the softmax of a row sits in four lanes,
// and its eight probabilities are exactly the k slots of a B operand if A
// uses the same order of positions, 4q..4q+3 and 16+4q..16+4q+3 for quad q.
// So a lane reads those eight positions' values, VEC = 8 (4 for DIM 64)
// consecutive elements each, 256 contiguous bytes per 16 lanes, and an
// in-lane transposition (one byte permute per two elements) makes the VEC A
// operands: operand j holds elements VEC * (l%16) + j. Nothing crosses LDS
// until the four waves, which take every fourth step, join at the end.
//
// Measured, BF16, heads of 128: 32 sequences of one token over 146 k positions
// in all, 32 heads on 8: 121 us for 596 MB, 4.9 TB/s, bound by HBM. One token
// over 1000 positions, 8 heads on 1: 8.3 us a call, bound by round trips to
// memory that follow one another (lengths, table, keys, join of 8 parts).
#pragma once

#include "attn.h"

namespace gdp {

// Transposes 8 positions x VEC elements of 16 bits held by one lane into VEC
// fragments of 8 positions: fragment j = element j of positions 0..7.
template <int VEC>
__device__ __forceinline__ void transpose8(const uint32_t (&in)[8][VEC / 2], u32x4 (&out)[VEC])
{
#pragma unroll
    for (int j = 0; j < VEC; ++j)
#pragma unroll
        for (int p = 0; p < 4; ++p)
            out[j][p] = __builtin_amdgcn_perm(in[2 * p + 1][j / 2], in[2 * p][j / 2],
                                              j % 2 ? 0x07060302u : 0x05040100u);
}

constexpr int kJoin = 16;

// Two waves per SIMD where the accumulators leave room for them.
template <class T, int DIM, int NB>
__global__ __launch_bounds__(256, DIM * NB <= 256 && DIM < 256 ? 2 : 1) void attn_rows(AttnArgs a)
{
    constexpr int ROWS = 16 * NB;
    constexpr int WAVES = 4;
    constexpr int KS = DIM / 32;                     // k-steps of Q K^T
    constexpr int VEC = DIM >= 128 ? 8 : DIM / 16;   // consecutive elements per lane and value row
    constexpr int HALF = DIM / (16 * VEC);           // 16 * VEC element blocks of a value row
    constexpr int PITCH = DIM + 4;
    constexpr int STEP = 32;
    constexpr bool TWO_PARTS = NB == 1;              // of the probabilities
    // The largest weight is 2^ABOVE, in FP16 the largest power of the type: weights
    // down to 2^-29 of it are normal numbers.
    constexpr float ABOVE = T::kId == BLK_F16 ? 15.0f : 0.0f;
    constexpr int PER = DIM / 4;               // threads per row when rows leave
    constexpr int RSTEP = 64 * WAVES / PER;    // rows per pass then
    constexpr int PASSES = (ROWS + RSTEP - 1) / RSTEP;
    __shared__ __align__(16) float s_o[WAVES][ROWS * PITCH];
    __shared__ float s_m[WAVES][ROWS], s_l[WAVES][ROWS];
    __shared__ u32x2 s_gate[PASSES][64 * WAVES];
    __shared__ int s_flag;

    AttnUnit u;
    if (!find_unit<ROWS>(a, blockIdx.x, u))
        return;
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int col = lane % 16, quad = lane / 16;

    // The tile's queries as B operands; rows past the last read it again and
    // see nothing.
    u32x4 qf[NB][KS];
    int see_lo[NB], see_hi[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        const int r = nb * 16 + col;
        int tok, head;
        row_place(a, u, u.row0 + min(r, u.nrows - 1), tok, head);
        const char *p = a.q + tok * a.q_stride + head * a.q_head + quad * 16;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
            qf[nb][ks] = *reinterpret_cast<const u32x4 *>(p + ks * 64);
        const int pos = u.len - u.n + tok - u.tok0;
        see_hi[nb] = r < u.nrows ? pos + 1 : 0;
        see_lo[nb] = a.window > 0 ? pos - a.window + 1 : 0;
    }
    // Positions that every row of the tile sees need no mask.
    const int i0 = a.by_group(u.row0), i1 = a.by_group(u.row0 + u.nrows - 1);
    const int all_hi = u.len - u.n + i0 + 1;
    const int all_lo = a.window > 0 ? u.len - u.n + i1 - a.window + 1 : 0;

    f32x4 acc[NB][HALF][VEC];
    float top[NB], sum[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        top[nb] = -INFINITY;
        sum[nb] = 0.f;
#pragma unroll
        for (int h = 0; h < HALF; ++h)
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                acc[nb][h][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    const int32_t *table = a.table + (int64_t)u.seq * a.table_stride;
    const int64_t head_off = (int64_t)u.kvh * a.head_stride;
    auto page_of = [&](int p) { return table[min(p >> a.page_shift, a.table_width - 1)]; };
    // Per step: the pages of the lane's two key rows and of its two groups of
    // four value rows (four aligned positions share a page).
    struct Pages {
        int k[2], v[2];
    };
    auto load_pages = [&](int base) {
        Pages pg;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            pg.k[t] = page_of(base + 16 * t + col);
            pg.v[t] = page_of(base + 16 * t + 4 * quad);
        }
        return pg;
    };
    u32x4 kf[2][KS];
    uint32_t vr[HALF][8][VEC / 2];
    auto load_k = [&](int base, const Pages &pg) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            int64_t off;
            kv_offset(a, pg.k[t], base + 16 * t + col, head_off, off);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
                kf[t][ks] = *reinterpret_cast<const u32x4 *>(a.k + off + quad * 16 + ks * 64);
        }
    };
    auto load_v = [&](int base, const Pages &pg) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            int64_t off;
            kv_offset(a, pg.v[t], base + 16 * t + 4 * quad, head_off, off);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int h = 0; h < HALF; ++h) {
                    const char *p = a.v + off + (int64_t)i * a.token_stride + (h * 16 * VEC + col * VEC) * 2;
                    if constexpr (VEC == 8) {
                        const u32x4 x = *reinterpret_cast<const u32x4 *>(p);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            vr[h][4 * t + i][e] = x[e];
                    } else {
                        const u32x2 x = *reinterpret_cast<const u32x2 *>(p);
                        vr[h][4 * t + i][0] = x.x;
                        vr[h][4 * t + i][1] = x.y;
                    }
                }
        }
    };

    int base = u.lo + wave * STEP;
    Pages pg = {}, next = {};
    if (base < u.hi) {
        pg = load_pages(base);
        next = load_pages(base + WAVES * STEP);
        load_k(base, pg);
        load_v(base, pg);
    }
    // The gate waits in LDS for the end, read by the thread that will use it.
    const int d = 4 * (threadIdx.x % PER), r0 = threadIdx.x / PER;
    if (a.gate)
#pragma unroll
        for (int k = 0; k < PASSES; ++k) {
            int tok, head;
            row_place(a, u, u.row0 + min(r0 + k * RSTEP, u.nrows - 1), tok, head);
            s_gate[k][threadIdx.x] = load_gate(a, tok, head, d);
        }
    for (; base < u.hi; base += WAVES * STEP) {
        const int after = base + WAVES * STEP;
        f32x4 s[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                s[nb][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
                    s[nb][t] = T::mfma16(kf[t][ks], qf[nb][ks], s[nb][t]);
            }
        // The keys are in the scores: the next step's may take their registers.
        const Pages coming = load_pages(min(after + WAVES * STEP, u.hi - 1));
        if (after < u.hi)
            load_k(after, next);
        bool ok[2];
#pragma unroll
        for (int t = 0; t < 2; ++t)
            ok[t] = (unsigned)pg.v[t] < (unsigned)a.n_pages;
        const bool masked = base < all_lo || base + STEP > all_hi || base + STEP > u.hi || !__all(ok[0] && ok[1]);
        bool poisoned = false;
        if (masked) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int p = base + 16 * t + 4 * quad + i;
                    const bool held = ok[t] && p < u.hi;
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
                        if (!(held && p >= see_lo[nb] && p < see_hi[nb]))
                            s[nb][t][i] = -INFINITY;
                    // What lies past the last token is not the cache's: 0 * NaN.
#pragma unroll
                    for (int h = 0; h < HALF; ++h)
#pragma unroll
                        for (int e = 0; e < VEC / 2; ++e)
                            vr[h][4 * t + i][e] = held ? vr[h][4 * t + i][e] : 0u;
                }
            // A value that only some rows see may be an infinity or a NaN, which
            // a zero weight does not silence in a product: it is left out of
            // the product and added to the rows that see it.
            FiniteCheck<T> check;
#pragma unroll
            for (int h = 0; h < HALF; ++h)
#pragma unroll
                for (int p = 0; p < 8; ++p)
#pragma unroll
                    for (int e = 0; e < VEC / 2; ++e)
                        check.add(vr[h][p][e]);
            poisoned = __any(check.fails());
            if (poisoned)
#pragma unroll
                for (int h = 0; h < HALF; ++h)
#pragma unroll
                    for (int p = 0; p < 8; ++p)
#pragma unroll
                        for (int e = 0; e < VEC / 2; ++e)
                            vr[h][p][e] = finite_only<T>(vr[h][p][e]);
        }
        u32x4 pf[NB], rest[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            float m = -INFINITY;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[nb][t][i] *= a.scale_log2;
                    m = fmaxf(m, s[nb][t][i]);
                }
            m = fmaxf(top[nb], max_quads(m) - ABOVE);
            if (__any(m > top[nb])) {
                const float f = exp2_fast(top[nb] - (m == -INFINITY ? 0.f : m));
                top[nb] = m;
                sum[nb] *= f;
#pragma unroll
                for (int h = 0; h < HALF; ++h)
#pragma unroll
                    for (int j = 0; j < VEC; ++j)
                        acc[nb][h][j] *= f;
            }
            const float safe = m == -INFINITY ? 0.f : m;
            float p[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                p[e] = exp2_fast(s[nb][e / 4][e % 4] - safe);
                sum[nb] += p[e];
            }
            // Probabilities in 16 bits for the matrix instruction: each within
            // half a unit of the type, errors that average out over a row (the
            // largest is a power of two); the sum keeps the unrounded ones. Of
            // 16 rows what rounding left is multiplied as well, in the time
            // that the loads take anyway (of 32 rows of 256 it takes 12 %).
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                pf[nb][e] = T::pack(p[2 * e], p[2 * e + 1]);
                if constexpr (TWO_PARTS)
                    rest[nb][e] = T::pack(p[2 * e] - T::lo(pf[nb][e]), p[2 * e + 1] - T::hi(pf[nb][e]));
            }
        }
#pragma unroll
        for (int h = 0; h < HALF; ++h) {
            u32x4 vt[VEC];
            transpose8<VEC>(vr[h], vt);
#pragma unroll
            for (int j = 0; j < VEC; ++j)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    if constexpr (TWO_PARTS)
                        acc[nb][h][j] = T::mfma16(vt[j], rest[nb], acc[nb][h][j]);
                    acc[nb][h][j] = T::mfma16(vt[j], pf[nb], acc[nb][h][j]);
                }
        }
        if (poisoned)
            for (int pos = 0; pos < STEP; ++pos) {
                int64_t off;
                if (base + pos >= u.hi || !kv_offset(a, page_of(base + pos), base + pos, head_off, off))
                    continue;
                const char *p = a.v + off + VEC * 4 * quad * 2;
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    const int slot = pos / 16 * 4 + pos % 4;
                    const uint32_t pair = slot < 2 ? pf[nb][0] : slot < 4 ? pf[nb][1] : slot < 6 ? pf[nb][2] : pf[nb][3];
                    const float w = __shfl(slot % 2 ? T::hi(pair) : T::lo(pair), pos / 4 % 4 * 16 + col);
                    if (base + pos < see_lo[nb] || base + pos >= see_hi[nb])
                        continue;
#pragma unroll
                    for (int h = 0; h < HALF; ++h)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int j = 0; j < VEC; j += 2) {
                                const uint32_t x =
                                    *reinterpret_cast<const uint32_t *>(p + (h * 16 * VEC + VEC * i + j) * 2);
                                if (!__builtin_isfinite(T::lo(x)))
                                    acc[nb][h][j][i] += w * T::lo(x);
                                if (!__builtin_isfinite(T::hi(x)))
                                    acc[nb][h][j + 1][i] += w * T::hi(x);
                            }
                }
            }
        if (after < u.hi)
            load_v(after, next);
        pg = next;
        next = coming;
    }

    // Join the waves: each leaves its rows, maxima and sums in LDS.
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        const int r = nb * 16 + col;
        sum[nb] = sum_quads(sum[nb]);
        if (quad == 0) {
            s_m[wave][r] = top[nb];
            s_l[wave][r] = sum[nb];
        }
#pragma unroll
        for (int h = 0; h < HALF; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < VEC; j += 4)
                    *reinterpret_cast<f32x4 *>(s_o[wave] + r * PITCH + h * 16 * VEC + VEC * (4 * quad + i) + j) =
                        f32x4{acc[nb][h][j][i], acc[nb][h][j + 1][i], acc[nb][h][j + 2][i], acc[nb][h][j + 3][i]};
    }
    __syncthreads();

    // Out of the unit: straight to the output if the tile has one split.
    // Otherwise the rows are published in the unit's slot. With 32 rows a
    // second launch joins them. With 16 the arrival is counted; the last of
    // every kJoin consecutive splits joins those, and where there are more
    // splits the joins are joined the same way, each result in the slot of its
    // first split. A join thus reads at most kJoin slots, all loads in flight,
    // and always in split order: the result does not depend on who came last.
    // (When it was chosen: one token over 1000 positions 9.7 us, with the second
    // launch 12.4; 24 rows x 16 sequences of up to 16384 positions 24.7 to 39
    // us, with the second launch 20.)
    auto leave = [&](int r, f32x4 v, float m, float l) {
        int tok, head;
        row_place(a, u, u.row0 + r, tok, head);
        write_out<T>(a, tok, head, d, v, l, a.gate ? s_gate[(r - r0) / RSTEP][threadIdx.x] : u32x2{0, 0});
        if (d == 0)
            write_lse(a, tok, head, m, l);
    };
    const Slots<DIM, ROWS, NB == 1 ? kDeviceScope : 0> slots(a);
#pragma unroll 1
    for (int r = r0; r < u.nrows; r += RSTEP) {
        float m = s_m[0][r];
#pragma unroll
        for (int w = 1; w < WAVES; ++w)
            m = fmaxf(m, s_m[w][r]);
        const float safe = m == -INFINITY ? 0.f : m;
        float l = 0.f;
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const float f = exp2_fast(s_m[w][r] - safe);
            l += f * s_l[w][r];
            v += f * *reinterpret_cast<const f32x4 *>(s_o[w] + r * PITCH + d);
        }
        if (u.splits == 1)
            leave(r, v, m, l);
        else
            slots.put(u.slot0 + u.split, r, d, v, m, l);
    }
    if (u.splits == 1 || NB > 1)
        return;
#pragma unroll 1
    for (int stride = 1, level = 0;; stride *= kJoin, ++level) {
        const int first = u.split / (stride * kJoin) * (stride * kJoin);
        const int members = min(kJoin, (u.splits - first + stride - 1) / stride);
        // Alone at its level (257 splits: the last one, of the second level): the
        // slot stays as it is, and there is nothing to count.
        if (members == 1)
            continue;
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (threadIdx.x == 0) {
            // Counters of the levels lie at slots of different remainders, and
            // among the tile's own: two members are more than `level` slots apart.
            uint32_t *c = a.counters + u.slot0 + first + level;
            const uint32_t before = __hip_atomic_fetch_add(c, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            const bool last = before == (uint32_t)(members - 1);
            if (last)
                __hip_atomic_store(c, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            s_flag = last;
        }
        __syncthreads();
        if (!s_flag)
            return;
        const bool done = first == 0 && stride * kJoin >= u.splits;
#pragma unroll 1
        for (int r = r0; r < u.nrows; r += RSTEP) {
            float m, l;
            const f32x4 v =
                members <= kJoin / 2 ? slots.template join<kJoin / 2>(u.slot0 + first, stride, members, r, d, m, l)
                                     : slots.template join<kJoin>(u.slot0 + first, stride, members, r, d, m, l);
            if (done)
                leave(r, v, m, l);
            else
                slots.put(u.slot0 + first, r, d, v, m, l);
        }
        if (done)
            return;
    }
}

}  // namespace gdp
