// The second launch of the paged attention: joins the parts that row tiles
// were cut in.
#pragma once

#include "attn.h"

namespace gdp {

// Threads in groups of DIM / 4, each thread four elements of a row. Where a
// tile has at most kJoinRun splits a group joins a row by itself; with more, a
// workgroup joins one row: group g takes kJoinRun consecutive splits of every
// GROUPS * kJoinRun, and the groups' results meet in LDS, in order. (Joined in
// the tile kernel by the last of 16 workgroups, splits of 64 rows cost 30 us a
// level.) Bound by its launch and three dependent reads: 7 us for 808 rows of
// up to 32 splits each (15 MB), 5 us where next to nothing was split.
constexpr int kJoinRun = 8;

template <class T, int DIM, int ROWS>
__global__ __launch_bounds__(kJoinThreads) void attn_join(AttnArgs a)
{
    constexpr int PER = DIM / 4;
    constexpr int GROUPS = kJoinThreads / PER;
    __shared__ f32x4 s_o[GROUPS][PER];
    __shared__ float s_m[GROUPS], s_l[GROUPS];
    Partition<ROWS> part(a);
    auto joins = [](const Partition<ROWS> &p) { return p.joins(kJoinRun, GROUPS); };
    const int total = part.total(joins);
    const Slots<DIM, ROWS, 0> slots(a);
    const int g = threadIdx.x / PER, d = 4 * (threadIdx.x % PER);
    for (int id = blockIdx.x; id < total; id += gridDim.x) {
        AttnUnit u;
        int tiles;
        const int local = part.find(id, joins, u, tiles);
        const bool few = u.splits <= kJoinRun;
        const int rows = u.n * a.group, per = few ? GROUPS : 1, blocks = (rows + per - 1) / per;
        u.kvh = local / blocks;
        const int row = (local - u.kvh * blocks) * per + (few ? g : 0);
        if (few && row >= rows)
            continue;
        const int tile = row / ROWS, r = row % ROWS;
        const int first = u.slot0 + (u.kvh * tiles + tile) * u.splits;
        int tok, head;
        row_place(a, u, row, tok, head);
        const u32x2 gate = a.gate && (few || g == 0) ? load_gate(a, tok, head, d) : u32x2{0, 0};
        float top, sum;
        if (few) {
            const f32x4 v = slots.template join<kJoinRun>(first, 1, u.splits, r, d, top, sum);
            write_out<T>(a, tok, head, d, v, sum, gate);
            if (d == 0)
                write_lse(a, tok, head, top, sum);
            continue;
        }
        top = -INFINITY;
        sum = 0.f;
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
        for (int s = g * kJoinRun; s < u.splits; s += GROUPS * kJoinRun) {
            float m, l;
            const f32x4 v = slots.template join<kJoinRun>(first + s, 1, min(kJoinRun, u.splits - s), r, d, m, l);
            const float big = fmaxf(top, m), safe = big == -INFINITY ? 0.f : big;
            const float f = exp2_fast(top - safe), h = exp2_fast(m - safe);
            acc = acc * f + v * h;
            sum = sum * f + l * h;
            top = big;
        }
        s_o[g][d / 4] = acc;
        if (d == 0) {
            s_m[g] = top;
            s_l[g] = sum;
        }
        __syncthreads();
        if (g == 0) {
            const int used = min(GROUPS, (u.splits + kJoinRun - 1) / kJoinRun);
            for (int i = 1; i < used; ++i)
                top = fmaxf(top, s_m[i]);
            const float safe = top == -INFINITY ? 0.f : top;
            acc = f32x4{0.f, 0.f, 0.f, 0.f};
            sum = 0.f;
            for (int i = 0; i < used; ++i) {
                const float f = exp2_fast(s_m[i] - safe);
                acc += s_o[i][d / 4] * f;
                sum += s_l[i] * f;
            }
            write_out<T>(a, tok, head, d, acc, sum, gate);
            if (d == 0)
                write_lse(a, tok, head, top, sum);
        }
        __syncthreads();
    }
}

}  // namespace gdp
