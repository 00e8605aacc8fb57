// The second launch of the paged attention: joins the parts that row tiles
// were cut in.
#pragma once

#include "attn.h"

namespace gdp {

// Joins the splits of a tile kernel's rows, one row per workgroup and pass:
// threads in groups of DIM / 4, group g takes kJoinRun consecutive splits of
// every kJoinThreads / (DIM / 4) * kJoinRun, each thread four elements; the
// groups' results meet in LDS, in order. Splits of 64 to 128 rows are too much
// for one workgroup per tile: joined in the tile kernel by the last of 16
// workgroups they cost 30 us a level.
constexpr int kJoinRun = 8;

template <class T, int DIM, int ROWS>
__global__ __launch_bounds__(kJoinThreads) void attn_join(AttnArgs a)
{
    constexpr int PER = DIM / 4;
    constexpr int GROUPS = kJoinThreads / PER;
    __shared__ f32x4 s_o[GROUPS][PER];
    __shared__ float s_m[GROUPS], s_l[GROUPS];
    Partition<ROWS> part(a);
    auto joins = [](const Partition<ROWS> &p) { return p.joins(); };
    const int total = part.total(joins);
    const Slots<DIM, ROWS> slots(a);
    const int g = threadIdx.x / PER, lane = threadIdx.x % PER;
    for (int id = blockIdx.x; id < total; id += gridDim.x) {
        AttnUnit u;
        int tiles;
        const int local = part.find(id, joins, u, tiles);
        const int rows = u.n * a.group;
        u.kvh = local / rows;
        const int row = local - u.kvh * rows;
        const int tile = row / ROWS;
        const int first = u.slot0 + (u.kvh * tiles + tile) * u.splits;
        int tok, head;
        row_place(a, u, row, tok, head);
        const u32x2 gate = a.gate ? load_gate(a, tok, head, 4 * lane) : u32x2{0, 0};
        float top = -INFINITY, sum = 0.f;
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
        for (int s = g * kJoinRun; s < u.splits; s += GROUPS * kJoinRun) {
            float m, l;
            const f32x4 v = slots.template join<kJoinRun>(first + s, 1, min(kJoinRun, u.splits - s), row - tile * ROWS,
                                                          4 * lane, m, l);
            const float big = fmaxf(top, m), safe = big == -INFINITY ? 0.f : big;
            const float f = exp2_fast(top - safe), h = exp2_fast(m - safe);
            acc = acc * f + v * h;
            sum = sum * f + l * h;
            top = big;
        }
        s_o[g][lane] = acc;
        if (lane == 0) {
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
                acc += s_o[i][lane] * f;
                sum += s_l[i] * f;
            }
            write_out<T>(a, tok, head, 4 * lane, acc, sum, gate);
            if (lane == 0)
                write_lse(a, tok, head, top, sum);
        }
        __syncthreads();
    }
}

}  // namespace gdp
