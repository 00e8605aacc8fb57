// Products with 4-bit weights and group scales (include/block.h, blk_w4_*):
//     out[m, n] = sum over groups g of s[n, g] * sum over k in g of (q[n, k] - z[n, g]) x[m, k].
//
// The weights become matrix operands without a conversion instruction: four
// bits or'ed to the end of an FP16 number are that number plus q units of its
// last place, z comes off by one packed subtraction, and BF16 takes two more
// operations on the bits (weight_operand; the conversion of signed nibbles
// takes longer: 2304 x 8192, one token 7.3 us, this way 6.2). So an operand is
// q - z itself, exact: an activation meets nothing else, be it an infinity or
// an outlier on weights of zero. Products are exact, sums FP32, and the scale
// multiplies the group's FP32 sum, so no weight is ever rounded.
//
// Memory bound at the token counts it is for (16 tokens: 64 operations per
// weight byte). A workgroup owns RB blocks of 16 rows and 16 NT tokens; its
// waves split K, each unit of 128 k is one 16-byte load per lane and row
// block, 1 KB contiguous per wave. Measured, BF16: 2304 x 8192, groups of 128,
// one token: 6.2 us (9.9 MB at 1.6 TB/s: 144 row blocks fill little over half
// the card, and the time is a launch, two loads' latency, the operands and the
// join of the waves); 8192 x 4096, groups of 64, 32 tokens: 9.4 us, bound by
// the activations that every workgroup reads from L2.
#include <limits.h>

#include "block_common.h"

namespace gdp {
namespace {

constexpr int kUnitK = 128;            // k per 16-byte load of a lane

// FP16 number with the weight's four bits at its end, and what BF16 operands
// are scaled by (see weight_operand).
template <class T>
constexpr uint32_t w4_magic()
{
    return T::kId == BLK_BF16 ? 0x5800u : 0x6400u;
}
constexpr float kBf16Scale = 524288.f;

struct W4Args {
    const u32x4 *w;                    // [row block][unit][lane]
    const char *scale;                 // [row block][unit][128 / G][16 rows], 16 bits
    const char *zero;                  // same shape: w4_magic + z; nullptr: z = 8
    const char *x;
    char *out;
    int64_t x_stride, out_stride;      // bytes
    int n, k, m, units, blocks;
    int wide_out;                      // output rows take 8-byte stores
};

// The eight weights of w as an operand, q - z in both types (z twice in `z`, as
// the number that is taken off).
//   FP16: 1024 + q by a shift and an and-or, less 1024 + z.
//   BF16 has no packed subtraction: (128 + q / 8) - (128 + z / 8) in FP16. The
//   exponent of (q - z) / 8, 12 to 15 or 0, has its upper three bits alike
//   (011) wherever it is not zero: kept in place with the sign, and repeated
//   above the other two and the significand three bits further down, they make
//   the BF16 number (q - z) 2^-19, or zero.
template <class T>
__device__ __forceinline__ u32x4 weight_operand(uint32_t w, uint32_t z, uint32_t nibbles)
{
    constexpr uint32_t magic = w4_magic<T>() * 0x10001u;
    u32x4 f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t q = ((w >> (4 * j)) & nibbles) | magic;
        const uint32_t h = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, q) - __builtin_bit_cast(f16x2, z));
        f[j] = T::kId == BLK_BF16 ? (h & 0xf000f000u) | (h >> 3 & 0x0fff0fffu) : h;
    }
    return f;
}

// CH units of a wave are loaded at once, weights, scales and activations, all
// in flight before the first product.
//
// Activations are read along the rows, 256 bytes per 16 lanes, and turned to
// operands (column l % 16, k 8 (l / 16) + 0..7 of each 32) by way of LDS,
// 16-byte pieces permuted so that neither side meets a bank conflict: read as
// operands, every four lanes would touch four rows (8192 x 3968, 16 tokens:
// 10.4 us, this way 8.1). DIRECT reads them as operands all the same: for one
// or two tokens the lanes' rows coincide (one token: 6.2 us against 7.6).
template <class T, int G, int RB, int NT, int CH, int WAVES, bool DIRECT>
__global__ __launch_bounds__(64 * WAVES) void w4_kernel(W4Args a)
{
    constexpr bool BF = T::kId == BLK_BF16;
    constexpr int GPU_ = kUnitK / G;   // groups per unit
    constexpr int SPG = G / 32;        // k-steps per group
    // Each wave's activations of a unit, 16 tokens x 256 bytes per block; at the
    // end the waves' sums.
    constexpr int XB = 16 * kUnitK * 2;
    constexpr int LDSB = WAVES * (NT * XB > RB * NT * 1024 ? NT * XB : RB * NT * 1024);
    __shared__ __align__(16) char s_mem[LDSB];
    f32x4(&s_part)[WAVES][RB * NT][kWave] = *reinterpret_cast<f32x4(*)[WAVES][RB * NT][kWave]>(s_mem);
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int col = lane % 16, quad = lane / 16;
    const int rb0 = blockIdx.x * RB;
    const int tok0 = blockIdx.y * 16 * NT;
    const int u0 = (int)((int64_t)wave * a.units / WAVES), u1 = (int)((int64_t)(wave + 1) * a.units / WAVES);

    char *xl = s_mem + wave * NT * XB;
    const char *xp[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            xp[t][i] = a.x + (int64_t)min(tok0 + 16 * t + (DIRECT ? col : 4 * i + quad), a.m - 1) * a.x_stride;
    int64_t block[RB];                 // the row blocks' first units; past the last block, the last again
#pragma unroll
    for (int r = 0; r < RB; ++r)
        block[r] = (int64_t)min(rb0 + r, a.blocks - 1) * a.units;

    f32x4 acc[RB][NT];
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t)
            acc[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    // (in a vector register, which an and-or can take next to the other constant)
    uint32_t nibbles = 0x000f000fu;
    asm volatile("" : "+v"(nibbles));

    for (int first = u0; first < u1; first += CH) {
        u32x4 w[CH][RB], xf[CH][NT][4];
        u32x2 sc[CH][GPU_][RB];
        uint32_t zc[CH][GPU_][RB];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            // Units past the wave's last load that one again; k past the
            // matrix loads its last eight again. Neither is used.
            const int u = min(first + c, u1 - 1);
#pragma unroll
            for (int r = 0; r < RB; ++r)
                w[c][r] = a.w[(block[r] + u) * kWave + lane];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    xf[c][t][i] = *reinterpret_cast<const u32x4 *>(
                        xp[t][i] + (int64_t)min(u * kUnitK + 8 * (DIRECT ? 4 * i + quad : col), a.k - 8) * 2);
#pragma unroll
            for (int g = 0; g < GPU_; ++g)
#pragma unroll
                for (int r = 0; r < RB; ++r) {
                    const int64_t group = ((block[r] + u) * GPU_ + g) * 32;
                    sc[c][g][r] = *reinterpret_cast<const u32x2 *>(a.scale + group + quad * 8);
                    // (as loaded: an operation on it here would wait for it)
                    zc[c][g][r] = w4_magic<T>() | 8u;
                    if (a.zero)
                        zc[c][g][r] = *reinterpret_cast<const uint16_t *>(a.zero + group + col * 2);
                }
        }
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            if (first + c >= u1)
                break;
            if constexpr (!DIRECT) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int tok = 4 * i + quad;
                        *reinterpret_cast<u32x4 *>(xl + t * XB + tok * 256 + (col ^ tok) * 16) = xf[c][t][i];
                    }
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        xf[c][t][s] =
                            *reinterpret_cast<const u32x4 *>(xl + t * XB + col * 256 + ((4 * s + quad) ^ col) * 16);
            }
#pragma unroll
            for (int g = 0; g < GPU_; ++g) {
                if ((first + c) * kUnitK + G * g >= a.k)
                    break;
#pragma unroll
                for (int r = 0; r < RB; ++r) {
                    f32x4 part[NT];
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        part[t] = f32x4{0.f, 0.f, 0.f, 0.f};
                    const uint32_t z = __builtin_amdgcn_perm(0u, zc[c][g][r], 0x01000100u);
#pragma unroll
                    for (int s = 0; s < SPG; ++s) {
                        const u32x4 wf = weight_operand<T>(w[c][r][g * SPG + s], z, nibbles);
#pragma unroll
                        for (int t = 0; t < NT; ++t)
                            part[t] = T::mfma16(wf, xf[c][t][g * SPG + s], part[t]);
                    }
                    const u32x2 s2 = sc[c][g][r];
                    const float sf[4] = {T::lo(s2.x), T::hi(s2.x), T::lo(s2.y), T::hi(s2.y)};
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            acc[r][t][i] += sf[i] * part[t][i];
                }
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t)
            s_part[wave][r * NT + t][lane] = acc[r][t];
    __syncthreads();
    for (int i = wave; i < RB * NT; i += WAVES) {
        const int r = i / NT, t = i % NT;
        f32x4 v = s_part[0][i][lane];
#pragma unroll
        for (int w = 1; w < WAVES; ++w)
            v += s_part[w][i][lane];
        if constexpr (BF)
            v *= kBf16Scale;
        const int tok = tok0 + 16 * t + col;
        const int row = (rb0 + r) * 16 + 4 * quad;
        if (tok >= a.m || row >= a.n)
            continue;
        char *o = a.out + (int64_t)tok * a.out_stride + (int64_t)row * 2;
        const u32x2 p = {T::pack(v.x, v.y), T::pack(v.z, v.w)};
        if (a.wide_out) {
            *reinterpret_cast<u32x2 *>(o) = p;
        } else {
            const uint16_t h[4] = {(uint16_t)p.x, (uint16_t)(p.x >> 16), (uint16_t)p.y, (uint16_t)(p.y >> 16)};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (row + e < a.n)
                    reinterpret_cast<uint16_t *>(o)[e] = h[e];
        }
    }
}

// Packing: the operand order of the weights. Dword s of lane l's 16 bytes
// holds the eight weights of row l % 16, k = 128 unit + 32 s + 8 (l / 16) +
// 0..7, element 2j at bit 4j and 2j + 1 at bit 16 + 4j. Rows past n and k past
// the matrix are zero.
__global__ void w4_pack_kernel(const uint8_t *q, int64_t row_bytes, u32x4 *dst, int n, int k, int units, int64_t total)
{
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= total)
        return;
    const int lane = (int)(id % kWave);
    const int u = (int)(id / kWave % units);
    const int row = (int)(id / kWave / units) * 16 + lane % 16;
    u32x4 v;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        const int k0 = u * kUnitK + 32 * s + 8 * (lane / 16);
        uint32_t w = 0;
        if (row < n && k0 < k)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t b = q[row * row_bytes + k0 / 2 + j];
                w |= (b & 15u) << (4 * j) | (b >> 4) << (16 + 4 * j);
            }
        v[s] = w;
    }
    dst[id] = v;
}

template <class T>
__global__ void w4_pack_scales_kernel(const uint16_t *scales, const uint8_t *zeros, uint16_t *dscale, uint16_t *dzero,
                                      int n, int groups, int padded, int64_t total)
{
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= total)
        return;
    const int g = (int)(id / 16 % padded);
    const int row = (int)(id / 16 / padded) * 16 + (int)(id % 16);
    const bool in = row < n && g < groups;
    dscale[id] = in ? scales[(int64_t)row * groups + g] : 0;
    if (zeros) {
        // z of one byte, 0..15.
        dzero[id] = (uint16_t)(w4_magic<T>() | (in ? zeros[(int64_t)row * groups + g] & 15u : 8u));
    }
}

struct W4Plan {
    void (*fn)(W4Args);
    int rb, nt, waves;
};

// Rounds that `wgs` workgroups take, one per compute unit at a time.
int rounds(int64_t wgs) { return (int)((wgs + 255) / 256); }

// Row blocks per workgroup by the rounds that result, times what a round takes
// relative to the others. (Times in us, BF16, no zeros, k = 8192 if not stated.
// 4096 rows are one round of one block, 5120 the first two.)
//   up to 16 tokens   4096 rows: one block 8.1, two 10.8; 5120 rows: 12.6, 10.6;
//                     12288 rows: 18.9, 16.8: 3 to 4
//   more, tiles of 32 32 tokens, 4096 rows: one block 11.3, two 13.2, four 20.6;
//                     5120 rows: 16.7, 13.1, 20.6; 12288 rows: 23.3, 24.2, 22.1;
//                     64 tokens, 12288 rows: 42.3, 36.7, 40.4; 1000 tokens, 8192
//                     rows: 414, 357, 298: 17 to 20 to 32
template <class T, int G>
W4Plan pick(int m, int blocks, int units)
{
    if (m <= 16) {
        const bool two = 4 * rounds((blocks + 1) / 2) < 3 * rounds(blocks);
        // Short k: one unit per wave and turn (k = 2048, 8192 rows, 4 tokens: 4.5;
        // two of 16 waves 6.1).
        if (units < 32)
            return two ? W4Plan{w4_kernel<T, G, 2, 1, 1, 8, false>, 2, 1, 8}
                       : W4Plan{w4_kernel<T, G, 1, 1, 1, 8, false>, 1, 1, 8};
        // (one token, 4096 rows: 6.9, the next 7.5; 12288 rows: 15.0, two blocks 16.5)
        if (m <= 2)
            return {w4_kernel<T, G, 1, 1, 4, 8, true>, 1, 1, 8};
        return two ? W4Plan{w4_kernel<T, G, 2, 1, 1, 8, false>, 2, 1, 8}
                   : W4Plan{w4_kernel<T, G, 1, 1, 2, 16, false>, 1, 1, 16};
    }
    const int64_t tiles = (m + 31) / 32;
    const int64_t one = 17ll * rounds(blocks * tiles), two = 20ll * rounds((blocks + 1) / 2 * tiles),
                  four = 32ll * rounds((blocks + 3) / 4 * tiles);
    if (one <= two && one <= four)
        return {w4_kernel<T, G, 1, 2, 2, 8, false>, 1, 2, 8};
    if (two <= four)
        return {w4_kernel<T, G, 2, 2, 1, 16, false>, 2, 2, 16};
    return {w4_kernel<T, G, 4, 2, 2, 8, false>, 4, 2, 8};
}

template <class T>
W4Plan pick(int group, int m, int blocks, int units)
{
    return group == 32   ? pick<T, 32>(m, blocks, units)
           : group == 64 ? pick<T, 64>(m, blocks, units)
                         : pick<T, 128>(m, blocks, units);
}

struct Layout {
    int units, blocks, padded;
    size_t w, scale;                   // bytes of the weights, of the scales (and of the zeros)
};

bool layout(const blk_w4 *w, Layout &l)
{
    if (w->n < 1 || w->k < 1 || w->n > (1 << 24) || w->k > (1 << 24) || (w->group != 32 && w->group != 64 && w->group != 128) ||
        w->k % w->group || (w->dtype != BLK_BF16 && w->dtype != BLK_F16))
        return false;
    l.units = (w->k + kUnitK - 1) / kUnitK;
    l.blocks = (w->n + 15) / 16;
    l.padded = l.units * (kUnitK / w->group);
    l.w = (size_t)l.blocks * l.units * 1024;
    l.scale = (size_t)l.blocks * l.padded * 32;
    return true;
}

}  // namespace
}  // namespace gdp

using namespace gdp;

extern "C" {

size_t blk_w4_packed_bytes(const blk_w4 *w)
{
    Layout l;
    return w && layout(w, l) ? l.w + l.scale * (w->has_zeros ? 2 : 1) : 0;
}

int blk_w4_pack(const blk_w4 *w, const void *q, const void *scales, const void *zeros, void *packed, void *stream)
{
    Layout l;
    if (!w)
        return PROJ_ERR_NULL;
    if (!layout(w, l))
        return PROJ_ERR_ARG;
    if (!q || !scales || !packed || !zeros != !w->has_zeros)
        return PROJ_ERR_NULL;
    if (!aligned_to(packed, 16) || !aligned_to(scales, 2))
        return PROJ_ERR_ALIGN;
    const int64_t wt = (int64_t)l.blocks * l.units * kWave, st = (int64_t)l.blocks * l.padded * 16;
    if (wt / 256 >= INT_MAX || st / 256 >= INT_MAX)
        return PROJ_ERR_ARG;
    char *p = static_cast<char *>(packed);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    hipLaunchKernelGGL(w4_pack_kernel, dim3((unsigned)((wt + 255) / 256)), dim3(256), 0, s,
                       static_cast<const uint8_t *>(q), (int64_t)w->k / 2, reinterpret_cast<u32x4 *>(p), w->n, w->k,
                       l.units, wt);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return hip_fail(e);
    auto *kernel = w->dtype == BLK_BF16 ? w4_pack_scales_kernel<BF16> : w4_pack_scales_kernel<F16>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)((st + 255) / 256)), dim3(256), 0, s,
                       static_cast<const uint16_t *>(scales), static_cast<const uint8_t *>(zeros),
                       reinterpret_cast<uint16_t *>(p + l.w), reinterpret_cast<uint16_t *>(p + l.w + l.scale), w->n,
                       w->k / w->group, l.padded, st);
    e = hipGetLastError();
    return e == hipSuccess ? PROJ_OK : hip_fail(e);
}

int blk_w4_run(const blk_w4 *w, const void *packed, const void *x, int64_t x_stride, int m, void *out,
               int64_t out_stride, void *stream)
{
    Layout l;
    if (!w)
        return PROJ_ERR_NULL;
    x_stride = stride_of(x_stride, m);
    out_stride = stride_of(out_stride, m);
    if (!layout(w, l) || m < 0 || m > (1 << 20) || x_stride < 0 || x_stride % 8 || out_stride < 0 ||
        x_stride >= ((int64_t)1 << 40) || out_stride >= ((int64_t)1 << 40) || !rows_apart<1>(w->n, {out_stride}, {m}))
        return PROJ_ERR_ARG;
    if (m == 0)
        return PROJ_OK;
    if (!packed || !x || !out)
        return PROJ_ERR_NULL;
    if (!aligned_to(packed, 16) || !aligned_to(x, 16) || !aligned_to(out, 2))
        return PROJ_ERR_ALIGN;
    const char *p = static_cast<const char *>(packed);
    W4Args a{};
    a.w = reinterpret_cast<const u32x4 *>(p);
    a.scale = p + l.w;
    a.zero = w->has_zeros ? p + l.w + l.scale : nullptr;
    a.x = static_cast<const char *>(x);
    a.out = static_cast<char *>(out);
    a.x_stride = x_stride * 2;
    a.out_stride = out_stride * 2;
    a.n = w->n;
    a.k = w->k;
    a.m = m;
    a.units = l.units;
    a.blocks = l.blocks;
    a.wide_out = w->n % 4 == 0 && out_stride % 4 == 0 && aligned_to(out, 8);
    const W4Plan plan = w->dtype == BLK_BF16 ? pick<BF16>(w->group, m, l.blocks, l.units)
                                             : pick<F16>(w->group, m, l.blocks, l.units);
    void *params[1] = {&a};
    const hipError_t e = hipLaunchKernel(
        reinterpret_cast<const void *>(plan.fn),
        dim3((l.blocks + plan.rb - 1) / plan.rb, (m + 16 * plan.nt - 1) / (16 * plan.nt)), dim3(64 * plan.waves), params,
        0, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? PROJ_OK : hip_fail(e);
}

}  // extern "C"
