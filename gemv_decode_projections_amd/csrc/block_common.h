// Shared pieces of the decode-block operators (include/block.h): element
// types, lane exchanges, coherent workspace access, host-side checks.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <array>

#include "../../include/block.h"
#include "../../include/proj.h"
#include "common.h"

namespace gdp {

// Records a failed HIP call for proj_last_hip_error; returns PROJ_ERR_HIP.
int hip_fail(hipError_t e);

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

struct BF16 {
    static constexpr int kId = BLK_BF16;
    static __device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) { return mfma16x16x32(a, b, c); }
    static __device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return pack_bf16x2(lo, hi); }
    static __device__ __forceinline__ float lo(uint32_t u) { return __builtin_bit_cast(float, u << 16); }
    static __device__ __forceinline__ float hi(uint32_t u) { return __builtin_bit_cast(float, u & 0xffff0000u); }
    static constexpr uint32_t kExponent = 0x7f80u;
};

struct F16 {
    static constexpr int kId = BLK_F16;
    static __device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                      0, 0);
    }
    static __device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                      0, 0);
    }
    // Round to nearest, ties to even (the packed conversion instruction truncates).
    static __device__ __forceinline__ uint32_t pack(float lo, float hi)
    {
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, f16x2));
    }
    static __device__ __forceinline__ float lo(uint32_t u) { return (float)__builtin_bit_cast(f16x2, u).x; }
    static __device__ __forceinline__ float hi(uint32_t u) { return (float)__builtin_bit_cast(f16x2, u).y; }
    static constexpr uint32_t kExponent = 0x7c00u;
};

// Whether packed values hold an infinity or a NaN: two operations per pair,
// the largest magnitude bits, and one comparison at the end.
template <class T>
struct FiniteCheck {
    typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
    u16x2 top = {0, 0};
    __device__ __forceinline__ void add(uint32_t u)
    {
        top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, u & 0x7fff7fffu));
    }
    __device__ __forceinline__ bool fails() const { return top.x >= T::kExponent || top.y >= T::kExponent; }
};
// Both values with those replaced by zero.
template <class T>
__device__ __forceinline__ uint32_t finite_only(uint32_t u)
{
    constexpr uint32_t e = T::kExponent;
    return ((u & e) == e ? 0u : u & 0xffffu) | ((u & (e << 16)) == (e << 16) ? 0u : u & 0xffff0000u);
}

// x combined with the lane 16 / 32 away, in the vector unit (no LDS trip).
__device__ __forceinline__ float other16(float x, float &same)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    same = __builtin_bit_cast(float, (uint32_t)r[0]);
    return __builtin_bit_cast(float, (uint32_t)r[1]);
}
__device__ __forceinline__ float other32(float x, float &same)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    same = __builtin_bit_cast(float, (uint32_t)r[0]);
    return __builtin_bit_cast(float, (uint32_t)r[1]);
}
__device__ __forceinline__ float max32(float x)
{
    float a;
    const float b = other32(x, a);
    return fmaxf(a, b);
}
__device__ __forceinline__ float sum32(float x)
{
    float a;
    const float b = other32(x, a);
    return a + b;
}
// Maximum / sum over the four lanes that share lane % 16.
__device__ __forceinline__ float max_quads(float x)
{
    float a;
    const float b = other16(x, a);
    return max32(fmaxf(a, b));
}
__device__ __forceinline__ float sum_quads(float x)
{
    float a;
    const float b = other16(x, a);
    return sum32(a + b);
}

// Buffer cache policy that bypasses the XCD-local L2 (device scope), for
// data that workgroups on different XCDs exchange inside one launch.
constexpr int kDeviceScope = 16;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// The stride of a dimension, nothing where it has one entry: views carry any
// number there.
inline int64_t stride_of(int64_t stride, int64_t count) { return count == 1 ? 0 : stride; }

// Whether rows of `width` elements, counts[i] of them strides[i] apart, lie
// apart from one another: every dimension steps over all that the closer ones span.
template <int N>
bool rows_apart(int64_t width, std::array<int64_t, N> strides, std::array<int64_t, N> counts)
{
    int64_t span = width;
    bool done[N] = {};
    for (int k = 0; k < N; ++k) {
        int next = -1;
        for (int i = 0; i < N; ++i)
            if (!done[i] && (next < 0 || strides[i] < strides[next]))
                next = i;
        done[next] = true;
        if (counts[next] <= 1)
            continue;
        if (strides[next] < span)
            return false;
        span += strides[next] * (counts[next] - 1);
    }
    return true;
}

inline bool aligned_to(const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

}  // namespace gdp
