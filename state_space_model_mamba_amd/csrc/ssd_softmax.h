// Softmax helpers shared by the kernels over packed prompts, padded caches and paged
// caches (ssd_attn.hip, ssd_paged.hip).
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "ssd_mma.h"

namespace ssd {
namespace mx {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.f;
constexpr float kNoMax = -3e38f;   // m before the first visible key (finite: m - m is 0)
// |scale| log2 e.  A scale of 0 weights all visible keys alike; it is kept off 0 so
// that a masked score (-inf) times it stays -inf, and finite so that a score of 0 times
// it stays 0.
inline float score_factor(float scale)
{
    return std::clamp(std::abs(scale) * kLog2e, 1.17549435e-38f, 3.40282347e38f);
}

// s c - m, the product rounded before the difference as it is in m: for the largest
// score of a row exactly 0 however large it is.  (Fused, the rounding of m remains;
// the row's weights have it in common, but past 2^30 it overflows the exponential.)
__device__ __forceinline__ float below_max(float s, float c, float m)
{
#pragma clang fp contract(off)
    return s * c - m;
}

// A piece of a query's row with the opposite sign.
template <typename T> __device__ __forceinline__ typename Piece<T>::V flip(typename Piece<T>::V v);
template <> __device__ __forceinline__ bf16x8 flip<__bf16>(bf16x8 v)
{
    u32x4 u = __builtin_bit_cast(u32x4, v);
    return __builtin_bit_cast(bf16x8, u ^ 0x80008000u);
}
template <> __device__ __forceinline__ f32x4 flip<float>(f32x4 v)
{
    return -v;
}

}  // namespace mx
}  // namespace ssd
