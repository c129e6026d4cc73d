// What the attention kernels over pools with block scales share: a block's
// scales as they are used, and the split of q's values into 8-bit terms.
#pragma once

#include "pkv_device.cuh"

namespace pkv {

// A block's scales: K's, log2 of V's, 2^-W / V's (weights are 2^W times their value).
struct alignas(16) Scales {
  float k, log_v, inv_v, pad;
};

// [2^-60, 2^60]; a NaN is the least
__device__ __forceinline__ float clamp_scale(float s) { return s >= 0x1p-60f ? fminf(s, 0x1p60f) : 0x1p-60f; }

template <int W>
__device__ __forceinline__ Scales make_scales(float2 kv) {
  Scales s;
  s.k = clamp_scale(kv.x);
  const float c = clamp_scale(kv.y);
  s.log_v = log2f(c);  // exact for powers of two
  s.inv_v = __fdiv_rn(1.f / (1 << W), c);
  s.pad = 0.f;
  return s;
}

// Two values as E4M3 terms hi + lo (pairs of codes, the low byte's first): what is
// left of a value by its first term is exact, and rounded to the second.
__device__ __forceinline__ void split_e4m3(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3) & 0xFFFFu;
  const uint32_t back = e4m3x2_to_f16x2(hi);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&back));
  lo = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a - f.x, b - f.y), __NV_SATFINITE, __NV_E4M3) & 0xFFFFu;
}

}  // namespace pkv
