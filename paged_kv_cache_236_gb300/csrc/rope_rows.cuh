// What the kernels that rotate rows share: vectors of row elements, stores of
// rows and of E4M3 codes, and the angle of a position as a fraction of a turn.
#pragma once

#include <cuda_fp8.h>
#include <math.h>

#include "pkv_device.cuh"

namespace pkv {

typedef unsigned __int128 u128;

template <typename U, int N>
struct alignas(sizeof(U) * N) Vec {
  U e[N];
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ void from_f(float x, float& y) { y = x; }
__device__ __forceinline__ void from_f(float x, uint16_t& y) { y = __bfloat16_as_ushort(__float2bfloat16_rn(x)); }

// A pool's scale and two floats with lo <= 1 / value <= hi, next to each other
// or the same (powers of two); 0 and infinity where they would not be normal.
struct CodeScale {
  float value, lo, hi;
};
inline CodeScale code_scale(float s) {  // s positive and finite
  if (!(s >= 0x1p-120f && s <= 0x1p120f)) return {s, 0.f, INFINITY};
  float lo = (float)(1.0 / (double)s), hi = lo;
  // (the products are exact in double)
  while ((double)lo * (double)s > 1.0) lo = nextafterf(lo, 0.f);
  while ((double)hi * (double)s < 1.0) hi = nextafterf(hi, INFINITY);
  return {s, lo, hi};
}

// E4M3 codes of x / scale (IEEE division, nearest even, saturating), as
// paged_kv_write_fp8 encodes.  Rounding is monotone, so that x / scale, and its
// code, lies between those of x lo and x hi: where the two codes are one, it is the
// code, and only else (one value in 10^5 or so) is anything divided.  With a division
// to each value, and its branches, 16384 tokens took rope_write.cu 82 us, so 72, and
// norm_rope.cu 85, so 74.3.
template <int N>
__device__ __forceinline__ void store_codes(uint8_t* dst, const float (&x)[N], const CodeScale& s) {
  Vec<uint8_t, N> o;
  if constexpr (N >= 2) {
    uint32_t differ = 0;
    const f32x2 lo = pk2(s.lo, s.lo), hi = pk2(s.hi, s.hi);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const f32x2 v = pk2(x[i], x[i + 1]);
      const uint32_t a = __nv_cvt_float2_to_fp8x2(up2(mul2(v, lo)), __NV_SATFINITE, __NV_E4M3);
      differ |= a ^ __nv_cvt_float2_to_fp8x2(up2(mul2(v, hi)), __NV_SATFINITE, __NV_E4M3);
      o.e[i] = (uint8_t)a;
      o.e[i + 1] = (uint8_t)(a >> 8);
    }
    if (differ) {
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const uint32_t a = __nv_cvt_float2_to_fp8x2(
            make_float2(__fdiv_rn(x[i], s.value), __fdiv_rn(x[i + 1], s.value)), __NV_SATFINITE, __NV_E4M3);
        o.e[i] = (uint8_t)a;
        o.e[i + 1] = (uint8_t)(a >> 8);
      }
    }
  } else {
    o.e[0] = (uint8_t)__nv_cvt_float_to_fp8(__fdiv_rn(x[0], s.value), __NV_SATFINITE, __NV_E4M3);
  }
  *reinterpret_cast<Vec<uint8_t, N>*>(dst) = o;
}
template <typename U, int N>
__device__ __forceinline__ void store_rows(U* dst, const float (&x)[N]) {
  Vec<U, N> o;
#pragma unroll
  for (int i = 0; i < N; ++i) from_f(x[i], o.e[i]);
  *reinterpret_cast<Vec<U, N>*>(dst) = o;
}

// The fraction of a turn, times 2^64, at a position, of a frequency in radians
// per position: |f| = m * 2^(e - 52) with a whole m < 2^53, and 1 / (2 pi) as a
// whole number of 2^-64 or 2^-128.
constexpr uint64_t kInv2Pi = 0x28BE60DB9391054Aull, kInv2PiLow = 0x7F09D5F47D4D3770ull;

// Any position and frequency: turns of 2^-128, the top half of the product's 128
// bits, a position's sign in its weight of 2^64.
static __device__ __noinline__ int64_t far_angle(int64_t pos, double f) {
  const uint64_t bits = (uint64_t)__double_as_longlong(f);
  const int e = (int)((bits >> 52) & 2047) - 1023;
  const uint64_t m = (bits & 0xFFFFFFFFFFFFFull) | (e == -1023 ? 0 : 1ull << 52);
  const int sh = 52 - (e == -1023 ? -1022 : e);  // m * 2^128 / (2 pi) >> sh
  const u128 low = (u128)m * kInv2PiLow, high = (u128)m * kInv2Pi + (uint64_t)(low >> 64);  // high * 2^64 + low's low half
  u128 r;
  if (sh >= 192) r = 0;
  else if (sh >= 64) r = high >> (sh - 64);
  else if (sh >= 0) r = (high << (64 - sh)) | (uint64_t)low >> sh;
  else r = sh > -128 ? ((high << 64) | (uint64_t)low) << -sh : 0;
  if (bits >> 63) r = 0 - r;
  const uint64_t part = (uint64_t)r, p = (uint64_t)pos;
  return (int64_t)(p * (uint64_t)(r >> 64) + __umul64hi(p, part) - (pos < 0 ? part : 0));
}

// Positions of 32 bits and frequencies below 2: a frequency in turns of 2^-64 is
// off by at most 3 of them, the angle by less than 2^-31 of a turn.  (The others' way for
// all: 3 % of a mixed step's time.)
__device__ __forceinline__ int64_t angle_of(int64_t pos, double f) {
  const uint64_t bits = (uint64_t)__double_as_longlong(f);
  const int e = (int)((bits >> 52) & 2047) - 1023;
  if (pos != (int)pos || e > 0) return far_angle(pos, f);
  const uint64_t m = (bits & 0xFFFFFFFFFFFFFull) | (e == -1023 ? 0 : 1ull << 52);
  const uint64_t lo = m * kInv2Pi, hi = __umul64hi(m, kInv2Pi);
  const int sh = 52 - (e == -1023 ? -1022 : e);  // m * 2^64 / (2 pi) >> sh
  const uint64_t r = sh >= 128 ? 0 : sh >= 64 ? hi >> (sh - 64) : (lo >> sh) | (hi << (64 - sh));
  return pos * (int64_t)(bits >> 63 ? 0 - r : r);
}

// cos and sin (times amp) of an angle that angle_of gave
__device__ __forceinline__ float2 turn_of(int64_t angle, float amp) {
  float s, c;
  sincospif(__ll2float_rn(angle) * 1.0842021724855044e-19f, &s, &c);  // 2^-63: half turns
  return make_float2(c * amp, s * amp);
}

}  // namespace pkv
