// Rotary positions of a step's q and k, and the slot-mapping scatter of its
// K/V rows, in one pass (paged_kv_write_rope, paged_kv_write_rope_fp8).
//
// "ADR 004: Paged Attention Serving Integration", Decision 4: the model
// writes each layer's K/V into the block allocator; the rows it writes are
// the rotated ones.  For pair i of a head at position p, with the angle
// a = p * inv_freq[i]:
//   y1 = amp * (x1 cos a - x2 sin a),   y2 = amp * (x2 cos a + x1 sin a),
// the pair being elements (i, i + rotary/2) or, interleaved, (2i, 2i + 1);
// elements from rotary on are copied.
//
// The angle: a position of 2^17 and a frequency of 1 leave an fp32 product
// 2^-7 radians off, so the angle is kept in turns as a 64-bit fraction: the
// frequency in turns per position, a multiple of 2^-64 or, for far positions,
// 2^-128 (its 53-bit mantissa times 2^64 / (2 pi), shifted: integer arithmetic,
// the SM's fp64 units are few), times the position modulo 1.  sincospif of its
// signed value, rounded to fp32, is then good to fp32: that last rounding, 24
// bits over half a turn, makes the rotated value's error 5.5e-8 (RMS, relative)
// where exact angles would leave 3.7e-8, below what any 16-bit output shows.
//
// HBM-bound: q, k and v are read once and q_out and the pool rows written
// once; a separate rotation would move q and k twice.  A warp takes one token,
// or, with few tokens, some of its heads.  It computes the token's angles once
// (shared by its lanes through shared memory); then a lane owns one place of
// a head, two 16-byte vectors (kVec pairs of the rotary part, or two vectors
// past it), keeps that place's (cos, sin) in registers and goes through the
// heads, kBatch heads' loads in flight at a time.  The first version, a block
// of 256 threads to one or two tokens with the angles read from shared memory
// for every head, spent its time on instructions and the block's barrier
// (16384 tokens into FP8 pools: 168 us, 82 this way: 4.5 TB/s; 4216 tokens in
// bf16: 27 and 25 us).
// Values are rotated in fp32 and rounded once, to the output's type: an FP8
// pool takes the code of the fp32 value, with no rounding to the row's type
// in between.
#include <cuda_fp8.h>
#include <math.h>

#include <algorithm>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

struct RopeParams {
  const void* q;
  const void* k;
  const void* v;
  const int64_t* positions;
  const double* inv_freq;
  const int64_t* slots;
  void* q_out;
  void* kc;
  void* vc;
  int64_t T, num_slots, q_stride, k_stride, v_stride;  // strides in elements
  int Hq, Hkv, D, half;  // half: pairs per head (rotary / 2)
  int interleaved, splits;  // splits: warps that share a token's heads
  float amp, k_scale, v_scale;
  int* err;
};

constexpr int kWarps = 4;   // of a block
constexpr int kBatch = 2;   // heads a lane loads at a time

typedef unsigned __int128 u128;

template <typename U, int N>
struct alignas(sizeof(U) * N) Vec {
  U e[N];
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ void from_f(float x, float& y) { y = x; }
__device__ __forceinline__ void from_f(float x, uint16_t& y) { y = __bfloat16_as_ushort(__float2bfloat16_rn(x)); }

// E4M3 codes of x / scale (IEEE division, nearest even, saturating), as
// paged_kv_write_fp8 encodes.
template <int N>
__device__ __forceinline__ void store_codes(uint8_t* dst, const float (&x)[N], float scale) {
  Vec<uint8_t, N> o;
  if constexpr (N >= 2) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const uint32_t two = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(x[i], scale), __fdiv_rn(x[i + 1], scale)),
                                                    __NV_SATFINITE, __NV_E4M3);
      o.e[i] = (uint8_t)two;
      o.e[i + 1] = (uint8_t)(two >> 8);
    }
  } else {
    o.e[0] = (uint8_t)__nv_cvt_float_to_fp8(__fdiv_rn(x[0], scale), __NV_SATFINITE, __NV_E4M3);
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
__device__ __noinline__ int64_t far_angle(int64_t pos, double f) {
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

// F8: the pools hold E4M3 codes.  U: the rows' element (uint16_t: bf16 bits).
template <typename U, int VEC, bool F8, bool INTER>
__global__ void __launch_bounds__(kWarps * 32, 5) rope_write_kernel(const RopeParams p) {
  pdl_launch_dependents();  // what follows with programmatic launch reads nothing written here before it waits
  extern __shared__ float2 trig_all[];  // [warps][half]
  typedef Vec<U, VEC> V;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t w = (int64_t)blockIdx.x * kWarps + warp;
  const int64_t tok = w / p.splits;
  const int split = (int)(w - tok * p.splits);
  if (tok >= p.T) return;
  float2* trig = trig_all + warp * p.half;
  // this token's rows on their way to L2 while the angles are computed
  if (p.splits == 1) {
    auto fetch = [&](const void* rows, int64_t stride, int heads) {
      const char* at = static_cast<const char*>(rows) + tok * stride * (int64_t)sizeof(U);
      for (int i = lane * 128; i < heads * p.D * (int)sizeof(U); i += 32 * 128)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(at + i));
    };
    fetch(p.q, p.q_stride, p.Hq);
    fetch(p.k, p.k_stride, p.Hkv);
    fetch(p.v, p.v_stride, p.Hkv);
  }
  const int64_t pos = p.positions[tok];
  int64_t slot = p.slots[tok];
  if (slot >= p.num_slots) {
    if (lane == 0 && split == 0) raise_error(p.err, PKV_DEVERR_SLOT_OUT_OF_RANGE);
    slot = -1;
  }
  for (int j = lane; j < p.half; j += 32) {
    float s, c;
    sincospif(__ll2float_rn(angle_of(pos, p.inv_freq[j])) * 1.0842021724855044e-19f, &s, &c);  // 2^-63: half turns
    trig[j] = make_float2(c * p.amp, s * p.amp);
  }
  __syncwarp();

  const int places = (p.D / VEC + 1) / 2;  // of a head; the last may hold one vector
  const int rot_places = p.half / VEC;
  const int side = places < 32 ? 32 / places : 1;  // heads side by side
  const int y = places < 32 ? lane / places : 0;
  if (y >= side) return;
  const int hstep = side * p.splits;
  for (int x = places < 32 ? lane - y * places : lane; x < places; x += 32) {
    const bool rot = x < rot_places;
    // the place's two columns
    const int ca = rot ? (INTER ? 2 * x * VEC : x * VEC) : 2 * p.half + 2 * (x - rot_places) * VEC;
    const int cb = rot && !INTER ? p.half + x * VEC : ca + VEC;
    const bool two = cb + VEC <= p.D;
    float2 cs[VEC];
    if (rot) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) cs[e] = trig[x * VEC + e];
    }
    // this warp's heads of one of q, k, v (src: the token's head 0)
    auto go = [&](const U* src, int heads, auto put) {
      for (int h0 = split * side + y; h0 < heads; h0 += kBatch * hstep) {
        V a[kBatch], b[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int h = h0 + i * hstep;
          if (h < heads) {
            a[i] = *reinterpret_cast<const V*>(src + (int64_t)h * p.D + ca);
            if (two) b[i] = *reinterpret_cast<const V*>(src + (int64_t)h * p.D + cb);
          }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int h = h0 + i * hstep;
          if (h < heads) put(h, a[i], b[i]);
        }
      }
    };
    auto turned = [&](const V& a, const V& b, float (&ya)[VEC], float (&yb)[VEC]) {
      if (!rot) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          ya[e] = to_f(a.e[e]);
          yb[e] = two ? to_f(b.e[e]) : 0.f;
        }
      } else if (INTER) {
        // the 2 * VEC elements a, b hold pairs (0, 1), (2, 3), ...
        float in[2 * VEC], out[2 * VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          in[e] = to_f(a.e[e]);
          in[VEC + e] = to_f(b.e[e]);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          out[2 * e] = fmaf(in[2 * e], cs[e].x, -in[2 * e + 1] * cs[e].y);
          out[2 * e + 1] = fmaf(in[2 * e + 1], cs[e].x, in[2 * e] * cs[e].y);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          ya[e] = out[e];
          yb[e] = out[VEC + e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float x1 = to_f(a.e[e]), x2 = to_f(b.e[e]);
          ya[e] = fmaf(x1, cs[e].x, -x2 * cs[e].y);
          yb[e] = fmaf(x2, cs[e].x, x1 * cs[e].y);
        }
      }
    };
    U* qo = static_cast<U*>(p.q_out) + tok * p.Hq * (int64_t)p.D;
    go(static_cast<const U*>(p.q) + tok * p.q_stride, p.Hq, [&](int h, const V& a, const V& b) {
      float ya[VEC], yb[VEC];
      turned(a, b, ya, yb);
      U* dst = qo + (int64_t)h * p.D;
      store_rows<U, VEC>(dst + ca, ya);
      if (two) store_rows<U, VEC>(dst + cb, yb);
    });
    if (slot < 0) continue;
    const int64_t at = slot * p.Hkv * (int64_t)p.D;
    go(static_cast<const U*>(p.k) + tok * p.k_stride, p.Hkv, [&](int h, const V& a, const V& b) {
      float ya[VEC], yb[VEC];
      turned(a, b, ya, yb);
      const int64_t to = at + (int64_t)h * p.D;
      if constexpr (F8) {
        store_codes<VEC>(static_cast<uint8_t*>(p.kc) + to + ca, ya, p.k_scale);
        if (two) store_codes<VEC>(static_cast<uint8_t*>(p.kc) + to + cb, yb, p.k_scale);
      } else {
        store_rows<U, VEC>(static_cast<U*>(p.kc) + to + ca, ya);
        if (two) store_rows<U, VEC>(static_cast<U*>(p.kc) + to + cb, yb);
      }
    });
    go(static_cast<const U*>(p.v) + tok * p.v_stride, p.Hkv, [&](int h, const V& a, const V& b) {
      const int64_t to = at + (int64_t)h * p.D;
      if constexpr (F8) {
        float ya[VEC], yb[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          ya[e] = to_f(a.e[e]);
          yb[e] = two ? to_f(b.e[e]) : 0.f;
        }
        store_codes<VEC>(static_cast<uint8_t*>(p.vc) + to + ca, ya, p.v_scale);
        if (two) store_codes<VEC>(static_cast<uint8_t*>(p.vc) + to + cb, yb, p.v_scale);
      } else {
        *reinterpret_cast<V*>(static_cast<U*>(p.vc) + to + ca) = a;
        if (two) *reinterpret_cast<V*>(static_cast<U*>(p.vc) + to + cb) = b;
      }
    });
  }
}

pkv_status fail(pkv_status st, const char* msg) {
  set_last_error(msg);
  return st;
}

template <typename U, int VEC, bool F8>
cudaError_t launch_v(const RopeParams& p, dim3 grid, size_t smem, cudaStream_t s) {
  if (p.interleaved)
    rope_write_kernel<U, VEC, F8, true><<<grid, kWarps * 32, smem, s>>>(p);
  else
    rope_write_kernel<U, VEC, F8, false><<<grid, kWarps * 32, smem, s>>>(p);
  return cudaGetLastError();
}

template <typename U, bool F8>
cudaError_t launch(const RopeParams& p0, bool vec, int sms, cudaStream_t s) {
  RopeParams p = p0;
  constexpr int kV = 16 / sizeof(U);
  const int places = (p.D / (vec ? kV : 1) + 1) / 2, side = places < 32 ? 32 / places : 1;
  // few tokens: a token's heads are spread over several warps, down to one
  // load of each lane
  const int most = (std::max(p.Hq, p.Hkv) + side - 1) / side;
  p.splits = 1;
  while (p.T * p.splits < (int64_t)sms * 8 && p.splits < most) p.splits *= 2;
  const dim3 grid((unsigned)((p.T * p.splits + kWarps - 1) / kWarps));
  const size_t smem = (size_t)kWarps * p.half * sizeof(float2);
  return vec ? launch_v<U, kV, F8>(p, grid, smem, s) : launch_v<U, 1, F8>(p, grid, smem, s);
}

pkv_status rope_write(RopeParams p, int64_t num_blocks, int block_size, int rotary, pkv_dtype dtype, bool f8,
                      void* stream) {
  set_last_error("");
  if (dtype != PKV_DTYPE_BF16 && dtype != PKV_DTYPE_F32) return fail(PKV_ERR_UNSUPPORTED, "dtype");
  if (p.T < 0 || num_blocks <= 0 || block_size <= 0 || p.Hq <= 0 || p.Hkv <= 0 || p.D <= 0)
    return fail(PKV_ERR_INVALID_ARG, "sizes must be positive (num_tokens >= 0)");
  if (rotary <= 0 || rotary % 2 != 0 || rotary > p.D)
    return fail(PKV_ERR_INVALID_ARG, "rotary_dim must be even, positive and at most head_dim");
  if (p.D > 1024) return fail(PKV_ERR_UNSUPPORTED, "head_dim above 1024");
  const int64_t row_q = (int64_t)p.Hq * p.D, row = (int64_t)p.Hkv * p.D;
  if (row > (1 << 24) || row_q > (1 << 24)) return fail(PKV_ERR_UNSUPPORTED, "heads * head_dim too large");
  if (!(p.amp > 0.f) || !isfinite(p.amp)) return fail(PKV_ERR_INVALID_ARG, "amplitude must be positive and finite");
  if (f8 && (!(p.k_scale > 0.f) || !isfinite(p.k_scale) || !(p.v_scale > 0.f) || !isfinite(p.v_scale)))
    return fail(PKV_ERR_INVALID_ARG, "k_scale and v_scale must be positive and finite");
  if (p.q_stride == 0) p.q_stride = row_q;
  if (p.k_stride == 0) p.k_stride = row;
  if (p.v_stride == 0) p.v_stride = row;
  if (p.q_stride < row_q || p.k_stride < row || p.v_stride < row)
    return fail(PKV_ERR_INVALID_ARG, "token stride smaller than heads * head_dim");
  if (p.T > (int64_t)1 << 30) return fail(PKV_ERR_UNSUPPORTED, "num_tokens too large");
  if (p.T == 0) return PKV_OK;
  if (!p.q || !p.k || !p.v || !p.positions || !p.inv_freq || !p.slots || !p.q_out || !p.kc || !p.vc)
    return fail(PKV_ERR_INVALID_ARG, "null pointer");
  const size_t es = dtype == PKV_DTYPE_BF16 ? 2 : 4;
  auto bits = [](const void* x) { return reinterpret_cast<uintptr_t>(x); };
  if ((bits(p.kc) | bits(p.vc)) & 15u) return fail(PKV_ERR_INVALID_ARG, "caches must be 16-byte aligned");
  if ((bits(p.q) | bits(p.k) | bits(p.v) | bits(p.q_out)) & (es - 1) || (bits(p.positions) | bits(p.slots) | bits(p.inv_freq)) & 7u)
    return fail(PKV_ERR_INVALID_ARG, "a tensor is not aligned to its elements");
  int sms = 0;
  pkv_status st = device_state(&sms, &p.err);
  if (st != PKV_OK) return st;
  p.half = rotary / 2;
  p.num_slots = num_blocks * block_size;
  // 16-byte vectors where every row, every head and the rotary halves allow them
  const int V = (int)(16 / es);
  const bool vec = p.D % V == 0 && p.half % V == 0 && p.q_stride % V == 0 && p.k_stride % V == 0 &&
                   p.v_stride % V == 0 && ((bits(p.q) | bits(p.k) | bits(p.v) | bits(p.q_out)) & 15u) == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (es == 2)
    e = f8 ? launch<uint16_t, true>(p, vec, sms, s) : launch<uint16_t, false>(p, vec, sms, s);
  else
    e = f8 ? launch<float, true>(p, vec, sms, s) : launch<float, false>(p, vec, sms, s);
  if (e != cudaSuccess) return cuda_error(e, "paged_kv_write_rope launch");
  return PKV_OK;
}

}  // namespace
}  // namespace pkv

extern "C" {

pkv_status paged_kv_write_rope(const void* q, const void* k, const void* v, const int64_t* positions,
                               const double* inv_freq, const int64_t* slot_mapping, void* q_out, void* k_cache,
                               void* v_cache, int64_t num_tokens, int64_t num_blocks, int32_t block_size,
                               int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t rotary_dim,
                               int32_t interleaved, float amplitude, int64_t q_token_stride, int64_t k_token_stride,
                               int64_t v_token_stride, pkv_dtype dtype, void* stream) {
  pkv::RopeParams p{q, k, v, positions, inv_freq, slot_mapping, q_out, k_cache, v_cache, num_tokens, 0,
                    q_token_stride, k_token_stride, v_token_stride, num_q_heads, num_kv_heads, head_dim, 0,
                    interleaved ? 1 : 0, 0, amplitude, 1.f, 1.f, nullptr};
  return pkv::rope_write(p, num_blocks, block_size, rotary_dim, dtype, false, stream);
}

pkv_status paged_kv_write_rope_fp8(const void* q, const void* k, const void* v, const int64_t* positions,
                                   const double* inv_freq, const int64_t* slot_mapping, void* q_out, void* k_cache,
                                   void* v_cache, int64_t num_tokens, int64_t num_blocks, int32_t block_size,
                                   int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t rotary_dim,
                                   int32_t interleaved, float amplitude, int64_t q_token_stride,
                                   int64_t k_token_stride, int64_t v_token_stride, pkv_dtype dtype, float k_scale,
                                   float v_scale, void* stream) {
  pkv::RopeParams p{q, k, v, positions, inv_freq, slot_mapping, q_out, k_cache, v_cache, num_tokens, 0,
                    q_token_stride, k_token_stride, v_token_stride, num_q_heads, num_kv_heads, head_dim, 0,
                    interleaved ? 1 : 0, 0, amplitude, k_scale, v_scale, nullptr};
  return pkv::rope_write(p, num_blocks, block_size, rotary_dim, dtype, true, stream);
}

}  // extern "C"
