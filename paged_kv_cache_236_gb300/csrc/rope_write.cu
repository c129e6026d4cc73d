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
// frequency in turns per position, rounded to a multiple of 2^-64 (a few fp64
// operations per frequency and block), times the position modulo 2^64 is the
// fraction of a turn exactly but for p * 2^-53 relative of the frequency's own
// rounding.  sincospif of its signed value is then good to fp32.  All of a
// token's heads share its rotary/2 (cos, sin) pairs, in shared memory.
//
// HBM-bound: q, k and v are read once and q_out and the pool rows written
// once; a separate rotation would move q and k twice.  A thread holds kVec
// pairs (two 16-byte vectors of one head), two heads' worth in flight.
// Values are rotated in fp32 and rounded once, to the output's type: an FP8
// pool takes the code of the fp32 value, with no rounding to the row's type
// in between.
#include <cuda_fp8.h>
#include <math.h>

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
  int interleaved, tokens_per_cta;
  float amp, k_scale, v_scale;
  int* err;
};

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;  // tokens of a CTA

template <typename U, int N>
struct alignas(sizeof(U) * N) Vec {
  U e[N];
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ void from_f(float x, float& y) { y = x; }
__device__ __forceinline__ void from_f(float x, uint16_t& y) { y = __bfloat16_as_ushort(__float2bfloat16_rn(x)); }

// E4M3 code of x / scale (IEEE division, nearest even, saturating), as
// paged_kv_write_fp8 encodes.
__device__ __forceinline__ uint8_t code_of(float x, float scale) {
  return (uint8_t)__nv_cvt_float_to_fp8(__fdiv_rn(x, scale), __NV_SATFINITE, __NV_E4M3);
}

// One head row's unit x of a token: VEC pairs (the first half / VEC units) or
// VEC copied elements.
template <typename U, int VEC>
struct Unit {
  Vec<U, VEC> a, b;
};

// F8: the pools hold E4M3 codes.  U: the rows' element (uint16_t: bf16 bits).
template <typename U, int VEC, bool F8>
__global__ void __launch_bounds__(kThreads) rope_write_kernel(const RopeParams p) {
  pdl_launch_dependents();  // what follows with programmatic launch reads nothing written here before it waits
  extern __shared__ float2 trig[];  // [tokens][half]
  const int64_t t0 = (int64_t)blockIdx.x * p.tokens_per_cta;
  const int nt = (int)min((int64_t)p.tokens_per_cta, p.T - t0);
  for (int i = threadIdx.y * blockDim.x + threadIdx.x; i < nt * p.half; i += blockDim.x * blockDim.y) {
    const int t = i / p.half, j = i - t * p.half;
    const double turns = p.inv_freq[j] * 0.15915494309189535;  // 1 / (2 pi)
    const long long fix = __double2ll_rn((turns - rint(turns)) * 18446744073709551616.0);
    const long long ang = (long long)((unsigned long long)p.positions[t0 + t] * (unsigned long long)fix);
    float s, c;
    sincospif(__ll2float_rn(ang) * 1.0842021724855044e-19f, &s, &c);  // 2^-63: half turns
    trig[i] = make_float2(c * p.amp, s * p.amp);
  }
  __syncthreads();

  const int heads = p.Hq + 2 * p.Hkv;
  const int rot_units = p.half / VEC;
  const int units = rot_units + (p.D - 2 * p.half) / VEC;  // of a rotated head
  const int vunits = p.D / VEC;
  const int rows = nt * heads;
  for (int r = blockIdx.y * blockDim.y + threadIdx.y; r < rows; r += gridDim.y * blockDim.y) {
    const int t = r / heads, h = r - t * heads;
    const int64_t tok = t0 + t;
    const bool is_q = h < p.Hq;
    int64_t slot = 0;
    if (!is_q) {
      slot = p.slots[tok];
      if (slot >= p.num_slots) {
        if (threadIdx.x == 0) raise_error(p.err, PKV_DEVERR_SLOT_OUT_OF_RANGE);
        slot = -1;
      }
      if (slot < 0) continue;
    }
    if (h >= p.Hq + p.Hkv) {  // v: copied, or encoded
      const int hv = h - p.Hq - p.Hkv;
      const U* src = static_cast<const U*>(p.v) + tok * p.v_stride + (int64_t)hv * p.D;
      const int64_t at = (slot * p.Hkv + hv) * p.D;
      for (int x = threadIdx.x; x < vunits; x += blockDim.x) {
        const Vec<U, VEC> a = *reinterpret_cast<const Vec<U, VEC>*>(src + x * VEC);
        if constexpr (F8) {
          Vec<uint8_t, VEC> o;
#pragma unroll
          for (int i = 0; i < VEC; ++i) o.e[i] = code_of(to_f(a.e[i]), p.v_scale);
          *reinterpret_cast<Vec<uint8_t, VEC>*>(static_cast<uint8_t*>(p.vc) + at + x * VEC) = o;
        } else {
          *reinterpret_cast<Vec<U, VEC>*>(static_cast<U*>(p.vc) + at + x * VEC) = a;
        }
      }
      continue;
    }
    const int hk = h - p.Hq;
    const U* src = is_q ? static_cast<const U*>(p.q) + tok * p.q_stride + (int64_t)h * p.D
                        : static_cast<const U*>(p.k) + tok * p.k_stride + (int64_t)hk * p.D;
    const int64_t at = is_q ? (tok * p.Hq + h) * (int64_t)p.D : (slot * p.Hkv + hk) * (int64_t)p.D;
    U* dst = is_q ? static_cast<U*>(p.q_out) : static_cast<U*>(p.kc);
    auto put = [&](int col, const float (&y)[VEC]) {
      if (F8 && !is_q) {
        Vec<uint8_t, VEC> o;
#pragma unroll
        for (int i = 0; i < VEC; ++i) o.e[i] = code_of(y[i], p.k_scale);
        *reinterpret_cast<Vec<uint8_t, VEC>*>(static_cast<uint8_t*>(p.kc) + at + col) = o;
      } else {
        Vec<U, VEC> o;
#pragma unroll
        for (int i = 0; i < VEC; ++i) from_f(y[i], o.e[i]);
        *reinterpret_cast<Vec<U, VEC>*>(dst + at + col) = o;
      }
    };
    for (int x = threadIdx.x; x < units; x += blockDim.x) {
      if (x >= rot_units) {  // past the rotary part
        const int col = 2 * p.half + (x - rot_units) * VEC;
        const Vec<U, VEC> a = *reinterpret_cast<const Vec<U, VEC>*>(src + col);
        float y[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) y[i] = to_f(a.e[i]);
        put(col, y);
        continue;
      }
      const int ca = p.interleaved ? 2 * x * VEC : x * VEC;
      const int cb = p.interleaved ? ca + VEC : p.half + x * VEC;
      const Vec<U, VEC> a = *reinterpret_cast<const Vec<U, VEC>*>(src + ca);
      const Vec<U, VEC> b = *reinterpret_cast<const Vec<U, VEC>*>(src + cb);
      const float2* cs = trig + t * p.half + x * VEC;
      float ya[VEC], yb[VEC];
      if (p.interleaved) {
        // the 2 * VEC elements a, b hold pairs (0, 1), (2, 3), ...
        float in[2 * VEC], out[2 * VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          in[i] = to_f(a.e[i]);
          in[VEC + i] = to_f(b.e[i]);
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          out[2 * i] = fmaf(in[2 * i], cs[i].x, -in[2 * i + 1] * cs[i].y);
          out[2 * i + 1] = fmaf(in[2 * i + 1], cs[i].x, in[2 * i] * cs[i].y);
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          ya[i] = out[i];
          yb[i] = out[VEC + i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float x1 = to_f(a.e[i]), x2 = to_f(b.e[i]);
          ya[i] = fmaf(x1, cs[i].x, -x2 * cs[i].y);
          yb[i] = fmaf(x2, cs[i].x, x1 * cs[i].y);
        }
      }
      put(ca, ya);
      put(cb, yb);
    }
  }
}

pkv_status fail(pkv_status st, const char* msg) {
  set_last_error(msg);
  return st;
}

template <typename U, bool F8>
cudaError_t launch(const RopeParams& p0, bool vec, int sms, cudaStream_t s) {
  RopeParams p = p0;
  constexpr int kV = 16 / sizeof(U);
  const int V = vec ? kV : 1;
  const int units = p.half / V + (p.D - 2 * p.half) / V;
  dim3 block((unsigned)(units < kThreads ? units : kThreads), 1, 1);
  block.y = kThreads / block.x;
  // one token a CTA until there are a few waves of them
  int64_t per = p.T / ((int64_t)sms * 16);
  per = per < 1 ? 1 : per > kMaxTokens ? kMaxTokens : per;
  p.tokens_per_cta = (int)per;
  const int64_t ctas = (p.T + per - 1) / per;
  const int heads = p.Hq + 2 * p.Hkv;
  // few tokens: a token's heads are spread over several CTAs
  int split = 1;
  while (ctas * split < sms && split * (int)block.y < heads) split *= 2;
  dim3 grid((unsigned)ctas, (unsigned)split, 1);
  const size_t smem = (size_t)per * p.half * sizeof(float2);
  if (vec)
    rope_write_kernel<U, kV, F8><<<grid, block, smem, s>>>(p);
  else
    rope_write_kernel<U, 1, F8><<<grid, block, smem, s>>>(p);
  return cudaGetLastError();
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
