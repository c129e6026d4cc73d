// The write into pools of E4M3 codes with a scale for each block and kv head
// (paged_kv_write_fp8block, declared in paged_kv_fp8block.h).
//
// For the rows x that a call brings to block b, head h, K and V apart:
//   need = 2^E, the least with max|x| <= 448 2^E;  new = max(old, need)
//   code = E4M3(x / new);  earlier codes c, where new > old: E4M3(c old / new)
// with old = 0 where the call writes the block's first slot.  Scales are powers
// of two: the division only moves the exponent, and so does a block's growth.
//
// All of a block's rows meet in one CTA (its leader token's: the one at the
// block's lowest offset in this call), so a maximum needs no second launch and
// no atomics on the scales.  Who else writes the block is found
//   - up to kScanTokens tokens: by going over all slots in every CTA (a decode
//     step is one launch);
//   - past that: through a table slot -> token in the workspace that a first
//     launch fills.  Its other entries are whatever was there: an entry counts
//     only if the token that it names has that slot.
// A warp takes one (head, K or V) of the block: the rows' loads are all in
// flight before the maximum, the rows stay in registers until they are encoded.
//
// HBM-bound for prompts (rows in once, codes out once): 16384 tokens of 8 heads of
// 128 in bf16 25.4 us, of which the table's launch (4 us) and the leaders' three
// dependent reads are a third; its instructions (49 % of the issue slots) come next,
// so that a lane keeps its column and maxima are taken two at a time.  A
// decode step is a launch and four dependent reads (slot, old scale, rows, codes of a
// block that grows): 12.3 us with the call.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <math.h>

#include <algorithm>

#include "paged_kv_fp8block.h"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kScanTokens = 512;
// (16384 tokens: 8 warps with 8 tokens 25.9 us, with 16 27.2, with 32 33; 16 warps
// 33.4, which leaves a thread too few registers, 4 warps 28.8)
constexpr int kMaxWarps = 8;
constexpr int kGroup = 8;  // tokens of a CTA past kScanTokens
constexpr int kMaxBlock = 64;
constexpr int kHold = 8;    // 8-element pieces of a block's rows that a lane keeps in registers

struct WriteParams {
  const void* k;
  const void* v;
  const int64_t* slots;
  uint8_t* kc;
  uint8_t* vc;
  float* ks;
  float* vs;
  int* token_of;  // [num_slots], or NULL: scan
  int64_t T, num_slots, k_stride, v_stride;  // strides in elements
  int bs, log_bs, Hkv, D;
  int* err;
};

// token_of[slot] = token
__global__ void __launch_bounds__(256) slot_table_kernel(const WriteParams p) {
  pdl_launch_dependents();  // the rows' kernel, which waits before it reads the table or writes
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (t >= p.T) return;
  const int64_t s = p.slots[t];
  if (s >= p.num_slots) raise_error(p.err, PKV_DEVERR_SLOT_OUT_OF_RANGE);
  if (s >= 0 && s < p.num_slots) p.token_of[s] = (int)t;
}

template <typename U>
struct Raw8;  // eight row elements as they are loaded
template <>
struct Raw8<uint16_t> {
  uint4 w;
  __device__ __forceinline__ void load(const uint16_t* p, bool vec) {
    if (vec) {
      w = *reinterpret_cast<const uint4*>(p);
    } else {
      w = make_uint4(p[0] | (uint32_t)p[1] << 16, p[2] | (uint32_t)p[3] << 16, p[4] | (uint32_t)p[5] << 16,
                     p[6] | (uint32_t)p[7] << 16);
    }
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf16_lo(in[i]);
      x[2 * i + 1] = bf16_hi(in[i]);
    }
  }
  // the largest |x|, a NaN left out: two at a time
  struct Top {
    __nv_bfloat162 m = __floats2bfloat162_rn(0.f, 0.f);
    __device__ __forceinline__ void add(const Raw8& r) {
      const uint32_t in[4] = {r.w.x, r.w.y, r.w.z, r.w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) m = __hmax2(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&in[i])));
    }
    __device__ __forceinline__ float value() const { return fmaxf(__low2float(m), __high2float(m)); }
  };
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p, bool vec) {
    if (vec) {
      a = *reinterpret_cast<const float4*>(p);
      b = *reinterpret_cast<const float4*>(p + 4);
    } else {
      a = make_float4(p[0], p[1], p[2], p[3]);
      b = make_float4(p[4], p[5], p[6], p[7]);
    }
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  struct Top {
    float m = 0.f;
    __device__ __forceinline__ void add(const Raw8& r) {
      float x[8];
      r.get(x);
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x[e]));
    }
    __device__ __forceinline__ float value() const { return m; }
  };
};

// Codes of eight values times `by`, and the values of eight codes.
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float by) {
  uint32_t c[4];
  const f32x2 by2 = pk2(by, by);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = __nv_cvt_float2_to_fp8x2(up2(mul2(pk2(x[2 * i], x[2 * i + 1]), by2)), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[2], c[3], 0x5410));
}
__device__ __forceinline__ void values8(uint2 c, float (&x)[8]) {
  const uint32_t in[2] = {c.x, c.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t h = e4m3x2_to_f16x2(in[i >> 1] >> (16 * (i & 1)) & 0xFFFFu);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

// Exponent of the least power of two whose 448-fold (1.75 * 2^8) reaches top
// (finite or not, >= 0), within [-60, 60].
__device__ __forceinline__ int need_exponent(float top) {
  const uint32_t b = __float_as_uint(top);
  const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(e, -60), 60);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// One (head, K or V) of a block, by a warp.  members[o]: the token that writes
// offset o, or -1; rows[r], r < n_rows: those tokens and their offsets.
// PIECES: 8-element pieces of a row (head_dim / 8) where that is 8 or 16 and
// rows allow 16-byte loads, so that a lane keeps its column; 0: any.
template <typename U, int PIECES>
__device__ __forceinline__ void write_unit(const WriteParams& p, int64_t block, const int* members, const int2* rows,
                                           int n_rows, int h, bool is_v, bool vec, int lane) {
  const U* src = static_cast<const U*>(is_v ? p.v : p.k) + (int64_t)h * p.D;
  const int64_t stride = is_v ? p.v_stride : p.k_stride;
  uint8_t* pool = (is_v ? p.vc : p.kc) + (block * p.bs * p.Hkv + h) * p.D;  // offset o at o * Hkv * D
  const int pitch = p.Hkv * p.D;  // at most 2^24, 64 rows of it
  float* scale_at = (is_v ? p.vs : p.ks) + block * p.Hkv + h;
  const bool begins = members[0] >= 0;
  const float held = begins ? 0.f : *scale_at;
  const int pieces = PIECES ? PIECES : p.D / 8;
  // the lane's j-th piece: of row row_of(j), elements col_of(j) ..
  constexpr int kStep = PIECES ? 32 / PIECES : 1;
  const int r0 = lane / pieces, c0 = 8 * (lane - r0 * pieces);
  auto row_of = [&](int j) { return PIECES ? r0 + kStep * j : (lane + 32 * j) / pieces; };
  auto col_of = [&](int j) { return PIECES ? c0 : 8 * (lane + 32 * j - row_of(j) * pieces); };
  auto load = [&](int j, Raw8<U>& x) { x.load(src + rows[row_of(j)].x * stride + col_of(j), PIECES || vec); };
  Raw8<U> raw[kHold];
#pragma unroll
  for (int j = 0; j < kHold; ++j)
    if (row_of(j) < n_rows) load(j, raw[j]);
  typename Raw8<U>::Top most;
#pragma unroll
  for (int j = 0; j < kHold; ++j)
    if (row_of(j) < n_rows) most.add(raw[j]);
#pragma unroll 1
  for (int j = kHold; row_of(j) < n_rows; ++j) {
    Raw8<U> x;
    load(j, x);
    most.add(x);
  }
  float top = most.value();
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float need = pow2(need_exponent(top));
  const float old = held > 0.f ? held : 0.f;  // (a NaN is none)
  const float now = fmaxf(old, need), inv = 1.f / now;
  auto put = [&](int j, const Raw8<U>& raw) {
    float x[8];
    raw.get(x);
    *reinterpret_cast<uint2*>(pool + rows[row_of(j)].y * pitch + col_of(j)) = codes8(x, inv);
  };
#pragma unroll
  for (int j = 0; j < kHold; ++j)
    if (row_of(j) < n_rows) put(j, raw[j]);
#pragma unroll 1
  for (int j = kHold; row_of(j) < n_rows; ++j) {
    Raw8<U> x;
    load(j, x);
    put(j, x);
  }
  if (!begins && now > old) {
    // the codes that stay, at the new scale
    const float ratio = old * inv;
    for (int i = 0; row_of(i) < p.bs; i += 4) {
      uint2 codes[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int o = row_of(i + j);
        if (o < p.bs && members[o] < 0) codes[j] = *reinterpret_cast<const uint2*>(pool + o * pitch + col_of(i + j));
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int o = row_of(i + j);
        if (o < p.bs && members[o] < 0) {
          float x[8];
          values8(codes[j], x);
          *reinterpret_cast<uint2*>(pool + o * pitch + col_of(i + j)) = codes8(x, ratio);
        }
      }
    }
  }
  if (lane == 0 && now != held) *scale_at = now;
}

// CTAs an SM: 16384 tokens in fp32 with one 56 us, two 35.9, three (registers spill) 53.
template <typename U, int PIECES>
__global__ void __launch_bounds__(kMaxWarps * 32, sizeof(U) == 2 && PIECES ? 3 : 2) write_blocks_kernel(const WriteParams p, int vec) {
  // a CTA's blocks (those led by its tokens): the tokens by offset; those there are, with their offsets
  __shared__ int members[kGroup][kMaxBlock];
  __shared__ int2 rows[kGroup][kMaxBlock];
  __shared__ int n_rows[kGroup];
  __shared__ int64_t block_of[kGroup];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int per = p.token_of ? kGroup : 1;
  const int64_t t0 = (int64_t)blockIdx.x * per;
  if (!p.token_of) {
    const int64_t s = p.slots[t0];
    if (s < 0 || s >= p.num_slots) {
      if (s >= 0 && threadIdx.x == 0) raise_error(p.err, PKV_DEVERR_SLOT_OUT_OF_RANGE);
      return;
    }
    const int64_t b = s >> p.log_bs;
    for (int o = threadIdx.x; o < p.bs; o += blockDim.x) members[0][o] = -1;
    __syncthreads();
    for (int t = threadIdx.x; t < p.T; t += blockDim.x) {
      const int64_t o = p.slots[t] - b * p.bs;
      if (o >= 0 && o < p.bs) atomicMax(&members[0][o], t);
    }
    if (threadIdx.x == 0) block_of[0] = b;
    __syncthreads();
  }
  // each token's block, if the token leads it: by a warp, with the rows of the
  // CTA's tokens on their way to L2 meanwhile (they are mostly its blocks')
  if (p.token_of) {
    const int lines = (p.Hkv * p.D * (int)sizeof(U) + 127) / 128;
    for (int i = threadIdx.x; i < kGroup * lines; i += blockDim.x) {
      const int64_t t = t0 + i / lines, at = (int64_t)(i % lines) * (128 / (int)sizeof(U));
      if (t < p.T) {
        asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const U*>(p.k) + t * p.k_stride + at));
        asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const U*>(p.v) + t * p.v_stride + at));
      }
    }
    pdl_wait();  // the slot table is complete
  }
  for (int g = warp; g < per; g += warps) {
    const int64_t t = t0 + g;
    int count = 0;
    const int64_t s = t < p.T ? p.slots[t] : -1;
    if (s >= 0 && s < p.num_slots) {
      const int64_t b = s >> p.log_bs;
      const int mine = (int)s & (p.bs - 1);
      int who[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int o = lane + 32 * j;
        who[j] = -1;
        if (o < p.bs) {
          if (!p.token_of) {
            who[j] = members[0][o];
          } else {
            const int c = p.token_of[b * p.bs + o];
            if (c >= 0 && c < p.T && p.slots[c] == b * p.bs + o) who[j] = c;
          }
        }
      }
      const uint32_t m0 = __ballot_sync(0xffffffffu, who[0] >= 0), m1 = __ballot_sync(0xffffffffu, who[1] >= 0);
      const uint64_t m = m0 | (uint64_t)m1 << 32;
      const int at_mine = __shfl_sync(0xffffffffu, mine < 32 ? who[0] : who[1], mine & 31);
      if (at_mine == t && (m & ((1ull << mine) - 1)) == 0) {
        count = __popcll(m);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int o = lane + 32 * j;
          if (o < p.bs) {
            members[g][o] = who[j];
            if (who[j] >= 0) rows[g][__popcll(m & ((1ull << o) - 1))] = make_int2(who[j], o);
          }
        }
        if (lane == 0) block_of[g] = b;
      }
    }
    if (lane == 0) n_rows[g] = count;
  }
  __syncthreads();
  const int units = 2 * p.Hkv;
  for (uint32_t led = __ballot_sync(0xffffffffu, lane < per && n_rows[lane] > 0); led != 0; led &= led - 1) {
    const int g = __ffs(led) - 1;
    for (int u = warp + blockIdx.y * warps; u < units; u += warps * gridDim.y)
      write_unit<U, PIECES>(p, block_of[g], members[g], rows[g], n_rows[g], u >> 1, u & 1, vec, lane);
  }
}

pkv_status fail(pkv_status st, const char* msg) {
  set_last_error(msg);
  return st;
}

}  // namespace
}  // namespace pkv

extern "C" {

size_t paged_kv_write_fp8block_workspace(int64_t num_tokens, int64_t num_blocks, int32_t block_size) {
  if (num_tokens <= pkv::kScanTokens || num_blocks <= 0 || block_size <= 0) return 0;
  return (size_t)num_blocks * block_size * sizeof(int);
}

pkv_status paged_kv_write_fp8block(const void* k, const void* v, const int64_t* slot_mapping, void* k_cache,
                                   void* v_cache, float* k_scales, float* v_scales, int64_t num_tokens,
                                   int64_t num_blocks, int32_t block_size, int32_t num_kv_heads, int32_t head_dim,
                                   int64_t k_token_stride, int64_t v_token_stride, void* workspace,
                                   size_t workspace_bytes, pkv_dtype dtype, void* stream) {
  using namespace pkv;
  set_last_error("");
  if (dtype != PKV_DTYPE_BF16 && dtype != PKV_DTYPE_F32) return fail(PKV_ERR_UNSUPPORTED, "dtype");
  if (num_tokens < 0 || num_blocks <= 0 || num_kv_heads <= 0 || head_dim <= 0)
    return fail(PKV_ERR_INVALID_ARG, "sizes must be positive (num_tokens >= 0)");
  if (block_size != 8 && block_size != 16 && block_size != 32 && block_size != 64)
    return fail(PKV_ERR_UNSUPPORTED, "block_size (supported: 8, 16, 32, 64)");
  if (head_dim % 16 != 0 || head_dim > 1024)
    return fail(PKV_ERR_UNSUPPORTED, "head_dim must be a multiple of 16, at most 1024");
  const int64_t row = (int64_t)num_kv_heads * head_dim;
  if (row > (1 << 24)) return fail(PKV_ERR_UNSUPPORTED, "num_kv_heads * head_dim too large");
  if (num_tokens > (int64_t)1 << 30) return fail(PKV_ERR_UNSUPPORTED, "num_tokens too large");
  if (num_blocks > ((int64_t)1 << 31) - 1) return fail(PKV_ERR_UNSUPPORTED, "num_blocks exceeds int32");
  if (k_token_stride == 0) k_token_stride = row;
  if (v_token_stride == 0) v_token_stride = row;
  if (k_token_stride < row || v_token_stride < row)
    return fail(PKV_ERR_INVALID_ARG, "token stride smaller than num_kv_heads * head_dim");
  if (num_tokens == 0) return PKV_OK;
  if (!k || !v || !slot_mapping || !k_cache || !v_cache || !k_scales || !v_scales)
    return fail(PKV_ERR_INVALID_ARG, "null pointer");
  auto bits = [](const void* x) { return reinterpret_cast<uintptr_t>(x); };
  const int es = dtype == PKV_DTYPE_BF16 ? 2 : 4;
  if ((bits(k_cache) | bits(v_cache)) & 15u) return fail(PKV_ERR_INVALID_ARG, "caches must be 16-byte aligned");
  if ((bits(k) | bits(v)) & (es - 1) || (bits(k_scales) | bits(v_scales)) & 3u || bits(slot_mapping) & 7u)
    return fail(PKV_ERR_INVALID_ARG, "a tensor is not aligned to its elements");
  const size_t want = paged_kv_write_fp8block_workspace(num_tokens, num_blocks, block_size);
  if (want > 0 && (!workspace || bits(workspace) & 15u || workspace_bytes < want))
    return fail(PKV_ERR_WORKSPACE, "workspace missing, too small or not 16-byte aligned");
  int sms = 0;
  WriteParams p{};
  pkv_status st = device_state(&sms, &p.err);
  if (st != PKV_OK) return st;
  p.k = k;
  p.v = v;
  p.slots = slot_mapping;
  p.kc = static_cast<uint8_t*>(k_cache);
  p.vc = static_cast<uint8_t*>(v_cache);
  p.ks = k_scales;
  p.vs = v_scales;
  p.token_of = want > 0 ? static_cast<int*>(workspace) : nullptr;
  p.T = num_tokens;
  p.num_slots = num_blocks * block_size;
  p.k_stride = k_token_stride;
  p.v_stride = v_token_stride;
  p.bs = block_size;
  p.log_bs = block_size == 8 ? 3 : block_size == 16 ? 4 : block_size == 32 ? 5 : 6;
  p.Hkv = num_kv_heads;
  p.D = head_dim;
  // 16 bytes at a time where every row start allows it
  const int vec = k_token_stride * es % 16 == 0 && v_token_stride * es % 16 == 0 && ((bits(k) | bits(v)) & 15u) == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p.token_of) {
    slot_table_kernel<<<(unsigned)((p.T + 255) / 256), 256, 0, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_error(e, "paged_kv_write_fp8block launch");
  }
  const int per = p.token_of ? kGroup : 1;
  const int warps = std::min(2 * p.Hkv, kMaxWarps);
  // more heads than a CTA has warps for: several CTAs to a block, while the SMs hold
  // them (16384 tokens with two in any case 31.5 us, with one 27.2)
  const int64_t groups = (p.T + per - 1) / per;
  const int64_t share = std::max<int64_t>(1, std::min<int64_t>((2 * p.Hkv + warps - 1) / warps, 3 * sms / groups));
  const dim3 grid((unsigned)groups, (unsigned)std::min<int64_t>(share, 1024));
  auto launch = [&](auto kernel) {
    return p.token_of ? launch_pdl(kernel, grid, dim3(warps * 32), 0, s, p, vec)
                      : (kernel<<<grid, warps * 32, 0, s>>>(p, vec), cudaGetLastError());
  };
  const int pieces = vec ? p.D / 8 : 0;
  cudaError_t e;
  if (es == 2)
    e = pieces == 16  ? launch(write_blocks_kernel<uint16_t, 16>)
        : pieces == 8  ? launch(write_blocks_kernel<uint16_t, 8>)
                       : launch(write_blocks_kernel<uint16_t, 0>);
  else
    e = pieces == 16  ? launch(write_blocks_kernel<float, 16>)
        : pieces == 8  ? launch(write_blocks_kernel<float, 8>)
                       : launch(write_blocks_kernel<float, 0>);
  if (e != cudaSuccess) return cuda_error(e, "paged_kv_write_fp8block launch");
  return PKV_OK;
}

}  // extern "C"
