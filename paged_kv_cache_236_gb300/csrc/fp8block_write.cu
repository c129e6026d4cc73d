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
// HBM-bound for prompts (rows in once, codes out once); a decode step is a launch
// and four dependent reads (slot, old scale, rows, codes of a block that grows).
#include <cuda_fp8.h>
#include <math.h>

#include <algorithm>

#include "paged_kv_fp8block.h"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kScanTokens = 512;
constexpr int kMaxWarps = 16;
constexpr int kGroup = 16;  // tokens of a CTA past kScanTokens
constexpr int kMaxBlock = 64;
constexpr int kHold = 16;   // 4-element pieces of a block's rows that a lane keeps in registers

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
  int bs, Hkv, D;
  int* err;
};

// token_of[slot] = token
__global__ void __launch_bounds__(256) slot_table_kernel(const WriteParams p) {
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (t >= p.T) return;
  const int64_t s = p.slots[t];
  if (s >= p.num_slots) raise_error(p.err, PKV_DEVERR_SLOT_OUT_OF_RANGE);
  if (s >= 0 && s < p.num_slots) p.token_of[s] = (int)t;
}

template <typename U>
struct Raw4;  // four row elements as they are loaded
template <>
struct Raw4<uint16_t> {
  uint2 w;
  __device__ __forceinline__ void load(const uint16_t* p, bool vec) {
    if (vec) {
      w = *reinterpret_cast<const uint2*>(p);
    } else {
      w.x = p[0] | (uint32_t)p[1] << 16;
      w.y = p[2] | (uint32_t)p[3] << 16;
    }
  }
  __device__ __forceinline__ float4 get() const {
    return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
  }
};
template <>
struct Raw4<float> {
  float4 w;
  __device__ __forceinline__ void load(const float* p, bool vec) {
    if (vec)
      w = *reinterpret_cast<const float4*>(p);
    else
      w = make_float4(p[0], p[1], p[2], p[3]);
  }
  __device__ __forceinline__ float4 get() const { return w; }
};

__device__ __forceinline__ uint32_t codes4(float4 x) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x.x, x.y), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x.z, x.w), __NV_SATFINITE, __NV_E4M3);
  return (lo & 0xFFFFu) | hi << 16;
}
__device__ __forceinline__ float4 values4(uint32_t c) {
  const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c & 0xFFFFu), __NV_E4M3);
  const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c >> 16), __NV_E4M3);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return make_float4(a.x, a.y, b.x, b.y);
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
// offset o, or -1; n_rows of them, their offsets in row_at.
template <typename U>
__device__ __forceinline__ void write_unit(const WriteParams& p, int64_t block, const int* members, const uint8_t* row_at,
                                           int n_rows, int h, bool is_v, bool vec, int lane) {
  const U* src = static_cast<const U*>(is_v ? p.v : p.k) + (int64_t)h * p.D;
  const int64_t stride = is_v ? p.v_stride : p.k_stride;
  uint8_t* pool = (is_v ? p.vc : p.kc) + (block * p.bs * p.Hkv + h) * p.D;  // offset o at o * Hkv * D
  const int64_t pitch = (int64_t)p.Hkv * p.D;
  float* scale_at = (is_v ? p.vs : p.ks) + block * p.Hkv + h;
  const bool begins = members[0] >= 0;
  const float held = begins ? 0.f : *scale_at;
  const int pieces = p.D / 4, total = n_rows * pieces;
  // piece i of the rows: row i / pieces, elements 4 (i % pieces) ..
  auto at = [&](int i, int& off, int& c) {
    const int r = i / pieces;
    c = 4 * (i - r * pieces);
    off = row_at[r];
  };
  auto top_of = [](float4 x) { return fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w))); };
  Raw4<U> raw[kHold];
#pragma unroll
  for (int j = 0; j < kHold; ++j) {
    const int i = lane + 32 * j;
    if (i < total) {
      int off, c;
      at(i, off, c);
      raw[j].load(src + members[off] * stride + c, vec);
    }
  }
  float top = 0.f;  // (a NaN is left out)
#pragma unroll
  for (int j = 0; j < kHold; ++j)
    if (lane + 32 * j < total) top = fmaxf(top, top_of(raw[j].get()));
  for (int i = lane + 32 * kHold; i < total; i += 32) {
    int off, c;
    at(i, off, c);
    Raw4<U> x;
    x.load(src + members[off] * stride + c, vec);
    top = fmaxf(top, top_of(x.get()));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float need = pow2(need_exponent(top));
  const float old = held > 0.f ? held : 0.f;  // (a NaN is none)
  const float now = fmaxf(old, need), inv = 1.f / now;
  if (!begins && now > old) {
    // the codes that stay, at the new scale
    const float ratio = old * inv;
    const int all = p.bs * pieces;
    for (int i0 = lane; i0 < all; i0 += 32 * 8) {
      uint32_t codes[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = i0 + 32 * j, o = i / pieces;
        if (i < all && members[o] < 0) codes[j] = *reinterpret_cast<const uint32_t*>(pool + o * pitch + 4 * (i - o * pieces));
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = i0 + 32 * j, o = i / pieces;
        if (i < all && members[o] < 0) {
          float4 x = values4(codes[j]);
          x = make_float4(x.x * ratio, x.y * ratio, x.z * ratio, x.w * ratio);
          *reinterpret_cast<uint32_t*>(pool + o * pitch + 4 * (i - o * pieces)) = codes4(x);
        }
      }
    }
  }
  auto put = [&](int i, float4 x) {
    int off, c;
    at(i, off, c);
    *reinterpret_cast<uint32_t*>(pool + off * pitch + c) = codes4(make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv));
  };
#pragma unroll
  for (int j = 0; j < kHold; ++j)
    if (lane + 32 * j < total) put(lane + 32 * j, raw[j].get());
  for (int i = lane + 32 * kHold; i < total; i += 32) {
    int off, c;
    at(i, off, c);
    Raw4<U> x;
    x.load(src + members[off] * stride + c, vec);
    put(i, x.get());
  }
  if (lane == 0 && now != held) *scale_at = now;
}

template <typename U>
__global__ void __launch_bounds__(kMaxWarps * 32) write_blocks_kernel(const WriteParams p, int vec) {
  // a CTA's blocks (those led by its tokens): the tokens by offset, the offsets written
  __shared__ int members[kGroup][kMaxBlock];
  __shared__ uint8_t row_at[kGroup][kMaxBlock];
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
    const int64_t b = s / p.bs;
    for (int o = threadIdx.x; o < p.bs; o += blockDim.x) members[0][o] = -1;
    __syncthreads();
    for (int t = threadIdx.x; t < p.T; t += blockDim.x) {
      const int64_t o = p.slots[t] - b * p.bs;
      if (o >= 0 && o < p.bs) atomicMax(&members[0][o], t);
    }
    if (threadIdx.x == 0) block_of[0] = b;
    __syncthreads();
  }
  // each token's block, if the token leads it: by a warp
  for (int g = warp; g < per; g += warps) {
    const int64_t t = t0 + g;
    int count = 0;
    const int64_t s = t < p.T ? p.slots[t] : -1;
    if (s >= 0 && s < p.num_slots) {
      const int64_t b = s / p.bs;
      const int mine = (int)(s - b * p.bs);
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
            if (who[j] >= 0) row_at[g][__popcll(m & ((1ull << o) - 1))] = (uint8_t)o;
          }
        }
        if (lane == 0) block_of[g] = b;
      }
    }
    if (lane == 0) n_rows[g] = count;
  }
  __syncthreads();
  const int units = 2 * p.Hkv;
  for (int g = 0; g < per; ++g) {
    if (n_rows[g] == 0) continue;
    for (int u = warp + blockIdx.y * warps; u < units; u += warps * gridDim.y)
      write_unit<U>(p, block_of[g], members[g], row_at[g], n_rows[g], u >> 1, u & 1, vec, lane);
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
  p.Hkv = num_kv_heads;
  p.D = head_dim;
  // four elements at a time where every row start allows it
  const int vec = k_token_stride % 4 == 0 && v_token_stride % 4 == 0 && ((bits(k) | bits(v)) & (4 * es - 1)) == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p.token_of) {
    slot_table_kernel<<<(unsigned)((p.T + 255) / 256), 256, 0, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_error(e, "paged_kv_write_fp8block launch");
  }
  const int per = p.token_of ? kGroup : 1;
  const int warps = std::min(2 * p.Hkv, kMaxWarps);
  // more heads than a CTA has warps for: several CTAs to a block
  const dim3 grid((unsigned)((p.T + per - 1) / per), (unsigned)std::min((2 * p.Hkv + warps - 1) / warps, 1024));
  if (es == 2)
    write_blocks_kernel<uint16_t><<<grid, warps * 32, 0, s>>>(p, vec);
  else
    write_blocks_kernel<float><<<grid, warps * 32, 0, s>>>(p, vec);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_error(e, "paged_kv_write_fp8block launch");
  return PKV_OK;
}

}  // extern "C"
