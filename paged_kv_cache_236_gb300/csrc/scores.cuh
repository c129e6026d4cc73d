// What the kernels of paged_attention_scores share: the plan of each
// sequence's work and the queues the kernels take it from.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math_constants.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

constexpr int kFewRows = 16;    // rows of a few-row sequence's kv head
constexpr int kFewChunk = 128;  // keys of a stats unit (few rows)
constexpr int kFewLeast = 32;   // of a short one
constexpr int kColChunk = 256;  // keys of a column unit (few rows)
constexpr int kTcRange = 1024;  // keys of an item of the tensor-core kernel
// Row tiles of a sequence the tensor-core kernel takes: a column item goes
// through all of them (8 key tiles each, below 1 us a tile), and the waits of
// the roles that stand by, up to two items long, end after 2 s.  (What one
// closing warp does before a column item is one row tile's, whatever the
// sequence: 4 rows a lane over at most 2^20 ranges of keys, some 0.5 s.)
constexpr int kMaxRowTiles = 1 << 16;
constexpr int kChunk = 256;   // keys of a work unit (more rows in fp32)
enum { kFew = 1, kTensor = 2, kOther = 3 };
constexpr int kColTile = 64;    // keys of its column unit
constexpr int kRowGroup = 32;   // its rows

// Offsets of each sequence's work, as prefix sums: the unit queues of the
// kernels below (few-row stats and columns; other rows' stats and columns),
// the tensor-core kernel's).
enum { kFewStat, kFewCol, kStat, kCol, kTcStat, kTcCol, kQueues };

struct SeqPlan {
  int64_t part, lse, logit;
  int L, n, row, chunks;
  int rows, pad;  // rows of a kv head; rows a key's logits are padded to (few rows)
  int kind;       // which kernels: kFew, kTensor, kOther (0: none)
  int tiles;      // row tiles of the tensor-core kernel (whole tokens that fit 128 rows)
  int chunk;      // keys of a chunk
};

struct ScoreParams {
  const void* q;
  const void* kc;
  const int32_t* tables;
  const int32_t* lens;
  const int32_t* qsl;
  const int32_t* rows;
  const float* scores;
  float* out;
  int64_t* off[kQueues];  // [B + 1] each: first unit of each sequence in the queues
  SeqPlan* plan;    // [B]
  int* tickets;     // tensor-core kernel: stats items done of each row tile (tile_ticket)
  int* ready;       // [B, Hkv] row tiles whose lse are complete
  int* counters;    // next of the tensor-core kernel's and of the few-row kernel's queue
  float2* part;     // (m, l) per (kv head, row, chunk) of a sequence
  float* lse;       // per (kv head, row) of a sequence
  float* logit;     // per (kv head, key, padded row) of a few-row sequence
  int64_t logit_cap;
  int few_chunk;    // keys of a stats unit (few rows)
  int max_query;    // the promised longest query, 0: none
  int own_plan;     // the few-row kernels make the plan themselves (no other kernel runs)
  int tensor;       // sequences of more rows go to the tensor-core kernel
  int tile_tok;     // tokens of a row tile: floor(128 / G)
  int64_t T, num_blocks;
  int B, Hq, Hkv, G, bs, bs_log, max_blocks, num_rows, max_len, causal;
  float scale_log2, decay;
  int* err;
  // Testing only (0 in every ordinary call): a limit of the tensor-core kernel's
  // waits other than 2 s, and the tile load of its first CTA that is left out.
  uint64_t wait_ns;
  int fault_tile;
};

// Row tiles that a call may have for each kv head, at most, and the ticket of
// one.  Sequences' ranges of queries are disjoint and ascend, so tiles counted
// from floor(first query / tokens a tile) + s never meet another sequence's.
__host__ __device__ constexpr int64_t most_tiles(int64_t B, int64_t T, int tile_tok) { return T / tile_tok + B; }
__device__ __forceinline__ int* tile_ticket(const ScoreParams& p, int s, int h, int qstart, int tiles, int tile) {
  return p.tickets + ((int64_t)(qstart / p.tile_tok + s) * p.Hkv + (int64_t)h * tiles + tile);
}

// The sequence s with off[s] <= u < off[s + 1] (the whole warp calls it).
__device__ __forceinline__ int find_seq(const int64_t* off, int B, int64_t u, int lane) {
  int lo = 0, len = B;
  while (len > 1) {
    const int step = (len + 31) / 32;
    const int i = lo + lane * step;
    const uint32_t le = __ballot_sync(0xffffffffu, lane * step < len && off[i] <= u);
    const int k = 31 - __clz(le);  // lane 0 always holds
    const int skip = k * step;
    lo += skip;
    len = min(step, len - skip);
  }
  return lo;
}

__device__ __forceinline__ int ld_acquire(const int* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void add_release(int* p, int v) {
  asm volatile("red.release.gpu.global.add.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// The reference that the exponentials of a running maximum m are taken against.
// A maximum of -inf is that of no keys or of logits of -inf, whose sum is 0, or
// of logits that are all NaN, whose sum is NaN and has to stay so.
__device__ __forceinline__ float max_ref(float m) { return m == -CUDART_INF_F ? 0.f : m; }

// Two E4M3 codes as an fp16 pair, exactly.
__device__ __forceinline__ uint32_t codes_to_f16(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
  return (uint32_t)h.x | ((uint32_t)h.y << 16);
}
// A bf16 pair as an fp16 pair: the 8 bits of mantissa fit; magnitudes above
// 65504 become infinite, those below 2^-14 are off by at most 2^-25.
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w) {
  const __half2 h = __floats2half2_rn(bf16_lo(w), bf16_hi(w));
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The tensor-core kernel for sequences of more than kFewRows rows of bf16
// queries (scores_mma.cu); f8: FP8 pools.
cudaError_t launch_scores_mma(const ScoreParams& p, int D, bool f8, const CUtensorMap& qmap, const CUtensorMap& kmap,
                              int sms, cudaStream_t s);

}  // namespace pkv
