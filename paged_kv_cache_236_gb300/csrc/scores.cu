// The attention weight paid to each cached token (paged_attention_scores,
// declared in paged_kv_budget.h).
//
// For the rows (query i, head g of the group) of one kv head of a sequence:
//   paid[j] = sum_r exp2(z[r][j] - lse[r]),   z = scale * log2(e) * q K^T,
//   lse[r] = log2 sum_j exp2(z[r][j]),
// with the causal mask at each row's position.  A row's normaliser needs all
// its keys before any weight is known, so the keys are passed over twice.
//
// A plan of the call (plan_block) checks each sequence and lays out its work.
//
// Few rows (at most 16: decode, short verify windows): few_kernel, then
// few_columns_kernel.  HBM-bound on K, which is read once: the logits are kept
// (4 bytes a row and key, 16 bytes next to K's 256 for a group of 4 in bf16)
// and the second pass reads them back, mostly from L2.  The stats units (a
// head's chunk of keys: logits, and each row's (max, sum) over the chunk)
// belong to warps, which take them from a counter (dealt out in turn instead,
// the slower SMs finished last: 69 us against 60 on the decode batch); the
// columns are cut into equal spans, one a warp: each row's lse from its
// chunks, the weights summed over the rows, the score update.
// Both passes in one kernel, the warp that ends a head's last chunk announcing
// its lse, was slower: the fence of every unit waits for the copies in flight
// (4 x 131072 keys: 274 us, 178 us without fences; the decode batch 84 us).
// When only these kernels have work, each block of few_kernel makes the plan
// itself, in shared memory, instead of a launch before it.
//
// More rows of bf16 queries (bf16 or FP8 pools): the tensor-core kernel of
// scores_mma.cu.
//
// More rows in fp32, whose products no tensor-core format keeps: stats_kernel,
// lse_kernel, columns_kernel, which compute the logits twice.
//
// Every sum has a fixed order (no float atomics).
//
// Measured: the decode batch (64 sequences of 512 to 4096 tokens, 8 kv heads of
// 128 in bf16) 77 us, 3.9 TB/s of K's 302 MB; 4 x 131072 keys 214 us, 5.0 TB/s of
// its 1.07 GB.  Short calls are bound by their three launches (the queue's
// counter or the plan, the stats, the columns) and one unit's latency (20 us).
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>
#include <math_constants.h>

#include <algorithm>

#include "paged_kv_budget.h"
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "scores.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kFewThreads = 128;
constexpr int kColThreads = 256;

__device__ __forceinline__ int64_t warp_scan(int64_t x, int lane) {  // inclusive
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  return x;
}

constexpr int kPlanThreads = 1024;

// Kept logits of a few-row sequence, rounded up so that the next one's start on
// 16 bytes: rows padded to 4 and more are read as float4, and an odd number of
// keys of rows padded to 2 ends between.
__device__ __forceinline__ int64_t logits_kept(const ScoreParams& p, int L, int pad) {
  return ((int64_t)p.Hkv * L * pad + 3) & ~(int64_t)3;
}
constexpr int kLogitSlack = 2;  // what the rounding adds to a sequence, at most

// Keys of a few-row stats unit: the launch's (few units: short ones, so that
// they spread over the SMs), longer for long sequences (fewer partials), whose
// block ids a warp's lanes hold.
__device__ __forceinline__ int few_chunk(const ScoreParams& p, int L) {
  return L <= 32768 ? p.few_chunk : min(512, 32 * p.bs);
}

// Whether sequence s, of queries a .. b - 1 and L tokens, is left out as
// invalid; high: the largest earlier entry of query_start_loc.
__device__ __forceinline__ bool bad_seq(const ScoreParams& p, int a, int b, int high, int L, int row) {
  return a < high || a < 0 || b < a || b > p.T || L < 0 || b - a > L || L > p.max_len ||
         L > (int64_t)p.max_blocks * p.bs || row >= p.num_rows || (p.max_query > 0 && b - a > p.max_query);
}

// A whole block makes the plan; threads = sequences, in passes of the block's
// size.  The sums are scanned within warps and then, one warp to a sum, over
// the warps.
__device__ __forceinline__ void plan_block(const ScoreParams& p) {
  enum { kPart = kQueues, kLse, kSums };  // sums 0 .. kQueues - 1: the queues
  __shared__ int64_t warp_sum[kSums + 1][32];
  __shared__ int64_t carry[kSums + 1];  // the last: kept logits
  __shared__ int top[32];
  __shared__ int top_carry;  // the largest query_start_loc entry so far
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x, warps = threads >> 5;
  if (tid <= kSums) carry[tid] = 0;
  if (tid == 0) top_carry = 0;
  // after a barrier: the exclusive sums over the warps of sums k0 .. k0 + n - 1, carried on
  auto over_warps = [&](int k0, int n) {
    __syncthreads();
    for (int k = k0 + warp; k < k0 + n; k += warps) {
      const int64_t w = lane < warps ? warp_sum[k][lane] : 0, x = warp_scan(w, lane);
      const int64_t c = carry[k];
      __syncwarp();
      warp_sum[k][lane] = c + x - w;
      if (lane == 31) carry[k] = c + x;
    }
    __syncthreads();
  };
  for (int s0 = 0; s0 < p.B; s0 += threads) {
    const int s = s0 + tid;
    SeqPlan sp{};
    sp.row = -1;
    int a = 0, b = 0, L = 0;
    if (s < p.B) {
      a = p.qsl[s];
      b = p.qsl[s + 1];
      L = p.lens[s];
      sp.row = p.rows ? p.rows[s] : s;
    }
    // a sequence whose queries start below an earlier entry is invalid: the
    // valid ones' query ranges are disjoint, and so are their partials
    int high = a;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, high, d);
      if (lane >= d) high = max(high, y);
    }
    if (lane == 31) top[warp] = high;
    __syncthreads();
    high = max(high, top_carry);
    for (int w = 0; w < warp; ++w) high = max(high, top[w]);
    if (s < p.B) {
      const int n = b - a;
      const bool bad = bad_seq(p, a, b, high, L, sp.row);
      if (bad && sp.row >= 0) raise_error(p.err, PKV_DEVERR_BAD_SEQUENCE);
      if (!bad && sp.row >= 0 && n > 0) {
        sp.L = L;
        sp.n = n;
        sp.rows = n * p.G;  // n tokens of the batch's T, and T * Hq fits 31 bits
      }
    }
    const bool want_few = sp.n > 0 && sp.rows <= kFewRows;
    const int pad = sp.rows <= 2 ? 2 : sp.rows <= 4 ? 4 : sp.rows <= 8 ? 8 : 16;
    const int64_t logits = want_few ? logits_kept(p, sp.L, pad) : 0;
    int64_t x = warp_scan(logits, lane);
    if (lane == 31) warp_sum[kSums][warp] = x;
    over_warps(kSums, 1);
    sp.logit = warp_sum[kSums][warp] + x - logits;
    if (tid == threads - 1) top_carry = high;
    const bool few = want_few && sp.logit + logits <= p.logit_cap;
    sp.kind = sp.n == 0 ? 0 : few ? kFew : p.tensor ? kTensor : kOther;
    sp.pad = few ? pad : 0;
    sp.chunk = sp.kind == kTensor ? kTcRange : sp.kind == kFew ? few_chunk(p, sp.L) : kChunk;
    sp.chunks = (sp.L + sp.chunk - 1) / sp.chunk;
    sp.tiles = sp.kind == kTensor ? (sp.n + p.tile_tok - 1) / p.tile_tok : 0;
    const int64_t work = (int64_t)p.Hkv * sp.chunks;
    int64_t v[kSums];
#pragma unroll
    for (int k = 0; k < kSums; ++k) v[k] = 0;
    v[kPart] = (work * sp.rows + 1) & ~(int64_t)1;  // even: the tensor-core kernel reads pairs
    if (sp.kind == kFew) {
      v[kFewStat] = work;
      v[kFewCol] = (int64_t)p.Hkv * ((sp.L + kColChunk - 1) / kColChunk);
    }
    v[kLse] = (int64_t)p.Hkv * sp.rows;
    if (sp.kind == kOther) {
      v[kStat] = work * ((sp.rows + kRowGroup - 1) / kRowGroup);
      v[kCol] = (int64_t)p.Hkv * ((sp.L + kColTile - 1) / kColTile);
    } else if (sp.kind == kTensor) {
      v[kTcStat] = work * sp.tiles;
      v[kTcCol] = work;
      v[kPart] = 2 * work * sp.rows;  // each of the two epilogue groups writes its own
    }
    int64_t at[kSums];
#pragma unroll
    for (int k = 0; k < kSums; ++k) {
      const int64_t y = warp_scan(v[k], lane);
      at[k] = y - v[k];
      if (lane == 31) warp_sum[k][warp] = y;
    }
    over_warps(0, kSums);
    if (s < p.B) {
#pragma unroll
      for (int k = 0; k < kQueues; ++k) p.off[k][s] = warp_sum[k][warp] + at[k];
      sp.part = warp_sum[kPart][warp] + at[kPart];
      sp.lse = warp_sum[kLse][warp] + at[kLse];
      p.plan[s] = sp;
    }
    __syncthreads();
  }
  if (tid < kQueues) p.off[tid][p.B] = carry[tid];
}

__global__ void __launch_bounds__(kPlanThreads) plan_scores_kernel(const ScoreParams p) {
  pdl_launch_dependents();  // few_kernel waits for this grid first of all
  if (p.tensor) {
    for (int64_t i = threadIdx.x; i < most_tiles(p.B, p.T, p.tile_tok) * p.Hkv; i += blockDim.x) p.tickets[i] = 0;
    for (int64_t i = threadIdx.x; i < (int64_t)p.B * p.Hkv; i += blockDim.x) p.ready[i] = 0;
  }
  if (threadIdx.x < 2) p.counters[threadIdx.x] = 0;
  plan_block(p);
}

// With own_plan: zeroes the few-row queue's counter while few_kernel, started
// early, makes its plan.
__global__ void start_few_kernel(int* counters) {
  pdl_launch_dependents();
  if (threadIdx.x < 2) counters[threadIdx.x] = 0;
}

// plan_block for few-row sequences only, at most two a thread: two scans
// between three barriers.
__device__ __forceinline__ void plan_few(const ScoreParams& p, int64_t* stat, int64_t* col, SeqPlan* plan, bool report) {
  __shared__ int64_t sum[4][8];
  __shared__ int top[8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int a[3], L[2], row[2];
#pragma unroll
  for (int i = 0; i < 3; ++i) a[i] = 2 * tid + i <= p.B ? p.qsl[2 * tid + i] : 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int s = 2 * tid + i;
    L[i] = s < p.B ? p.lens[s] : 0;
    row[i] = s < p.B ? p.rows ? p.rows[s] : s : -1;
  }
  int high = max(a[0], 2 * tid + 1 < p.B ? a[1] : a[0]);
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, high, d);
    if (lane >= d) high = max(high, y);
  }
  int before = __shfl_up_sync(0xffffffffu, high, 1);
  if (lane == 0) before = 0;
  if (lane == 31) top[warp] = high;
  __syncthreads();
  for (int w = 0; w < warp; ++w) before = max(before, top[w]);
  SeqPlan sp[2];
  int64_t v[4] = {0, 0, 0, 0};  // stats units, column units, partials, logits
  int64_t mine[2][4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    SeqPlan& q = sp[i];
    q = SeqPlan{};
    q.row = row[i];
    if (2 * tid + i < p.B) {
      const int n = a[i + 1] - a[i];
      const bool bad = bad_seq(p, a[i], a[i + 1], before, L[i], q.row);
      if (bad && q.row >= 0 && report) raise_error(p.err, PKV_DEVERR_BAD_SEQUENCE);
      if (!bad && q.row >= 0 && n > 0) {
        q.L = L[i];
        q.n = n;
        q.rows = n * p.G;
        q.kind = kFew;
        q.pad = q.rows <= 2 ? 2 : q.rows <= 4 ? 4 : q.rows <= 8 ? 8 : 16;
        q.chunk = few_chunk(p, q.L);
        q.chunks = (q.L + q.chunk - 1) / q.chunk;
      }
      before = max(before, a[i]);
    }
    mine[i][0] = (int64_t)p.Hkv * q.chunks;
    mine[i][1] = (int64_t)p.Hkv * ((q.L + kColChunk - 1) / kColChunk);
    mine[i][2] = mine[i][0] * q.rows;
    mine[i][3] = logits_kept(p, q.L, q.pad);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] += mine[i][k];
  }
  int64_t at[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t x = warp_scan(v[k], lane);
    at[k] = x - v[k];
    if (lane == 31) sum[k][warp] = x;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 4; ++k)
    for (int w = 0; w < warp; ++w) at[k] += sum[k][w];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int s = 2 * tid + i;
    if (s <= p.B) {  // the entry after the last sequence holds the totals
      stat[s] = at[0];
      col[s] = at[1];
    }
    if (s < p.B) {
      sp[i].part = at[2];
      sp[i].logit = at[3];
      plan[s] = sp[i];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) at[k] += mine[i][k];
  }
  if (tid == (int)blockDim.x - 1 && 2 * tid + 2 <= p.B) {  // two sequences to every thread
    stat[p.B] = at[0];
    col[p.B] = at[1];
  }
  __syncthreads();
}

// The few-row kernels' view of the plan: their two queues and the sequences,
// in shared memory when there are at most kHeldSeqs (a unit's look-up is then
// a few dozen cycles, not a chain of global reads).
constexpr int kHeldSeqs = 256;
struct Held {
  const int64_t* stat;
  const int64_t* col;
  const SeqPlan* plan;
};
__host__ __device__ constexpr int held_bytes(int B) {
  return B > kHeldSeqs ? 0 : 2 * (B + 1) * (int)sizeof(int64_t) + B * (int)sizeof(SeqPlan);
}
// own: make the plan here (and publish it, in block 0, for the columns
// kernel), else read the global one (after pdl_wait).
template <bool kMayOwn>
__device__ __forceinline__ Held hold_plan(const ScoreParams& p, uint8_t* smem) {
  Held h{p.off[kFewStat], p.off[kFewCol], p.plan};
  if (p.B > kHeldSeqs) return h;
  int64_t* offs = reinterpret_cast<int64_t*>(smem);
  SeqPlan* plans = reinterpret_cast<SeqPlan*>(offs + 2 * (p.B + 1));
  constexpr int kWords = sizeof(SeqPlan) / 8;
  const int64_t* src = reinterpret_cast<const int64_t*>(p.plan);
  int64_t* dst = reinterpret_cast<int64_t*>(plans);
  if (kMayOwn && p.own_plan) {
    plan_few(p, offs, offs + p.B + 1, plans, blockIdx.x == 0);
    if (blockIdx.x == 0) {
      for (int i = threadIdx.x; i <= p.B; i += blockDim.x) {
        p.off[kFewStat][i] = offs[i];
        p.off[kFewCol][i] = offs[p.B + 1 + i];
      }
      for (int i = threadIdx.x; i < p.B * kWords; i += blockDim.x) reinterpret_cast<int64_t*>(p.plan)[i] = dst[i];
    }
  } else {
    for (int i = threadIdx.x; i <= p.B; i += blockDim.x) {
      offs[i] = h.stat[i];
      offs[p.B + 1 + i] = h.col[i];
    }
    for (int i = threadIdx.x; i < p.B * kWords; i += blockDim.x) dst[i] = src[i];
    __syncthreads();
  }
  return Held{offs, offs + p.B + 1, plans};
}

// ---------------------------------------------------------------------------
// few rows
// ---------------------------------------------------------------------------
// Logits of 16 keys against 8 or 16 rows on one warp, in the accumulator
// layout of mma.m16n8k16: lane (g = lane / 4, t = lane % 4) holds keys g and
// g + 8, rows 2t and 2t + 1 (and 8 more of each with two row tiles).
//
// The contraction may run over d in any order, so lane t of a key takes whole
// 16-byte pieces of its row for its fragments, and the q fragments follow the
// same order.
//
// K comes through a ring of 16-key tiles in shared memory that is the warp's
// own, by asynchronous copies issued kStages tiles ahead, across units: while
// a warp ends one unit (its partials) the first tiles of its next
// are on their way.  With the tiles loaded into registers, two ahead but none
// across units, the decode batch took 95 us where the ring took 84 (77 us
// now): a unit of 32 KB is 12 us of streaming at the rate a warp gets, and
// about 10 us of its end and its successor's start were not covered.
//
// Row r's 16-byte piece i of a tile sits at piece i ^ 4 (r & 1), so that the
// eight lanes (two keys, four pieces) of a shared-memory read take all banks.

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// bf16 rows: 16-byte piece c of lane t is d = 32 c + 8 t .. + 7, two k-steps.
template <int D>
struct DotBf16 {
  static constexpr int kPieces = D / 32;  // 16-byte pieces of a key a lane holds
  static constexpr int kRowBytes = D * 2;
  static constexpr int kQBytes = D * 2;
  static constexpr int kStages = D == 128 ? 3 : 6;  // tiles of a warp's ring
  static constexpr int kBlocks = 4;                 // of an SM
  template <int NT>
  struct Q {
    uint4 w[NT][kPieces];
    int rows;
  };
  template <int NT>
  __device__ static void load_q(Q<NT>& q, int nt, const void* row, int t) {
#pragma unroll
    for (int c = 0; c < kPieces; ++c)
      q.w[nt][c] = row ? __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(row) + c * 64 + t * 16))
                       : make_uint4(0, 0, 0, 0);
  }
  template <int NT>
  __device__ static void dot(float (&acc)[NT][4], const uint4 (&k0)[kPieces], const uint4 (&k1)[kPieces], const Q<NT>& q) {
#pragma unroll
    for (int c = 0; c < kPieces; ++c)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mma_bf16(acc[nt], k0[c].x, k1[c].x, k0[c].y, k1[c].y, q.w[nt][c].x, q.w[nt][c].y);
        mma_bf16(acc[nt], k0[c].z, k1[c].z, k0[c].w, k1[c].w, q.w[nt][c].z, q.w[nt][c].w);
      }
  }
};

// E4M3 rows (D = 128): piece c of lane t is d = 64 c + 16 t .. + 15, four
// k-steps; codes are exact in fp16, and so is a bf16 q of ordinary magnitude
// (|q| < 65504; bits below 2^-24 are rounded away).
struct DotFp8 {
  static constexpr int kPieces = 2;
  static constexpr int kRowBytes = 128;
  static constexpr int kQBytes = 256;
  static constexpr int kStages = 6;
  static constexpr int kBlocks = 4;
  template <int NT>
  struct Q {
    uint32_t w[NT][16];
    int rows;
  };
  template <int NT>
  __device__ static void load_q(Q<NT>& q, int nt, const void* row, int t) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint4 v = row ? __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(row) + (c >> 1) * 128 + t * 32 +
                                                                 (c & 1) * 16))
                          : make_uint4(0, 0, 0, 0);
      q.w[nt][4 * c + 0] = bf16x2_to_f16x2(v.x);
      q.w[nt][4 * c + 1] = bf16x2_to_f16x2(v.y);
      q.w[nt][4 * c + 2] = bf16x2_to_f16x2(v.z);
      q.w[nt][4 * c + 3] = bf16x2_to_f16x2(v.w);
    }
  }
  template <int NT>
  __device__ static void dot(float (&acc)[NT][4], const uint4 (&k0)[2], const uint4 (&k1)[2], const Q<NT>& q) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint32_t x0[4] = {k0[c].x, k0[c].y, k0[c].z, k0[c].w}, x1[4] = {k1[c].x, k1[c].y, k1[c].z, k1[c].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t a0 = codes_to_f16(x0[i] & 0xffffu), a2 = codes_to_f16(x0[i] >> 16);
        const uint32_t a1 = codes_to_f16(x1[i] & 0xffffu), a3 = codes_to_f16(x1[i] >> 16);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_f16(acc[nt], a0, a1, a2, a3, q.w[nt][8 * c + 2 * i], q.w[nt][8 * c + 2 * i + 1]);
      }
    }
  }
};

// fp32 rows: no tensor-core format keeps fp32 products, so FMAs; piece c of
// lane t is d = 16 c + 4 t .. + 3, summed over the quad at the end.  q is read
// per piece (it stays in L1).
template <int D>
struct DotF32 {
  static constexpr int kPieces = D / 16;
  static constexpr int kRowBytes = D * 4;
  static constexpr int kQBytes = D * 4;
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kBlocks = D == 128 ? 3 : 4;
  template <int NT>
  struct Q {
    const float* row[NT];  // this lane's row g of each tile, exchanged by shuffles
    int t, rows;           // rows of the head
  };
  template <int NT>
  __device__ static void load_q(Q<NT>& q, int nt, const void* row, int t) {
    q.row[nt] = static_cast<const float*>(row);
    q.t = t;
  }
  template <int NT>
  __device__ static void dot(float (&acc)[NT][4], const uint4 (&k0)[kPieces], const uint4 (&k1)[kPieces], const Q<NT>& q) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll 2
      for (int r = 0; r < min(8, q.rows - nt * 8); ++r) {
        const float* row = reinterpret_cast<const float*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(q.row[nt]), r * 4));
        float x0 = 0.f, x1 = 0.f;
#pragma unroll
        for (int c = 0; c < kPieces; ++c) {
          const float4 w = __ldg(reinterpret_cast<const float4*>(row + 16 * c + 4 * q.t));
          x0 = fmaf(__uint_as_float(k0[c].x), w.x, x0);
          x1 = fmaf(__uint_as_float(k1[c].x), w.x, x1);
          x0 = fmaf(__uint_as_float(k0[c].y), w.y, x0);
          x1 = fmaf(__uint_as_float(k1[c].y), w.y, x1);
          x0 = fmaf(__uint_as_float(k0[c].z), w.z, x0);
          x1 = fmaf(__uint_as_float(k1[c].z), w.z, x1);
          x0 = fmaf(__uint_as_float(k0[c].w), w.w, x0);
          x1 = fmaf(__uint_as_float(k1[c].w), w.w, x1);
        }
        x0 += __shfl_xor_sync(0xffffffffu, x0, 1);
        x1 += __shfl_xor_sync(0xffffffffu, x1, 1);
        x0 += __shfl_xor_sync(0xffffffffu, x0, 2);
        x1 += __shfl_xor_sync(0xffffffffu, x1, 2);
        if ((r >> 1) == q.t) {
          if (r & 1) {
            acc[nt][1] = x0;
            acc[nt][3] = x1;
          } else {
            acc[nt][0] = x0;
            acc[nt][2] = x1;
          }
        }
      }
  }
};

// One unit of a warp's work: a head's chunk of keys.
struct Unit {
  int s, h, c;  // s < 0: none
  int kb, ke;   // keys kb .. ke - 1
  int blk;      // lane i: physical block of the chunk's i-th block, -1 outside the pool
};

// Issues the copies of the 16 keys at j into a ring tile;
// keys past the end and blocks outside the pool become zeros.  lane_src: the
// lane's place in a block (kv head, first key, piece).
template <typename Dot>
__device__ __forceinline__ void fetch_tile(const ScoreParams& p, const Unit& u, int j, uint32_t tile, int64_t lane_src,
                                           int64_t token_bytes, int lane) {
  constexpr int kChunks = Dot::kRowBytes / 16;                // of a key
  constexpr int kRows = 32 / kChunks < 1 ? 1 : 32 / kChunks;  // keys the warp copies at a time
  const int row0 = lane / kChunks, piece = lane % kChunks;
  const uint32_t dst = tile + row0 * Dot::kRowBytes;
  const uint32_t even = (uint32_t)piece << 4, odd = (uint32_t)(piece ^ 4) << 4;
  const uint32_t mine = kRows == 1 ? even : row0 & 1 ? odd : even;
  const int b0 = __shfl_sync(0xffffffffu, u.blk, ((j - u.kb) >> p.bs_log) & 31);
  const int b1 = __shfl_sync(0xffffffffu, u.blk, ((j + 8 - u.kb) >> p.bs_log) & 31);
  const uint8_t* base = static_cast<const uint8_t*>(p.kc) + lane_src;
  // 8 keys lie in one block
  const uint8_t* src0 = base + (((int64_t)b0 << p.bs_log) + (j & (p.bs - 1))) * token_bytes;
  const uint8_t* src1 = base + (((int64_t)b1 << p.bs_log) + ((j + 8) & (p.bs - 1))) * token_bytes;
  if (b0 >= 0 && b1 >= 0 && j + 16 <= u.ke) {
#pragma unroll
    for (int i = 0; i < 8; i += kRows) {
      copy16(dst + i * Dot::kRowBytes + (kRows == 1 && (i & 1) ? odd : mine), src0);
      copy16(dst + (8 + i) * Dot::kRowBytes + (kRows == 1 && (i & 1) ? odd : mine), src1);
      src0 += kRows * token_bytes;
      src1 += kRows * token_bytes;
    }
  } else {
#pragma unroll 1
    for (int i = 0; i < 16; i += kRows) {
      const int k = i & 7;
      const bool ok = (i < 8 ? b0 : b1) >= 0 && j + i + row0 < u.ke;
      const uint8_t* src = (i < 8 ? src0 : src1) + k * token_bytes;
      copy16(dst + i * Dot::kRowBytes + (kRows == 1 && (i & 1) ? odd : mine), ok ? src : p.kc, ok);
    }
  }
}

// The warp's running state of a stats unit.
template <typename Dot, int NT>
struct Stats {
  typename Dot::template Q<NT> q;
  int vis[NT][2];  // keys that rows nt * 8 + 2t, + 1 see
  float m[NT][2], l[NT][2];

  __device__ __forceinline__ void begin(const ScoreParams& p, const SeqPlan& sp, const Unit& u, int lane) {
    const int g = lane >> 2, t = lane & 3;
    const int qstart = __ldg(p.qsl + u.s);
    q.rows = sp.rows;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = nt * 8 + g, i = r / p.G;
      const void* row = r < sp.rows ? static_cast<const uint8_t*>(p.q) +
                                          ((int64_t)(qstart + i) * p.Hq + u.h * p.G + (r - i * p.G)) * Dot::kQBytes
                                    : nullptr;
      Dot::load_q(q, nt, row, t);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int mine = nt * 8 + 2 * t + e;
        // padding rows see nothing: their zeros against an infinite key are NaN
        vis[nt][e] = mine >= sp.rows ? 0 : p.causal ? min(sp.L, sp.L - sp.n + mine / p.G + 1) : sp.L;
        m[nt][e] = -CUDART_INF_F;
        l[nt][e] = 0.f;
      }
    }
  }

  // The 16 keys at j, in `tile`; z: where the lane keeps its logits of key
  // j + g (null: its rows are past the padding), those of j + g + 8 follow at
  // z8.
  __device__ __forceinline__ void use(const ScoreParams& p, int j, int ke, const uint8_t* tile, float* z, int z8, int lane) {
    const int g = lane >> 2, t = lane & 3;
    uint4 k0[Dot::kPieces], k1[Dot::kPieces];
    // piece 4i + t: the swizzle flips bit 2 of it, the low bit of i
    const uint8_t* row = tile + g * Dot::kRowBytes + (t << 4);
    const uint8_t* rows[2] = {row + (g & 1) * 64, row + ((g & 1) ^ 1) * 64};
#pragma unroll
    for (int i = 0; i < Dot::kPieces; ++i) {
      k0[i] = *reinterpret_cast<const uint4*>(rows[i & 1] + (i >> 1) * 128);
      k1[i] = *reinterpret_cast<const uint4*>(rows[i & 1] + (i >> 1) * 128 + 8 * Dot::kRowBytes);
    }
    float acc[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
    Dot::dot(acc, k0, k1, q);
    const int ja = j + g, jb = j + g + 8;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float za[2], zb[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        za[e] = acc[nt][e] * p.scale_log2;
        zb[e] = acc[nt][2 + e] * p.scale_log2;
        if (ja >= vis[nt][e]) za[e] = -CUDART_INF_F;
        if (jb >= vis[nt][e]) zb[e] = -CUDART_INF_F;
        const float mn = fmax3(m[nt][e], za[e], zb[e]);
        const float mu = max_ref(mn);
        l[nt][e] = fmaf(l[nt][e], fast_exp2(m[nt][e] - mu), fast_exp2(za[e] - mu) + fast_exp2(zb[e] - mu));
        m[nt][e] = mn;
      }
      if (z && (NT == 1 || z8 >= 128 || nt == 0)) {  // 16 padded rows: 8 more at z + 8
        if (ja < ke) *reinterpret_cast<float2*>(z + nt * 8) = make_float2(za[0], za[1]);
        if (jb < ke) *reinterpret_cast<float2*>(z + z8 + nt * 8) = make_float2(zb[0], zb[1]);
      }
    }
  }

  // (max, sum) of each row over the chunk: over the 8 lanes (keys) that share it.
  __device__ __forceinline__ void end(const ScoreParams& p, const SeqPlan& sp, const Unit& u, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mm = m[nt][e];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, d));
        float ll = l[nt][e] * fast_exp2(m[nt][e] - max_ref(mm));
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) ll += __shfl_xor_sync(0xffffffffu, ll, d);
        const int r = nt * 8 + 2 * t + e;
        if (g == 0 && r < sp.rows)
          p.part[sp.part + ((int64_t)u.h * sp.rows + r) * sp.chunks + u.c] = make_float2(mm, ll);
      }
  }
};

// lse of one row from its chunks' (max, sum), on a whole warp.
__device__ __forceinline__ float row_lse(const float2* part, int chunks, int lane) {
  float m = -CUDART_INF_F, l = 0.f;
  for (int c0 = 0; c0 < chunks; c0 += 128) {
    float2 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = c0 + i * 32 + lane;
      v[i] = c < chunks ? __ldcg(part + c) : make_float2(-CUDART_INF_F, 0.f);
    }
    const float mn = fmaxf(fmax3(m, v[0].x, v[1].x), fmaxf(v[2].x, v[3].x));
    const float mu = max_ref(mn);
    l *= fast_exp2(m - mu);
#pragma unroll
    for (int i = 0; i < 4; ++i) l = fmaf(v[i].y, fast_exp2(v[i].x - mu), l);
    m = mn;
  }
  float top = m;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  l *= fast_exp2(m - max_ref(top));
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
  return top + log2f(l);
}

// NT: tiles of 8 rows (1 where every sequence has at most 8 rows).
template <typename Dot, int NT>
__global__ void __launch_bounds__(kFewThreads, Dot::kBlocks) few_kernel(const ScoreParams p) {
  constexpr int kStages = Dot::kStages, kTileBytes = 16 * Dot::kRowBytes;
  pdl_launch_dependents();  // few_columns_kernel waits for this grid
  if (!p.own_plan) {  // the plan; else only the queue's counter is waited for, below
    pdl_wait();
    if (p.off[kFewStat][p.B] == 0) return;
  }
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Held held = hold_plan<true>(p, smem + kFewThreads / 32 * kStages * kTileBytes);
  const SeqPlan* plan = held.plan;
  if (p.own_plan) pdl_wait();
  const int64_t n_units = held.stat[p.B];
  uint8_t* ring = smem + warp * kStages * kTileBytes;
  const uint32_t ring_u32 = smem_u32(ring);

  int next = 0;  // lane 0: the unit after the one being looked up
  if (lane == 0) next = atomicAdd(p.counters + 1, 1);
  auto look_up = [&]() {
    Unit u{-1, 0, 0, 0, 0, -1};
    const int at = __shfl_sync(0xffffffffu, next, 0);
    if (at >= n_units) return u;
    if (lane == 0) next = atomicAdd(p.counters + 1, 1);
    u.s = find_seq(held.stat, p.B, at, lane);
    // heads innermost: neighbouring warps read neighbouring parts of the same tokens' rows
    const int w = (int)(at - held.stat[u.s]);
    u.c = w / p.Hkv;
    u.h = w - u.c * p.Hkv;
    u.kb = u.c * plan[u.s].chunk;
    u.ke = min(plan[u.s].L, u.kb + plan[u.s].chunk);
    if (lane < ((u.ke - u.kb + p.bs - 1) >> p.bs_log)) {  // chunk / bs <= 32 blocks
      u.blk = __ldg(p.tables + (int64_t)u.s * p.max_blocks + (u.kb >> p.bs_log) + lane);
      if (u.blk < 0 || u.blk >= p.num_blocks) {
        raise_error(p.err, PKV_DEVERR_BLOCK_OUT_OF_RANGE);
        u.blk = -1;
      }
    }
    return u;
  };

  int ahead_by = 0;                     // tiles issued and not used yet
  int put = 0, get = 0;                 // their ring slots: the next to fill, the next to use
  Unit now = look_up(), after{-1, 0, 0, 0, 0, -1};
  bool ahead = false;                   // the next tile to issue is `after`'s (or else `now`'s)
  int at = now.kb;                      // its first key
  constexpr int kChunks = Dot::kRowBytes / 16;
  const int64_t token_bytes = (int64_t)p.Hkv * Dot::kRowBytes;
  const int64_t lane_src = (lane / kChunks) * token_bytes + (lane % kChunks) * 16;
  // issue a tile of `now`, or then of `after`, if there is one and room for it
  auto issue = [&](bool may_go_on) {
    if (ahead_by == kStages) return false;
    if (!ahead && at >= now.ke) {
      if (!may_go_on) return false;
      ahead = true;
      at = after.kb;
    }
    if (ahead && at >= after.ke) return false;
    Unit u = now;
    if (ahead) u = after;
    fetch_tile<Dot>(p, u, at, ring_u32 + put * kTileBytes, lane_src + u.h * Dot::kRowBytes, token_bytes, lane);
    copy_commit();
    put = put + 1 == kStages ? 0 : put + 1;
    ++ahead_by;
    at += 16;
    return true;
  };
  // One loop with each step in one place: units are short, and what runs once
  // a unit is bound by the fetch of its instructions.
  Stats<Dot, NT> st;
  SeqPlan sp{};
  float* z = nullptr;
  int j = 0;
  bool fresh = true;  // `now` has not been begun
  while (now.s >= 0) {
    while (issue(!fresh)) {
    }
    if (fresh) {
      after = look_up();  // while the tiles come
      sp = plan[now.s];
      st.begin(p, sp, now, lane);
      const int g = lane >> 2, t2 = 2 * (lane & 3);
      z = t2 < sp.pad ? p.logit + sp.logit + ((int64_t)now.h * sp.L + now.kb + g) * sp.pad + t2 : nullptr;
      j = now.kb;
      fresh = false;
      continue;
    }
    if (j >= now.ke) {
      st.end(p, sp, now, lane);
      if (!ahead) at = after.kb;
      ahead = false;  // what was issued of `after` is now `now`'s
      now = after;
      fresh = true;
      continue;
    }
    if (ahead_by == kStages)
      copy_wait<kStages - 1>();
    else
      copy_wait<0>();
    __syncwarp();  // every lane's copies of the tile have landed
    st.use(p, j, now.ke, ring + get * kTileBytes, z, 8 * sp.pad, lane);
    __syncwarp();  // the tile may be overwritten
    get = get + 1 == kStages ? 0 : get + 1;
    --ahead_by;
    if (z) z += 16 * sp.pad;
    j += 16;
  }
  copy_wait<0>();
}

// lse of rows r0 .. r0 + 3 of a head from their chunks' (max, sum), on a whole
// warp, all four in flight; +inf past the rows (padding weighs nothing).
__device__ __forceinline__ void rows_lse(const float2* part, int chunks, int rows, int r0, int lane, float (&lse)[4]) {
  float m[4], l[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    m[r] = -CUDART_INF_F;
    l[r] = 0.f;
  }
  for (int c0 = 0; c0 < chunks; c0 += 64) {
    float2 v[4][2];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = c0 + i * 32 + lane;
        v[r][i] = r0 + r < rows && c < chunks ? __ldcg(part + (int64_t)(r0 + r) * chunks + c)
                                              : make_float2(-CUDART_INF_F, 0.f);
      }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float mn = fmax3(m[r], v[r][0].x, v[r][1].x);
      const float mu = max_ref(mn);
      l[r] = l[r] * fast_exp2(m[r] - mu) + (v[r][0].y * fast_exp2(v[r][0].x - mu) + v[r][1].y * fast_exp2(v[r][1].x - mu));
      m[r] = mn;
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    float top = m[r];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    float sum = l[r] * fast_exp2(m[r] - max_ref(top));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    lse[r] = r0 + r < rows ? top + log2f(sum) : CUDART_INF_F;
  }
}

// Weights and scores of keys kb .. ke - 1 of a head from the kept logits, on a
// warp, kAt keys a lane at a time; lse: 16 floats of the warp's own.
__device__ __forceinline__ void few_columns(const ScoreParams& p, const SeqPlan& sp, int h, int kb, int ke, float* lse,
                                            int lane) {
  constexpr int kAt = 4;
  const int pad = sp.pad, quads = (pad + 3) / 4;
  const float* z = p.logit + sp.logit + (int64_t)h * sp.L * pad;
  const int64_t at = ((int64_t)sp.row * p.Hkv + h) * p.max_len;
  __syncwarp();  // the last head's lse have been read
#pragma unroll 1
  for (int r0 = 0; r0 < pad; r0 += 4) {
    float x[4];
    rows_lse(p.part + sp.part + (int64_t)h * sp.rows * sp.chunks, sp.chunks, sp.rows, r0, lane, x);
    if (lane < 4) lse[r0 + lane] = lane == 0 ? x[0] : lane == 1 ? x[1] : lane == 2 ? x[2] : x[3];
  }
  __syncwarp();
  // The last n - 1 keys, which not every row sees: a logit of -inf keeps a row
  // out, but for one whose lse is NaN.
  const int part = max(kb, sp.L - sp.n + 1);
  if (p.causal && part < ke && __any_sync(0xffffffffu, lane < sp.rows && isnan(lse[min(lane, sp.rows - 1)]))) {
    const int j = part + lane;  // n - 1 keys are fewer than kFewRows
    if (j < ke) {
      float paid = 0.f;
#pragma unroll 1
      for (int r = (j - (sp.L - sp.n)) * p.G; r < sp.rows; ++r) paid += fast_exp2(__ldcg(z + (int64_t)j * pad + r) - lse[r]);
      p.out[at + j] = paid;
    }
    ke = part;
  }
#pragma unroll 1
  for (int j0 = kb + lane; j0 - lane < ke; j0 += kAt * 32) {
    float paid[kAt], old[kAt];
#pragma unroll
    for (int i = 0; i < kAt; ++i) {
      const int j = j0 + i * 32;
      old[i] = j < ke && j < sp.L - sp.n && p.decay != 0.f ? p.scores[at + j] : 0.f;
      paid[i] = 0.f;
    }
#pragma unroll 1
    for (int k = 0; k < quads; ++k) {
      const float4 l = *reinterpret_cast<const float4*>(lse + 4 * k);
      float4 x[kAt];
#pragma unroll
      for (int i = 0; i < kAt; ++i) {
        const int j = j0 + i * 32;
        x[i] = make_float4(0.f, 0.f, -CUDART_INF_F, -CUDART_INF_F);
        if (j < ke) {
          if (pad == 2) {
            const float2 v = __ldcg(reinterpret_cast<const float2*>(z + (int64_t)j * 2));
            x[i].x = v.x;
            x[i].y = v.y;
          } else {
            x[i] = __ldcg(reinterpret_cast<const float4*>(z + (int64_t)j * pad) + k);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kAt; ++i)
        paid[i] += (fast_exp2(x[i].x - l.x) + fast_exp2(x[i].y - l.y)) + (fast_exp2(x[i].z - l.z) + fast_exp2(x[i].w - l.w));
    }
#pragma unroll
    for (int i = 0; i < kAt; ++i) {
      const int j = j0 + i * 32;
      if (j < ke) p.out[at + j] = j < sp.L - sp.n && p.decay != 0.f ? fmaf(p.decay, old[i], paid[i]) : paid[i];
    }
  }
}

constexpr int kColBlocks = 4;  // of an SM

__global__ void __launch_bounds__(kColThreads, kColBlocks) few_columns_kernel(const ScoreParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(16) float lse[kColThreads / 32][kFewRows];
  const int lane = threadIdx.x & 31;
  pdl_wait();
  if (p.off[kFewCol][p.B] == 0) return;
  const Held held = hold_plan<false>(p, smem);
  // this warp's span of all heads' keys, in units of kColChunk keys of a head
  const int64_t n_units = held.col[p.B];
  const int warp = blockIdx.x * (kColThreads / 32) + (threadIdx.x >> 5), warps = gridDim.x * (kColThreads / 32);
  int64_t u = n_units * warp / warps;
  const int64_t end = n_units * (warp + 1) / warps;
  while (u < end) {
    const int s = find_seq(held.col, p.B, u, lane);
    const SeqPlan& sp = held.plan[s];
    const int w = (int)(u - held.col[s]), per_head = (sp.L + kColChunk - 1) / kColChunk;
    const int h = w / per_head, c = w - h * per_head, count = (int)min(end - u, (int64_t)(per_head - c));
    const int kb = c * kColChunk, ke = min(sp.L, (c + count) * kColChunk);
    u += count;
    few_columns(p, sp, h, kb, ke, lse[threadIdx.x >> 5], lane);
  }
}

// ---------------------------------------------------------------------------
// more rows in fp32
// ---------------------------------------------------------------------------
// A block's tile of the product: kRowGroup rows against kTileKeys keys; warp w has
// rows 8 w .. + 7, lane l keys l and l + 32.  Rows of shared memory are 4 floats
// longer than D, so that eight keys' 16-byte pieces take all banks.  For 4 values of
// d a warp reads 2 pieces of keys (4 cycles of shared memory each) and 8 of rows (a
// broadcast each) and makes 64 products a lane, 16 cycles of the SM's FMA lanes.
//
// Bound by latency: of a tile's 17000 cycles, four blocks beside each other, 6000 go
// into the copies, 8000 into the products (a third of the FMA rate over all).
// 40 rows against 16 x 8192 keys of 8 heads of 128: 993 us; 4 rows and 4 keys a
// thread, 16 lanes to a row group: 1186; 128 keys a tile and two blocks an SM: 1240;
// three blocks without spills: 1124.
constexpr int kTileThreads = 128;
constexpr int kWarpRows = kRowGroup / (kTileThreads / 32);
constexpr int kTileKeys = kColTile;
constexpr int kLaneKeys = kTileKeys / 32;
constexpr int kTileBlocks = 4;  // of an SM: some load while others multiply

template <int D>
struct Tile {
  static constexpr int kPitch = D + 4;
  static constexpr int kSmem = (kTileKeys + kRowGroup) * kPitch * (int)sizeof(float);
  const float* k;  // [kTileKeys][kPitch]
  const float* q;  // [kRowGroup][kPitch]

  // Rows of the row group rg of kv head h (past the end: zeros).  Ends with the
  // copies under way.
  __device__ static void load_q(const ScoreParams& p, const SeqPlan& sp, int qstart, int h, int rg, float* q) {
    const uint32_t dst = smem_u32(q);
    for (int i = threadIdx.x; i < kRowGroup * (D / 4); i += kTileThreads) {
      const int r = i / (D / 4), d = i % (D / 4) * 4, row = rg * kRowGroup + r;
      const bool ok = row < sp.rows;
      const int t = ok ? row / p.G : 0, g = ok ? row - t * p.G : 0;
      copy16(dst + (r * kPitch + d) * 4,
             static_cast<const float*>(p.q) + ((int64_t)(qstart + t) * p.Hq + h * p.G + g) * D + d, ok);
    }
  }
  // Keys j0 .. of kv head h (past the sequence, or in a block outside the pool: zeros).
  __device__ static void load_k(const ScoreParams& p, const SeqPlan& sp, const int32_t* bt, int h, int j0, float* k) {
    const uint32_t dst = smem_u32(k);
    constexpr int kLanes = D / 4;  // that read a key's row
    const int d = threadIdx.x % kLanes * 4, token = p.Hkv * D;
    const int64_t block = (int64_t)p.bs * token;
    const float* src = static_cast<const float*>(p.kc) + h * D + d;
#pragma unroll 4
    for (int key = threadIdx.x / kLanes; key < kTileKeys; key += kTileThreads / kLanes) {
      const int j = j0 + key;
      const int b = j < sp.L ? __ldg(bt + (j >> p.bs_log)) : 0;
      const bool in = b >= 0 && b < p.num_blocks;
      if (!in) raise_error(p.err, PKV_DEVERR_BLOCK_OUT_OF_RANGE);
      const bool ok = in && j < sp.L;
      const float* at = src + (int64_t)(ok ? b : 0) * block + (ok ? (int64_t)(j & (p.bs - 1)) * token : 0);
      copy16(dst + (key * kPitch + d) * 4, at, ok);
    }
  }
  // z[i][j]: logit (times scale * log2 e) of the warp's row i and key lane + 32 j.
  // fp32 products and sums, two of them at a time over even and odd d.
  __device__ __forceinline__ void product(float scale_log2, float (&z)[kWarpRows][kLaneKeys]) const {
    f32x2 acc[kWarpRows][kLaneKeys];
#pragma unroll
    for (int i = 0; i < kWarpRows; ++i)
#pragma unroll
      for (int j = 0; j < kLaneKeys; ++j) acc[i][j] = 0;
    const float* qr = q + (threadIdx.x >> 5) * kWarpRows * kPitch;
    const float* kr = k + (threadIdx.x & 31) * kPitch;
    // a step's pieces are read while the step before is multiplied
    ulonglong2 x[2][kWarpRows], y[2][kLaneKeys];
    auto read = [&](int at, int d) {
#pragma unroll
      for (int j = 0; j < kLaneKeys; ++j) y[at][j] = *reinterpret_cast<const ulonglong2*>(kr + j * 32 * kPitch + d);
#pragma unroll
      for (int i = 0; i < kWarpRows; ++i) x[at][i] = *reinterpret_cast<const ulonglong2*>(qr + i * kPitch + d);
    };
    auto multiply = [&](int at) {
#pragma unroll
      for (int i = 0; i < kWarpRows; ++i)
#pragma unroll
        for (int j = 0; j < kLaneKeys; ++j)
          acc[i][j] = fma2(x[at][i].y, y[at][j].y, fma2(x[at][i].x, y[at][j].x, acc[i][j]));
    };
    read(0, 0);
#pragma unroll 1
    for (int d = 0; d < D; d += 8) {
      read(1, d + 4);
      multiply(0);
      if (d + 8 < D) read(0, d + 8);
      multiply(1);
    }
#pragma unroll
    for (int i = 0; i < kWarpRows; ++i)
#pragma unroll
      for (int j = 0; j < kLaneKeys; ++j) {
        const float2 v = up2(acc[i][j]);
        z[i][j] = (v.x + v.y) * scale_log2;
      }
  }
};

// Keys that row `row` of a kv head sees.
__device__ __forceinline__ int keys_seen(const ScoreParams& p, const SeqPlan& sp, int row) {
  return row >= sp.rows ? 0 : p.causal ? sp.L - sp.n + row / p.G + 1 : sp.L;
}
// The same of rows row0 .. + 7, with one division.
__device__ __forceinline__ void keys_seen(const ScoreParams& p, const SeqPlan& sp, int row0, int (&see)[kWarpRows]) {
  int t = row0 / p.G, g = row0 - t * p.G;
#pragma unroll
  for (int i = 0; i < kWarpRows; ++i) {
    see[i] = row0 + i >= sp.rows ? 0 : p.causal ? sp.L - sp.n + t + 1 : sp.L;
    if (++g == p.G) {
      g = 0;
      ++t;
    }
  }
}

// (max, sum) of each row over a chunk of keys; a block's unit is a row group and
// a chunk.
template <int D>
__global__ void __launch_bounds__(kTileThreads, kTileBlocks) stats_kernel(const ScoreParams p) {
  using X = Tile<D>;
  extern __shared__ __align__(16) uint8_t smem[];
  float* k = reinterpret_cast<float*>(smem);
  float* q = k + kTileKeys * X::kPitch;
  const X tile{k, q};
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t total = p.off[kStat][p.B];
  for (int64_t u = blockIdx.x; u < total; u += gridDim.x) {
    const int s = find_seq(p.off[kStat], p.B, u, lane);
    const SeqPlan sp = p.plan[s];
    const int groups = (sp.rows + kRowGroup - 1) / kRowGroup;
    int64_t v = u - p.off[kStat][s];
    const int c = (int)(v % sp.chunks);
    v /= sp.chunks;
    const int rg = (int)(v % groups), h = (int)(v / groups);
    const int32_t* bt = p.tables + (int64_t)s * p.max_blocks;
    const int row0 = rg * kRowGroup + warp * kWarpRows;
    const int last = min(sp.rows, (rg + 1) * kRowGroup) - 1;
    const int ke = min(keys_seen(p, sp, last), (c + 1) * kChunk);  // no row of the group sees more
    float m[kWarpRows], l[kWarpRows];
    int seen[kWarpRows];
    keys_seen(p, sp, row0, seen);
#pragma unroll
    for (int i = 0; i < kWarpRows; ++i) {
      m[i] = -CUDART_INF_F;
      l[i] = 0.f;
    }
    for (int j0 = c * kChunk; j0 < ke; j0 += kTileKeys) {
      __syncthreads();  // the last tile has been read
      if (j0 == c * kChunk) X::load_q(p, sp, p.qsl[s], h, rg, q);
      X::load_k(p, sp, bt, h, j0, k);
      copy_commit();
      copy_wait<0>();
      __syncthreads();
      if (row0 >= sp.rows) continue;  // none of the warp's
      float z[kWarpRows][kLaneKeys];
      tile.product(p.scale_log2, z);
#pragma unroll
      for (int i = 0; i < kWarpRows; ++i) {
        const int see = seen[i] - j0 - lane;
#pragma unroll
        for (int j = 0; j < kLaneKeys; ++j)
          if (j * 32 >= see) z[i][j] = -CUDART_INF_F;
        float mn = m[i];
#pragma unroll
        for (int j = 0; j < kLaneKeys; ++j) mn = fmaxf(mn, z[i][j]);
        const float mu = max_ref(mn);
        l[i] *= fast_exp2(m[i] - mu);
#pragma unroll
        for (int j = 0; j < kLaneKeys; ++j) l[i] += fast_exp2(z[i][j] - mu);
        m[i] = mn;
      }
    }
#pragma unroll
    for (int i = 0; i < kWarpRows; ++i) {
      float mm = m[i];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, d));
      float ll = l[i] * fast_exp2(m[i] - max_ref(mm));
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) ll += __shfl_xor_sync(0xffffffffu, ll, d);
      if (lane == 0 && row0 + i < sp.rows)
        p.part[sp.part + ((int64_t)h * sp.rows + row0 + i) * sp.chunks + c] = make_float2(mm, ll);
    }
  }
}

// lse of each row (one warp a row); blockIdx.y: the sequence.
__global__ void __launch_bounds__(kThreads) lse_kernel(const ScoreParams p) {
  const int lane = threadIdx.x & 31;
  const SeqPlan sp = p.plan[blockIdx.y];
  if (sp.kind != kOther) return;
  for (int w = (blockIdx.x * kThreads + threadIdx.x) >> 5; w < p.Hkv * sp.rows; w += (gridDim.x * kThreads) >> 5) {
    const float x = row_lse(p.part + sp.part + (int64_t)w * sp.chunks, sp.chunks, lane);
    if (lane == 0) p.lse[sp.lse + w] = x;
  }
}

// The weights of kTileKeys keys summed over the rows, and their scores; a block's
// unit is a tile of keys and all row groups that see any of it.
template <int D>
__global__ void __launch_bounds__(kTileThreads, kTileBlocks) columns_kernel(const ScoreParams p) {
  using X = Tile<D>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float sums[kTileThreads / 32][kTileKeys];
  float* k = reinterpret_cast<float*>(smem);
  float* q = k + kTileKeys * X::kPitch;
  const X tile{k, q};
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t total = p.off[kCol][p.B];
  for (int64_t u = blockIdx.x; u < total; u += gridDim.x) {
    const int s = find_seq(p.off[kCol], p.B, u, lane);
    const SeqPlan sp = p.plan[s];
    const int groups = (sp.rows + kRowGroup - 1) / kRowGroup, tiles = (sp.L + kTileKeys - 1) / kTileKeys;
    const int64_t v = u - p.off[kCol][s];
    const int j0 = (int)(v % tiles) * kTileKeys, h = (int)(v / tiles);
    const int32_t* bt = p.tables + (int64_t)s * p.max_blocks;
    const int qstart = p.qsl[s];
    // the first row that sees key j0
    const int first = p.causal ? max(0, j0 - (sp.L - sp.n)) * p.G : 0;
    float paid[kLaneKeys] = {};
    for (int rg = first / kRowGroup; rg < groups; ++rg) {
      __syncthreads();  // the last tile, and the last unit's sums, have been read
      if (rg == first / kRowGroup) X::load_k(p, sp, bt, h, j0, k);
      X::load_q(p, sp, qstart, h, rg, q);
      copy_commit();
      const int row0 = rg * kRowGroup + warp * kWarpRows;
      float lse[kWarpRows];
#pragma unroll
      for (int i = 0; i < kWarpRows; ++i)
        lse[i] = row0 + i < sp.rows ? __ldg(p.lse + sp.lse + (int64_t)h * sp.rows + row0 + i) : 0.f;
      copy_wait<0>();
      __syncthreads();
      if (row0 >= sp.rows) continue;  // none of the warp's
      float z[kWarpRows][kLaneKeys];
      tile.product(p.scale_log2, z);
      int seen[kWarpRows];
      keys_seen(p, sp, row0, seen);
#pragma unroll
      for (int i = 0; i < kWarpRows; ++i) {
        const int see = seen[i] - j0 - lane;
#pragma unroll
        for (int j = 0; j < kLaneKeys; ++j) paid[j] += j * 32 < see ? fast_exp2(z[i][j] - lse[i]) : 0.f;
      }
    }
#pragma unroll
    for (int j = 0; j < kLaneKeys; ++j) sums[warp][lane + 32 * j] = paid[j];
    __syncthreads();
    const int j = j0 + threadIdx.x;
    if (threadIdx.x < kTileKeys && j < sp.L) {
      float x = 0.f;
#pragma unroll
      for (int r = 0; r < kTileThreads / 32; ++r) x += sums[r][threadIdx.x];
      const int64_t at = ((int64_t)sp.row * p.Hkv + h) * p.max_len + j;
      if (j < sp.L - sp.n && p.decay != 0.f) x = fmaf(p.decay, p.scores[at], x);
      p.out[at] = x;
    }
  }
}

pkv_status fail(pkv_status st, const char* msg) {
  set_last_error(msg);
  return st;
}

constexpr size_t kAlign = 256;
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

struct Layout {
  size_t off[kQueues], plan, tickets, ready, counters, lse, part, logit, least, total;
};

// Kept logits: at most 16 padded rows of each kv head, or twice the rows
// there are, times the keys; no more than kLogitMax is asked for.  The rounding
// of each sequence's comes on top, so that it never decides what fits.
constexpr size_t kLogitMax = (size_t)512 << 20;

// Tokens of a row tile of the tensor-core kernel.
int tile_tokens(int G) { return std::max(1, 128 / std::max(1, G)); }

Layout layout(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t keys) {
  Layout l{};
  size_t at = 0;
  for (int k = 0; k < kQueues; ++k) {
    l.off[k] = at;
    at = align_up(at + (size_t)(B + 1) * sizeof(int64_t));
  }
  l.plan = at;
  at = align_up(at + (size_t)B * sizeof(SeqPlan));
  l.tickets = at;
  at = align_up(at + (size_t)(most_tiles(B, T, tile_tokens((int)(Hq / Hkv))) * Hkv) * sizeof(int));
  l.ready = at;
  at = align_up(at + (size_t)(B * Hkv) * sizeof(int));
  l.counters = at;
  at = align_up(at + 2 * sizeof(int));
  l.lse = at;
  at = align_up(at + (size_t)(T * Hq) * sizeof(float));
  l.part = at;
  const size_t rows = (size_t)std::min(2 * T * Hq, kFewRows * B * Hkv);
  // few rows: a partial a row and chunk of kFewLeast keys or more.  Other rows: chunks of
  // 256; the tensor-core kernel's two partials a range of 1024 keys take no more than
  // one entry beside one a 512 keys.  A sequence's are rounded to pairs.
  const size_t parts = rows * (size_t)((keys + kFewLeast - 1) / kFewLeast) +
                       (size_t)(T * Hq) * (size_t)((keys + kChunk - 1) / kChunk + 1) + (size_t)B;
  at = align_up(at + parts * sizeof(float2));
  l.logit = l.least = at;
  l.total = align_up(at + std::min(rows * (size_t)keys * sizeof(float), kLogitMax) + (size_t)B * kLogitSlack * sizeof(float));
  return l;
}

template <typename Dot, int NT>
cudaError_t launch_few(const ScoreParams& p, int sms, cudaStream_t s) {
  constexpr int kRing = kFewThreads / 32 * Dot::kStages * 16 * Dot::kRowBytes;
  constexpr int kMost = kRing + held_bytes(kHeldSeqs);
  static unsigned long long done_mask = 0;  // devices set up
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(__atomic_load_n(&done_mask, __ATOMIC_ACQUIRE) & (1ull << (dev & 63)))) {
    e = cudaFuncSetAttribute(few_kernel<Dot, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (e != cudaSuccess) return e;
    __atomic_fetch_or(&done_mask, 1ull << (dev & 63), __ATOMIC_RELEASE);
  }
  const int smem = kRing + held_bytes(p.B);
  // as many blocks as are resident: shared memory is 228 KB an SM, 1 KB a block goes to the system and 2.5 KB to the plan's sums
  const dim3 grid(sms * std::max(1, std::min(Dot::kBlocks, 228 * 1024 / (smem + 3600))));
  if ((e = launch_pdl(few_kernel<Dot, NT>, grid, dim3(kFewThreads), smem, s, p)) != cudaSuccess) return e;
  return launch_pdl(few_columns_kernel, dim3(sms * kColBlocks), dim3(kColThreads), held_bytes(p.B), s, p);
}

// The plan and the few-row sequences.
template <typename Dot>
cudaError_t launch(const ScoreParams& p, bool one_tile, int sms, cudaStream_t s) {
  if (p.own_plan)
    start_few_kernel<<<1, 32, 0, s>>>(p.counters);
  else
    plan_scores_kernel<<<1, std::min(kPlanThreads, (p.B + 31) / 32 * 32), 0, s>>>(p);
  return one_tile ? launch_few<Dot, 1>(p, sms, s) : launch_few<Dot, 2>(p, sms, s);
}

template <int D>
cudaError_t launch_other(const ScoreParams& p, int sms, cudaStream_t s) {
  constexpr int kSmem = Tile<D>::kSmem;
  static unsigned long long done_mask = 0;  // devices set up
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(__atomic_load_n(&done_mask, __ATOMIC_ACQUIRE) & (1ull << (dev & 63)))) {
    for (const void* f : {(const void*)stats_kernel<D>, (const void*)columns_kernel<D>})
      if ((e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem)) != cudaSuccess) return e;
    __atomic_fetch_or(&done_mask, 1ull << (dev & 63), __ATOMIC_RELEASE);
  }
  const dim3 grid(sms * kTileBlocks), lse_grid(std::max(1, std::min(16, 2048 / p.B)), p.B);
  stats_kernel<D><<<grid, kTileThreads, kSmem, s>>>(p);
  lse_kernel<<<lse_grid, kThreads, 0, s>>>(p);
  columns_kernel<D><<<grid, kTileThreads, kSmem, s>>>(p);
  return cudaGetLastError();
}

ScoreParams score_params(const void* q, const void* kc, const int32_t* tables, const int32_t* lens, const int32_t* qsl,
                         const int32_t* rows, const float* scores, float* out, int B, int64_t T, int Hq, int Hkv,
                         int64_t num_blocks, int bs, int max_blocks, int num_rows, int max_len, int causal,
                         float decay) {
  ScoreParams p{};
  p.q = q;
  p.kc = kc;
  p.tables = tables;
  p.lens = lens;
  p.qsl = qsl;
  p.rows = rows;
  p.scores = scores;
  p.out = out;
  p.B = B;
  p.T = T;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.num_blocks = num_blocks;
  p.bs = bs;
  p.bs_log = bs == 8 ? 3 : bs == 16 ? 4 : bs == 32 ? 5 : 6;
  p.max_blocks = max_blocks;
  p.num_rows = num_rows;
  p.max_len = max_len;
  p.causal = causal ? 1 : 0;
  p.decay = decay;
  return p;
}

pkv_status scores_impl(ScoreParams p, int D, int max_query_len, bool f8, float k_scale, float scale, void* workspace, size_t ws_bytes,
                       pkv_dtype dtype, void* stream) {
  set_last_error("");
  if (dtype != PKV_DTYPE_BF16 && dtype != PKV_DTYPE_F32) return fail(PKV_ERR_UNSUPPORTED, "dtype");
  if (p.B < 0 || p.T < 0 || p.Hq <= 0 || p.Hkv <= 0 || D <= 0 || p.num_blocks <= 0 || p.bs <= 0 ||
      p.max_blocks <= 0 || p.num_rows <= 0 || p.max_len <= 0)
    return fail(PKV_ERR_INVALID_ARG, "sizes must be positive (num_seqs, num_tokens >= 0)");
  if (p.B > kMaxPlanSeqs) return fail(PKV_ERR_UNSUPPORTED, "too many sequences per call");
  if (p.Hq % p.Hkv != 0) return fail(PKV_ERR_INVALID_ARG, "num_q_heads not a multiple of num_kv_heads");
  p.G = p.Hq / p.Hkv;
  if (p.G > 128) return fail(PKV_ERR_UNSUPPORTED, "more than 128 q heads per kv head");
  if (D != 64 && D != 128) return fail(PKV_ERR_UNSUPPORTED, "head_dim (supported: 64, 128)");
  if (f8 && D != 128) return fail(PKV_ERR_UNSUPPORTED, "head_dim with an FP8 cache (supported: 128)");
  if (p.bs != 8 && p.bs != 16 && p.bs != 32 && p.bs != 64)
    return fail(PKV_ERR_UNSUPPORTED, "block_size (supported: 8, 16, 32, 64)");
  if (!(scale > 0.f) || !isfinite(scale)) return fail(PKV_ERR_INVALID_ARG, "scale must be positive and finite");
  if (!(p.decay >= 0.f) || !isfinite(p.decay)) return fail(PKV_ERR_INVALID_ARG, "decay must be finite and >= 0");
  if (max_query_len < 0) return fail(PKV_ERR_INVALID_ARG, "max_query_len must be >= 0");
  if (f8 && (!(k_scale > 0.f) || !isfinite(k_scale)))
    return fail(PKV_ERR_INVALID_ARG, "k_scale must be positive and finite");
  if ((int64_t)p.max_blocks * p.bs > (int64_t)1 << 30 || p.max_len > 1 << 30)
    return fail(PKV_ERR_UNSUPPORTED, "context too long");
  if (p.T > ((int64_t)1 << 31) / ((int64_t)p.Hq * D)) return fail(PKV_ERR_UNSUPPORTED, "num_tokens too large");
  const int64_t keys = std::min<int64_t>(p.max_len, (int64_t)p.max_blocks * p.bs);
  if (p.num_blocks > ((int64_t)1 << 31) - 1) return fail(PKV_ERR_UNSUPPORTED, "num_blocks exceeds int32");
  if ((p.B + p.T) * p.Hkv > (((int64_t)1 << 31) - 1) / ((keys + 127) / 128))
    return fail(PKV_ERR_UNSUPPORTED, "too much work for one call");
  // more rows of bf16 queries go to the tensor-core kernel (its operands come through tensor maps)
  p.tensor = dtype == PKV_DTYPE_BF16;
  p.tile_tok = tile_tokens(p.G);
  const int64_t most_tokens = std::min({p.T, keys, max_query_len > 0 ? (int64_t)max_query_len : p.T});
  if (p.tensor && most_tokens > (int64_t)kMaxRowTiles * p.tile_tok)
    return fail(PKV_ERR_UNSUPPORTED, "too many query rows per kv head of a sequence (split the queries over calls)");
  if (p.B == 0 || p.T == 0) return PKV_OK;
  if (!p.q || !p.kc || !p.tables || !p.lens || !p.qsl || !p.scores || !p.out)
    return fail(PKV_ERR_INVALID_ARG, "null pointer");
  auto bits = [](const void* x) { return reinterpret_cast<uintptr_t>(x); };
  if ((bits(p.q) | bits(p.kc)) & 15u) return fail(PKV_ERR_INVALID_ARG, "q and the cache must be 16-byte aligned");
  if (!workspace || (bits(workspace) & (kAlign - 1)))
    return fail(PKV_ERR_WORKSPACE, "workspace missing or not 256-byte aligned");
  const Layout lay = layout(p.B, p.T, p.Hq, p.Hkv, keys);
  if (ws_bytes < lay.least) return fail(PKV_ERR_WORKSPACE, "workspace smaller than required");
  int sms = 0;
  const pkv_status st = device_state(&sms, &p.err);
  if (st != PKV_OK) return st;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  for (int k = 0; k < kQueues; ++k) p.off[k] = reinterpret_cast<int64_t*>(ws + lay.off[k]);
  p.plan = reinterpret_cast<SeqPlan*>(ws + lay.plan);
  p.tickets = reinterpret_cast<int*>(ws + lay.tickets);
  p.ready = reinterpret_cast<int*>(ws + lay.ready);
  p.counters = reinterpret_cast<int*>(ws + lay.counters);
  p.lse = reinterpret_cast<float*>(ws + lay.lse);
  p.part = reinterpret_cast<float2*>(ws + lay.part);
  p.logit = reinterpret_cast<float*>(ws + lay.logit);
  p.logit_cap = (int64_t)((ws_bytes - lay.least) / sizeof(float));
  p.scale_log2 = (f8 ? scale * k_scale : scale) * 1.4426950408889634f;
  // every sequence has few rows (the plan holds them to the promised query
  // length), and their logits fit: the other kernels have nothing to do
  const int64_t most_rows = std::min<int64_t>(p.T, max_query_len > 0 ? max_query_len : p.T) * p.G;
  const bool only_few = most_rows <= kFewRows && std::min(2 * p.T * p.Hq, (int64_t)kFewRows * p.B * p.Hkv) * keys +
                                                         (int64_t)p.B * kLogitSlack <= p.logit_cap;
  p.own_plan = only_few && p.B <= kHeldSeqs;
  const bool one_tile = most_rows <= 8;
  // stats units there may be at most, against the warps that take them
  const int64_t units = (int64_t)p.B * p.Hkv * ((keys + kFewChunk - 1) / kFewChunk), warps = (int64_t)sms * 8;
  p.few_chunk = std::max(p.bs, 4 * units <= warps ? kFewLeast : 2 * units <= warps ? 2 * kFewLeast : kFewChunk);
  p.max_query = max_query_len;
  take_debug_fault(&p.fault_tile, &p.wait_ns);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  CUtensorMap qmap, kmap;
  pkv_status mst;
  if (p.tensor && !only_few) {
    if ((mst = rows_map(&qmap, p.q, p.T, p.Hq, D, p.G, p.tile_tok)) != PKV_OK) return mst;
    if ((mst = pool_map(&kmap, p.kc, p.num_blocks, p.bs, p.Hkv, D, f8)) != PKV_OK) return mst;
  }
  cudaError_t e;
  if (f8)
    e = launch<DotFp8>(p, one_tile, sms, s);
  else if (p.tensor)
    e = D == 128 ? launch<DotBf16<128>>(p, one_tile, sms, s) : launch<DotBf16<64>>(p, one_tile, sms, s);
  else
    e = D == 128 ? launch<DotF32<128>>(p, one_tile, sms, s) : launch<DotF32<64>>(p, one_tile, sms, s);
  if (e == cudaSuccess && !only_few)
    e = p.tensor ? launch_scores_mma(p, D, f8, qmap, kmap, sms, s)
                 : D == 128 ? launch_other<128>(p, sms, s) : launch_other<64>(p, sms, s);
  if (e != cudaSuccess) return cuda_error(e, "paged_attention_scores launch");
  return PKV_OK;
}

}  // namespace
}  // namespace pkv

extern "C" {

size_t paged_attention_scores_workspace_size(int32_t num_seqs, int64_t num_tokens, int32_t num_q_heads,
                                             int32_t num_kv_heads, int64_t max_context) {
  if (num_seqs < 0 || num_tokens < 0 || num_kv_heads <= 0 || num_q_heads <= 0 || max_context < 0) return 0;
  return pkv::layout(num_seqs, num_tokens, num_q_heads, num_kv_heads, max_context).total;
}

size_t paged_attention_scores_workspace_min(int32_t num_seqs, int64_t num_tokens, int32_t num_q_heads,
                                            int32_t num_kv_heads, int64_t max_context) {
  if (num_seqs < 0 || num_tokens < 0 || num_kv_heads <= 0 || num_q_heads <= 0 || max_context < 0) return 0;
  return pkv::layout(num_seqs, num_tokens, num_q_heads, num_kv_heads, max_context).least;
}

pkv_status paged_attention_scores(const void* q, const void* k_cache, const int32_t* block_tables,
                                  const int32_t* context_lens, const int32_t* query_start_loc,
                                  const int32_t* score_rows, const float* scores, float* scores_out,
                                  int32_t num_seqs, int64_t num_tokens, int32_t num_q_heads, int32_t num_kv_heads,
                                  int32_t head_dim, int64_t num_blocks, int32_t block_size,
                                  int32_t max_blocks_per_seq, int32_t num_rows, int32_t max_len,
                                  int32_t max_query_len, float scale, int32_t causal, float decay, void* workspace,
                                  size_t workspace_bytes, pkv_dtype dtype, void* stream) {
  const pkv::ScoreParams p =
      pkv::score_params(q, k_cache, block_tables, context_lens, query_start_loc, score_rows, scores, scores_out,
                        num_seqs, num_tokens, num_q_heads, num_kv_heads, num_blocks, block_size, max_blocks_per_seq,
                        num_rows, max_len, causal, decay);
  return pkv::scores_impl(p, head_dim, max_query_len, false, 1.f, scale, workspace, workspace_bytes, dtype, stream);
}

pkv_status paged_attention_scores_fp8kv(const void* q, const void* k_cache, const int32_t* block_tables,
                                        const int32_t* context_lens, const int32_t* query_start_loc,
                                        const int32_t* score_rows, const float* scores, float* scores_out,
                                        int32_t num_seqs, int64_t num_tokens, int32_t num_q_heads,
                                        int32_t num_kv_heads, int32_t head_dim, int64_t num_blocks,
                                        int32_t block_size, int32_t max_blocks_per_seq, int32_t num_rows,
                                        int32_t max_len, int32_t max_query_len, float scale, int32_t causal,
                                        float decay, float k_scale, void* workspace, size_t workspace_bytes,
                                        void* stream) {
  const pkv::ScoreParams p =
      pkv::score_params(q, k_cache, block_tables, context_lens, query_start_loc, score_rows, scores, scores_out,
                        num_seqs, num_tokens, num_q_heads, num_kv_heads, num_blocks, block_size, max_blocks_per_seq,
                        num_rows, max_len, causal, decay);
  return pkv::scores_impl(p, head_dim, max_query_len, true, k_scale, scale, workspace, workspace_bytes, PKV_DTYPE_BF16, stream);
}

}  // extern "C"
