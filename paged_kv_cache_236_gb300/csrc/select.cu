// The positions a budget keeps (paged_kv_select, declared in
// paged_kv_budget.h): of L scores per (sequence, kv head) the first num_sink,
// the last num_recent and the highest between, in ascending position order.
//
// A radix select: the scores map to 32-bit keys whose unsigned order is
// theirs (NaN lowest, -0 as +0); histograms of 11, 11 and 10 bits over the
// middle positions narrow down the value of the last key kept and how many
// equal to it are kept; a pass turns the keys into bit masks (above it, equal to
// it) of 32 positions each, and the masks, counted, say where each kept
// position goes, equals being taken from the lowest position.
//
// Bound by latency and instructions: a (sequence, head) has a few thousand
// scores.  Its keys are read from memory once and kept in shared memory for
// the passes over them; long rows are cut over the blocks of a cluster, which add up their
// histograms and counts through distributed shared memory.  The first digit
// takes 11 bits (sign, exponent, two bits of mantissa) so that scores of one
// magnitude do not all meet in one counter.  Measured: 512 rows of 512 to 4096
// scores 14 us, about half of it the call; 32 rows of 131072 scores 37 us (154
// with one block to a row).
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "paged_kv_budget.h"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kBins = 2048;
constexpr int kHeld = 16384;     // keys of a block kept in shared memory, at most
constexpr int kPerBlock = 8192;  // scores a block takes before a cluster is made larger
constexpr int kMaxCluster = 8;
constexpr int kAhead = 8;        // scores a thread loads at a time

struct SelectParams {
  const float* scores;
  const int32_t* rows;
  const int32_t* lens;
  int32_t* kept;
  int Hkv, num_rows, max_len, budget, sink, recent;
  int cluster, held;  // blocks of a (sequence, head); keys of shared memory each has
  int* err;
};

// Unsigned order of the keys = order of the scores; NaN 0, -inf 1 or more.
__device__ __forceinline__ uint32_t key_of(float x) {
  if (x != x) return 0u;
  const uint32_t b = __float_as_uint(x + 0.f);  // -0 -> +0
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ int warp_scan(int x, int lane) {  // inclusive
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  return x;
}

__device__ __forceinline__ void cluster_sync(int cluster) {
  if (cluster == 1)
    __syncthreads();
  else
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The ints at `p` (this block's shared memory) in block `rank` of the cluster.
__device__ __forceinline__ uint32_t peer_addr(const int* p, int rank) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  return at;
}
__device__ __forceinline__ int peer_int(const int* p, int rank) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(peer_addr(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ int4 peer_int4(const int* p, int rank) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(peer_addr(p, rank))
               : "memory");
  return v;
}

// kThreads: 256 where a row has at most 4096 scores (some of a block's work,
// the histograms' bins above all, does not depend on the row's length), 512
// for longer rows.
template <int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 512 ? 2 : 4) select_kernel(const SelectParams p) {
  constexpr int kWarps = kThreads / 32;
  constexpr int kPer = kBins / kThreads < 4 ? 4 : kBins / kThreads;  // bins of a thread
  extern __shared__ uint32_t keys[];            // [held], then masks [2][held / 32]
  __shared__ __align__(16) int hist[2][kBins];  // this block's counts (by digit parity; peers read them)
  __shared__ int sum[2 * kWarps];
  __shared__ int wsum[kWarps];
  __shared__ int counts[2];  // this block's keys above / equal to the last one kept (peers read them)
  __shared__ int s_bin, s_need, s_count;
  const int block = p.cluster == 1 ? 0 : blockIdx.x % p.cluster;
  const int sh = p.cluster == 1 ? blockIdx.x : blockIdx.x / p.cluster;
  const int s = sh / p.Hkv, h = sh - s * p.Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t* out = p.kept + (int64_t)sh * p.budget;
  const int row = p.rows ? p.rows[s] : s;
  int L = p.lens[s];
  if (row < 0 || row >= p.num_rows || L < 0 || L > p.max_len) {
    if (tid == 0 && block == 0 && row >= 0) raise_error(p.err, PKV_DEVERR_BAD_SEQUENCE);
    L = 0;
  }
  const int all = p.cluster * kThreads, me = block * kThreads + tid;
  if (L <= p.budget) {
    for (int i = me; i < p.budget; i += all) out[i] = i < L ? i : -1;
    return;  // all blocks of the cluster alike
  }
  int need = p.budget - p.sink - p.recent;  // of the L - sink - recent > need middle positions
  for (int i = me; i < p.sink; i += all) out[i] = i;
  for (int i = me; i < p.recent; i += all) out[p.budget - p.recent + i] = L - p.recent + i;
  if (need == 0) return;
  // this block's part of the middle: positions lo .. hi - 1
  const int middle = L - p.recent - p.sink, per = (middle + p.cluster - 1) / p.cluster;
  const int lo = p.sink + min(middle, block * per), hi = p.sink + min(middle, (block + 1) * per);
  const float* sc = p.scores + ((int64_t)row * p.Hkv + h) * p.max_len + lo;
  const int n = hi - lo, held = min(n, p.held);
  for (int i = tid; i < 2 * kBins; i += kThreads) (&hist[0][0])[i] = 0;
  __syncthreads();
  // digit 0 is counted as the keys arrive
  for (int i0 = tid; i0 < n; i0 += kAhead * kThreads) {
    float x[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) x[j] = i0 + j * kThreads < n ? sc[i0 + j * kThreads] : 0.f;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int i = i0 + j * kThreads;
      if (i < n) {
        const uint32_t k = key_of(x[j]);
        if (i < held) keys[i] = k;
        atomicAdd(&hist[0][k >> 21], 1);
      }
    }
  }
  uint32_t prefix = 0, mask = 0;
  bool whole = false;  // every key that starts like prefix is kept
#pragma unroll 1
  for (int digit = 0; digit < 3 && !whole; ++digit) {
    const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0;
    const int bins = digit == 2 ? 1024 : 2048;
    int* mine = hist[digit & 1];
    if (digit > 0) {
      auto count = [&](uint32_t k) {
        if ((k & mask) == prefix) atomicAdd(&mine[(k >> shift) & (bins - 1)], 1);
      };
#pragma unroll 4
      for (int i = tid; i < held; i += kThreads) count(keys[i]);
#pragma unroll 1
      for (int i = held + tid; i < n; i += kThreads) count(key_of(sc[i]));  // what shared memory could not hold
    }
    cluster_sync(p.cluster);  // the counts of every block are complete
    // thread t: the cluster's counts of kPer bins, the highest first
    int c[kPer], total = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) c[j] = 0;
    const int top = bins - 1 - kPer * tid;
    if (top >= 0) {
#pragma unroll
      for (int j = 0; j < kPer; j += 4) {
        const int* at = &mine[top - j - 3];
        if (p.cluster == 1) {
          const int4 v = *reinterpret_cast<const int4*>(at);
          c[j] = v.w;
          c[j + 1] = v.z;
          c[j + 2] = v.y;
          c[j + 3] = v.x;
        } else {
#pragma unroll 1
          for (int b0 = 0; b0 < p.cluster; b0 += 2) {  // a cluster has an even number of blocks
            const int4 v = peer_int4(at, b0), w = peer_int4(at, b0 + 1);
            c[j] += v.w + w.w;
            c[j + 1] += v.z + w.z;
            c[j + 2] += v.y + w.y;
            c[j + 3] += v.x + w.x;
          }
        }
      }
#pragma unroll
      for (int j = 0; j < kPer; ++j) total += c[j];
    }
    const int incl = warp_scan(total, lane);
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    int before = incl - total;
    for (int w = 0; w < warp; ++w) before += wsum[w];
    if (before < need && need <= before + total) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        if (before < need && need <= before + c[j]) {
          s_bin = top - j;
          s_need = need - before;
          s_count = c[j];
        }
        before += c[j];
      }
    }
    // the other digit's counts, read by peers before the barrier above, start again
    if (digit == 1)
      for (int i = tid; i < kBins; i += kThreads) hist[0][i] = 0;
    __syncthreads();
    prefix |= (uint32_t)s_bin << shift;
    mask |= (uint32_t)(bins - 1) << shift;
    need = s_need;
    whole = s_count == need;
  }
  auto above = [&](uint32_t k) { return whole ? k >= prefix : k > prefix; };
  auto equal = [&](uint32_t k) { return !whole && k == prefix; };
  // `need` of the keys equal to `prefix` are kept, from the lowest position.
  // A warp takes a run of the block's positions, in groups of 32.
  const int groups = (n + 31) >> 5, run = (groups + kWarps - 1) / kWarps, held_groups = held == n ? groups : held >> 5;
  const int ga = min(groups, warp * run), gb = min(groups, ga + run);
  uint32_t* masks = keys + ((p.held + 31) & ~31);  // a group's keys above, and equal
  int gt = 0, eq = 0;  // of the run, in every lane
  auto group_masks = [&](int g, uint32_t& mg, uint32_t& me) {
    const int i = 32 * g + lane;
    const uint32_t k = i < n ? g < held_groups ? keys[i] : key_of(sc[i]) : 0u;
    mg = __ballot_sync(0xffffffffu, i < n && above(k));
    me = __ballot_sync(0xffffffffu, i < n && equal(k));
  };
#pragma unroll 2
  for (int g = ga; g < gb; ++g) {
    uint32_t mg, me;
    group_masks(g, mg, me);
    if (g < held_groups && lane < 2) masks[2 * g + lane] = lane ? me : mg;
    gt += __popc(mg);
    eq += __popc(me);
  }
  if (lane == 0) {
    sum[2 * warp] = gt;
    sum[2 * warp + 1] = eq;
  }
  __syncthreads();
  int gt0 = 0, eq0 = 0;  // before this warp's run
  for (int w = 0; w < warp; ++w) {
    gt0 += sum[2 * w];
    eq0 += sum[2 * w + 1];
  }
  if (p.cluster > 1) {
    if (tid == kThreads - 1) {  // the last warp: the block's totals
      counts[0] = gt0 + gt;
      counts[1] = eq0 + eq;
    }
    cluster_sync(p.cluster);
    int g = lane < block ? peer_int(&counts[0], lane) : 0, e = lane < block ? peer_int(&counts[1], lane) : 0;
#pragma unroll
    for (int d = 4; d > 0; d >>= 1) {  // over the at most kMaxCluster lanes that read
      g += __shfl_xor_sync(0xffffffffu, g, d);
      e += __shfl_xor_sync(0xffffffffu, e, d);
    }
    gt0 += __shfl_sync(0xffffffffu, g, 0);
    eq0 += __shfl_sync(0xffffffffu, e, 0);
    cluster_sync(p.cluster);  // a block's shared memory outlives its readers
  }
  const uint32_t below = (1u << lane) - 1u;
  out += p.sink;
#pragma unroll 2
  for (int g = ga; g < gb; ++g) {
    uint32_t mg, me;
    if (g < held_groups) {
      mg = masks[2 * g];
      me = masks[2 * g + 1];
    } else {
      group_masks(g, mg, me);
    }
    const int e = eq0 + __popc(me & below);
    if ((mg >> lane & 1) || ((me >> lane & 1) && e < need))
      out[gt0 + __popc(mg & below) + min(e, need)] = lo + 32 * g + lane;
    gt0 += __popc(mg);
    eq0 += __popc(me);
  }
}

pkv_status fail(pkv_status st, const char* msg) {
  set_last_error(msg);
  return st;
}

}  // namespace
}  // namespace pkv

extern "C" pkv_status paged_kv_select(const float* scores, const int32_t* score_rows, const int32_t* context_lens,
                                      int32_t* kept, int32_t num_seqs, int32_t num_kv_heads, int32_t num_rows,
                                      int32_t max_len, int32_t budget, int32_t num_sink, int32_t num_recent,
                                      void* stream) {
  using namespace pkv;
  set_last_error("");
  if (num_seqs < 0 || num_kv_heads <= 0 || num_rows <= 0 || max_len <= 0)
    return fail(PKV_ERR_INVALID_ARG, "sizes must be positive (num_seqs >= 0)");
  if (budget <= 0 || num_sink < 0 || num_recent < 0 || (int64_t)num_sink + num_recent > budget)
    return fail(PKV_ERR_INVALID_ARG, "budget must be positive and hold num_sink + num_recent (each >= 0)");
  if (num_seqs > kMaxPlanSeqs || num_kv_heads > 1 << 15)
    return fail(PKV_ERR_UNSUPPORTED, "too many sequences or heads per call");
  if (max_len > 1 << 30 || budget > 1 << 30) return fail(PKV_ERR_UNSUPPORTED, "context too long");
  if (num_seqs == 0) return PKV_OK;
  if (!scores || !context_lens || !kept) return fail(PKV_ERR_INVALID_ARG, "null pointer");
  SelectParams p{scores, score_rows, context_lens, kept, num_kv_heads, num_rows, max_len, budget,
                 num_sink, num_recent, 1, 0, nullptr};
  int sms = 0;
  const pkv_status st = device_state(&sms, &p.err);
  if (st != PKV_OK) return st;
  // blocks of a (sequence, head) by the longest row there can be
  while (p.cluster < kMaxCluster && (int64_t)p.cluster * kPerBlock < max_len) p.cluster *= 2;
  p.held = (std::min((max_len + p.cluster - 1) / p.cluster, kHeld) + 31) & ~31;
  const int64_t grid = (int64_t)num_seqs * num_kv_heads * p.cluster;
  if (grid > ((int64_t)1 << 31) - 1) return fail(PKV_ERR_UNSUPPORTED, "too many sequences and heads");
  const size_t smem = (size_t)(p.held + p.held / 16) * sizeof(uint32_t);  // keys, and two masks for 32
  cudaError_t e = cudaSuccess;
  if (p.cluster > 1 || p.held > kPerBlock / 2) {  // with the static arrays, past the 48 KB every kernel may use
    static unsigned long long done_mask = 0;  // devices set up
    int dev = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return cuda_error(e, "cudaGetDevice");
    if (!(__atomic_load_n(&done_mask, __ATOMIC_ACQUIRE) & (1ull << (dev & 63)))) {
      e = cudaFuncSetAttribute(select_kernel<512>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (kHeld + kHeld / 16) * (int)sizeof(uint32_t));
      if (e != cudaSuccess) return cuda_error(e, "paged_kv_select set-up");
      __atomic_fetch_or(&done_mask, 1ull << (dev & 63), __ATOMIC_RELEASE);
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  const bool small = p.cluster == 1 && max_len <= kPerBlock / 2;
  cfg.blockDim = dim3(small ? 256 : 512);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.cluster > 1 ? 1 : 0;
  e = small ? cudaLaunchKernelEx(&cfg, select_kernel<256>, p) : cudaLaunchKernelEx(&cfg, select_kernel<512>, p);
  if (e != cudaSuccess) return cuda_error(e, "paged_kv_select launch");
  return PKV_OK;
}
