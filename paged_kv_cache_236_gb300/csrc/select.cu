// The positions a budget keeps (paged_kv_select, declared in
// paged_kv_budget.h): of L scores per (sequence, kv head) the first num_sink,
// the last num_recent and the highest between, in ascending position order.
//
// A radix select: the scores map to 32-bit keys whose unsigned order is
// theirs (NaN lowest, -0 as +0); four passes of 8-bit histograms over the
// middle positions narrow down the value of the last key kept and how many
// equal to it are kept; one more pass writes the kept positions in order,
// taking equals from the lowest position.
#include <cuda_runtime.h>
#include <stdint.h>

#include "paged_kv_budget.h"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 1024;

struct SelectParams {
  const float* scores;
  const int32_t* rows;
  const int32_t* lens;
  int32_t* kept;
  int Hkv, num_rows, max_len, budget, sink, recent;
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

__global__ void __launch_bounds__(kThreads) select_kernel(const SelectParams p) {
  __shared__ int hist[256];
  __shared__ int wsum[2][32];
  __shared__ int s_bin, s_need;
  const int s = blockIdx.x / p.Hkv, h = blockIdx.x - s * p.Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t* out = p.kept + (int64_t)blockIdx.x * p.budget;
  const int row = p.rows ? p.rows[s] : s;
  int L = p.lens[s];
  if (row < 0 || row >= p.num_rows || L < 0 || L > p.max_len) {
    if (tid == 0 && row >= 0) raise_error(p.err, PKV_DEVERR_BAD_SEQUENCE);
    L = 0;
  }
  if (L <= p.budget) {
    for (int i = tid; i < p.budget; i += kThreads) out[i] = i < L ? i : -1;
    return;
  }
  const float* sc = p.scores + ((int64_t)row * p.Hkv + h) * p.max_len;
  const int lo = p.sink, hi = L - p.recent;  // lo <= hi: sink + recent <= budget < L
  int need = p.budget - p.sink - p.recent;   // of the hi - lo > need middle positions
  for (int i = tid; i < p.sink; i += kThreads) out[i] = i;
  for (int i = tid; i < p.recent; i += kThreads) out[p.budget - p.recent + i] = hi + i;
  if (need == 0) return;
  uint32_t prefix = 0, mask = 0;
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    for (int i = lo + tid; i < hi; i += kThreads) {
      const uint32_t k = key_of(sc[i]);
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1);
    }
    __syncthreads();
    if (warp == 0) {
      // bins from the highest down, 8 a lane: the bin holding the need-th key
      int c[8], sum = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        c[j] = hist[255 - (lane * 8 + j)];
        sum += c[j];
      }
      const int incl = warp_scan(sum, lane);
      int before = incl - sum;
      if (before < need && need <= incl) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (before < need && need <= before + c[j]) {
            s_bin = 255 - (lane * 8 + j);
            s_need = need - before;
          }
          before += c[j];
        }
      }
    }
    __syncthreads();
    prefix |= (uint32_t)s_bin << shift;
    mask |= 255u << shift;
    need = s_need;
  }
  // `need` of the keys equal to `prefix` are kept, from the lowest position
  int base = p.sink, eq_seen = 0;
  for (int i0 = lo; i0 < hi; i0 += kThreads) {
    const int i = i0 + tid;
    const uint32_t k = i < hi ? key_of(sc[i]) : 0u;
    const bool gt = i < hi && k > prefix, eq = i < hi && k == prefix;
    const uint32_t beq = __ballot_sync(0xffffffffu, eq);
    const uint32_t below = (1u << lane) - 1u;
    if (lane == 0) wsum[0][warp] = __popc(beq);
    __syncthreads();
    int w = wsum[0][lane];
    int inc = warp_scan(w, lane);
    const int eq_total = __shfl_sync(0xffffffffu, inc, 31);
    const int eq_rank = eq_seen + __shfl_sync(0xffffffffu, inc - w, warp) + __popc(beq & below);
    const bool take = gt || (eq && eq_rank < need);
    const uint32_t bt = __ballot_sync(0xffffffffu, take);
    if (lane == 0) wsum[1][warp] = __popc(bt);
    __syncthreads();
    w = wsum[1][lane];
    inc = warp_scan(w, lane);
    const int total = __shfl_sync(0xffffffffu, inc, 31);
    const int at = base + __shfl_sync(0xffffffffu, inc - w, warp) + __popc(bt & below);
    if (take) out[at] = i;
    base += total;
    eq_seen += eq_total;
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
                 num_sink, num_recent, nullptr};
  int sms = 0;
  const pkv_status st = device_state(&sms, &p.err);
  if (st != PKV_OK) return st;
  select_kernel<<<(unsigned)((int64_t)num_seqs * num_kv_heads), kThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_error(e, "paged_kv_select launch");
  return PKV_OK;
}
