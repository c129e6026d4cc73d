// The attention weight paid to each cached token (paged_attention_scores,
// declared in paged_kv_budget.h).
//
// For the rows (query i, head g of the group) of one kv head of a sequence:
//   paid[j] = sum_r exp2(z[r][j] - lse[r]),   z = scale * log2(e) * q K^T,
//   lse[r] = log2 sum_j exp2(z[r][j]),
// with the causal mask at each row's position.  A row's normaliser needs all
// its keys before any weight is known, so the keys are passed over twice:
//   plan     per sequence: checks, and the offsets of its work and partials;
//   stats    (max, sum) of each row over each chunk of keys;
//   columns  lse from the chunks' (max, sum), then the weights, summed over
//            the rows key by key, and the score update.
// Every sum has a fixed order (no float atomics).
#include <cuda_fp8.h>
#include <math.h>
#include <math_constants.h>

#include <algorithm>

#include "paged_kv_budget.h"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kChunk = 256;   // keys of a work unit
constexpr int kRowGroup = 8;  // rows of a work unit
constexpr int kThreads = 256;

struct SeqPlan {
  int64_t stat_unit;  // first stats unit
  int64_t col_unit;   // first columns unit
  int64_t part;       // first partial (max, sum)
  int L, n, row, chunks;
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
  SeqPlan* plan;   // [B + 1]; the last entry holds the totals
  float2* part;    // (m, l) per (kv head, row, chunk) of a sequence
  float* lse;      // [T, Hq]
  int64_t T, num_blocks;
  int B, Hq, Hkv, G, bs, max_blocks, num_rows, max_len, causal;
  float scale_log2, decay;
  int* err;
};

__global__ void __launch_bounds__(1024) plan_scores_kernel(const ScoreParams p) {
  __shared__ int64_t part[3][32];
  __shared__ int64_t carry[3];
  __shared__ int top[32];
  __shared__ int top_carry;  // the largest query_start_loc entry so far
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < 3) carry[tid] = 0;
  if (tid == 3) top_carry = 0;
  __syncthreads();
  for (int s0 = 0; s0 < p.B; s0 += 1024) {
    const int s = s0 + tid;
    int L = 0, n = 0, row = -1, chunks = 0;
    int64_t v[3] = {0, 0, 0};
    // a sequence whose queries start below an earlier entry is invalid: the
    // valid ones' query ranges are disjoint, and so are their partials
    const int a = s < p.B ? p.qsl[s] : 0;
    int high = a;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, high, d);
      if (lane >= d) high = max(high, y);
    }
    if (lane == 31) top[warp] = high;
    __syncthreads();
    for (int w = 0; w < warp; ++w) high = max(high, top[w]);
    high = max(high, top_carry);
    if (s < p.B) {
      const int b = p.qsl[s + 1];
      L = p.lens[s];
      n = b - a;
      row = p.rows ? p.rows[s] : s;
      const bool bad = a < high || a < 0 || n < 0 || b > p.T || L < 0 || n > L || L > p.max_len ||
                       L > (int64_t)p.max_blocks * p.bs || row >= p.num_rows;
      if (bad && row >= 0) raise_error(p.err, PKV_DEVERR_BAD_SEQUENCE);
      if (bad || row < 0 || n == 0) L = n = 0;
      chunks = (L + kChunk - 1) / kChunk;
      const int64_t rows = (int64_t)n * p.G;
      v[0] = (int64_t)p.Hkv * ((rows + kRowGroup - 1) / kRowGroup) * chunks;
      v[1] = (int64_t)p.Hkv * chunks;
      v[2] = (int64_t)p.Hkv * rows * chunks;
    }
    int64_t ex[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      int64_t x = v[k];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
      }
      ex[k] = x - v[k];
      if (lane == 31) part[k][warp] = x;
    }
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const int64_t w = part[k][lane];
        int64_t x = w;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
          if (lane >= d) x += y;
        }
        part[k][lane] = carry[k] + x - w;
        if (lane == 31) carry[k] += x;
      }
    }
    __syncthreads();
    if (tid == 1023) top_carry = high;
    if (s < p.B)
      p.plan[s] = SeqPlan{part[0][warp] + ex[0], part[1][warp] + ex[1], part[2][warp] + ex[2], L, n, row, chunks};
    __syncthreads();
  }
  if (tid == 0) p.plan[p.B] = SeqPlan{carry[0], carry[1], carry[2], 0, 0, -1, 0};
}

// The sequence whose units hold unit u (kCol: columns units).
template <bool kCol>
__device__ __forceinline__ int find_seq(const ScoreParams& p, int64_t u) {
  int lo = 0, hi = p.B;  // plan[lo] <= u < plan[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    const int64_t at = kCol ? p.plan[mid].col_unit : p.plan[mid].stat_unit;
    if (at <= u)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// E of a lane's consecutive elements of a row, as fp32.
template <typename T, int E>
__device__ __forceinline__ void load_row(const T* p, float (&x)[E]) {
#pragma unroll
  for (int i = 0; i < E; ++i) x[i] = (float)p[i];
}

// Logits (times scale * log2 e) of a row group against one key: lane l
// returns the logit of row l >> 2 (kRowGroup == 8 rows, 4 lanes each).
template <int E>
__device__ __forceinline__ float group_dot(const float (&k)[E], const float (&q)[kRowGroup][E], int lane) {
  float a[kRowGroup];
#pragma unroll
  for (int r = 0; r < kRowGroup; ++r) {
    a[r] = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) a[r] = fmaf(k[i], q[r][i], a[r]);
  }
#pragma unroll
  for (int lvl = 0; lvl < 3; ++lvl) {
    const int off = 16 >> lvl, half = kRowGroup >> (lvl + 1);
    const bool up = lane & off;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float send = up ? a[i] : a[i + half];
      const float keep = up ? a[i + half] : a[i];
      a[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
    }
  }
  float x = a[0];
  x += __shfl_xor_sync(0xffffffffu, x, 2);
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x;
}

template <typename TQ, typename TK, int D>
struct Tile {
  static constexpr int E = D / 32;
  // Row group rg of kv head h: the lane's slice of each of its rows' q
  // (rows past the end: zeros).
  __device__ static void load_q(const ScoreParams& p, int qstart, int rows, int h, int rg, int lane,
                                float (&q)[kRowGroup][E]) {
#pragma unroll
    for (int r = 0; r < kRowGroup; ++r) {
      const int row = rg * kRowGroup + r;
      if (row < rows) {
        const int i = row / p.G, g = row - i * p.G;
        const TQ* src = static_cast<const TQ*>(p.q) + ((int64_t)(qstart + i) * p.Hq + h * p.G + g) * D + lane * E;
        load_row<TQ, E>(src, q[r]);
      } else {
#pragma unroll
        for (int j = 0; j < E; ++j) q[r][j] = 0.f;
      }
    }
  }
  // The lane's slice of key j of kv head h (a block outside the pool: zeros).
  __device__ static void load_k(const ScoreParams& p, const int32_t* bt, int j, int h, int lane, float (&k)[E]) {
    const int b = bt[j / p.bs];
    if (b >= 0 && b < p.num_blocks) {
      const TK* src =
          static_cast<const TK*>(p.kc) + (((int64_t)b * p.bs + j % p.bs) * p.Hkv + h) * D + lane * E;
      load_row<TK, E>(src, k);
    } else {
      raise_error(p.err, PKV_DEVERR_BLOCK_OUT_OF_RANGE);
#pragma unroll
      for (int i = 0; i < E; ++i) k[i] = 0.f;
    }
  }
};

template <typename TQ, typename TK, int D>
__global__ void __launch_bounds__(kThreads) stats_kernel(const ScoreParams p) {
  using X = Tile<TQ, TK, D>;
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
  const int64_t total = p.plan[p.B].stat_unit;
  for (int64_t u = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5; u < total; u += warps) {
    const int s = find_seq<false>(p, u);
    const SeqPlan sp = p.plan[s];
    const int rows = sp.n * p.G, groups = (rows + kRowGroup - 1) / kRowGroup;
    int64_t v = u - sp.stat_unit;
    const int c = (int)(v % sp.chunks);
    v /= sp.chunks;
    const int rg = (int)(v % groups), h = (int)(v / groups);
    float q[kRowGroup][X::E];
    X::load_q(p, p.qsl[s], rows, h, rg, lane, q);
    const int32_t* bt = p.tables + (int64_t)s * p.max_blocks;
    const int row = rg * kRowGroup + (lane >> 2);
    const int vis = row >= rows ? 0 : p.causal ? sp.L - sp.n + row / p.G + 1 : sp.L;
    const int ke = min(sp.L, (c + 1) * kChunk);
    float m = -CUDART_INF_F, l = 0.f;
    for (int j = c * kChunk; j < ke; ++j) {
      float k[X::E];
      X::load_k(p, bt, j, h, lane, k);
      const float z = group_dot<X::E>(k, q, lane) * p.scale_log2;
      if (j < vis) {
        const float mn = fmaxf(m, z);
        l = l * fast_exp2(m - mn) + fast_exp2(z - mn);
        m = mn;
      }
    }
    if (row < rows && (lane & 3) == 0) p.part[sp.part + ((int64_t)h * rows + row) * sp.chunks + c] = make_float2(m, l);
  }
}

// lse of each row (one warp a row).
__global__ void __launch_bounds__(kThreads) lse_kernel(const ScoreParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
  for (int64_t w = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5; w < p.T * p.Hq; w += warps) {
    const int t = (int)(w / p.Hq), hq = (int)(w - (int64_t)t * p.Hq);
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.qsl[mid] <= t)
        lo = mid;
      else
        hi = mid;
    }
    const SeqPlan sp = p.plan[lo];
    const int i = t - p.qsl[lo];
    if (i < 0 || i >= sp.n) continue;
    const int rows = sp.n * p.G, h = hq / p.G, row = i * p.G + (hq - h * p.G);
    const float2* part = p.part + sp.part + ((int64_t)h * rows + row) * sp.chunks;
    float m = -CUDART_INF_F, l = 0.f;
    for (int c = lane; c < sp.chunks; c += 32) m = fmaxf(m, part[c].x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    for (int c = lane; c < sp.chunks; c += 32) l += part[c].y * fast_exp2(part[c].x - m);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    if (lane == 0) p.lse[w] = m + log2f(l);
  }
}

template <typename TQ, typename TK, int D>
__global__ void __launch_bounds__(kThreads) columns_kernel(const ScoreParams p) {
  using X = Tile<TQ, TK, D>;
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
  const int64_t total = p.plan[p.B].col_unit;
  for (int64_t u = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5; u < total; u += warps) {
    const int s = find_seq<true>(p, u);
    const SeqPlan sp = p.plan[s];
    const int rows = sp.n * p.G, groups = (rows + kRowGroup - 1) / kRowGroup;
    const int64_t v = u - sp.col_unit;
    const int c = (int)(v % sp.chunks), h = (int)(v / sp.chunks);
    const int32_t* bt = p.tables + (int64_t)s * p.max_blocks;
    const int qstart = p.qsl[s];
    for (int j0 = c * kChunk; j0 < min(sp.L, (c + 1) * kChunk); j0 += 32) {
      const int nk = min(32, sp.L - j0);
      float paid = 0.f;  // of key j0 + lane
      for (int rg = 0; rg < groups; ++rg) {
        float q[kRowGroup][X::E];
        X::load_q(p, qstart, rows, h, rg, lane, q);
        const int row = rg * kRowGroup + (lane >> 2);
        const int i = row / p.G;
        const int vis = row >= rows ? 0 : p.causal ? sp.L - sp.n + i + 1 : sp.L;
        const float lse = row < rows ? p.lse[(int64_t)(qstart + i) * p.Hq + h * p.G + (row - i * p.G)] : 0.f;
        for (int j = 0; j < nk; ++j) {
          float k[X::E];
          X::load_k(p, bt, j0 + j, h, lane, k);
          const float z = group_dot<X::E>(k, q, lane) * p.scale_log2;
          float w = j0 + j < vis ? fast_exp2(z - lse) : 0.f;
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) w += __shfl_xor_sync(0xffffffffu, w, d);
          if (lane == j) paid += w;
        }
      }
      const int j = j0 + lane;
      if (j < sp.L) {
        const int64_t at = ((int64_t)sp.row * p.Hkv + h) * p.max_len + j;
        if (j < sp.L - sp.n && p.decay != 0.f) paid = fmaf(p.decay, p.scores[at], paid);
        p.out[at] = paid;
      }
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
  size_t plan, lse, part, total;
};

Layout layout(int64_t B, int64_t T, int64_t Hq, int64_t keys) {
  Layout l{};
  const size_t chunks = (size_t)((keys + kChunk - 1) / kChunk);
  l.plan = 0;
  l.lse = align_up((size_t)(B + 1) * sizeof(SeqPlan));
  l.part = align_up(l.lse + (size_t)(T * Hq) * sizeof(float));
  l.total = align_up(l.part + (size_t)(T * Hq) * chunks * sizeof(float2));
  return l;
}

template <typename TQ, typename TK, int D>
void launch(const ScoreParams& p, int sms, cudaStream_t s) {
  const int grid = sms * 8;
  stats_kernel<TQ, TK, D><<<grid, kThreads, 0, s>>>(p);
  lse_kernel<<<grid, kThreads, 0, s>>>(p);
  columns_kernel<TQ, TK, D><<<grid, kThreads, 0, s>>>(p);
}

pkv_status scores_impl(ScoreParams p, int D, bool f8, float k_scale, float scale, void* workspace, size_t ws_bytes,
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
  if (f8 && (!(k_scale > 0.f) || !isfinite(k_scale)))
    return fail(PKV_ERR_INVALID_ARG, "k_scale must be positive and finite");
  if ((int64_t)p.max_blocks * p.bs > (int64_t)1 << 30 || p.max_len > 1 << 30)
    return fail(PKV_ERR_UNSUPPORTED, "context too long");
  if (p.T > ((int64_t)1 << 31) / ((int64_t)p.Hq * D)) return fail(PKV_ERR_UNSUPPORTED, "num_tokens too large");
  if (p.B == 0 || p.T == 0) return PKV_OK;
  if (!p.q || !p.kc || !p.tables || !p.lens || !p.qsl || !p.scores || !p.out)
    return fail(PKV_ERR_INVALID_ARG, "null pointer");
  auto bits = [](const void* x) { return reinterpret_cast<uintptr_t>(x); };
  if ((bits(p.q) | bits(p.kc)) & 15u) return fail(PKV_ERR_INVALID_ARG, "q and the cache must be 16-byte aligned");
  if (!workspace || (bits(workspace) & (kAlign - 1)))
    return fail(PKV_ERR_WORKSPACE, "workspace missing or not 256-byte aligned");
  const Layout lay = layout(p.B, p.T, p.Hq, std::min<int64_t>(p.max_len, (int64_t)p.max_blocks * p.bs));
  if (ws_bytes < lay.total) return fail(PKV_ERR_WORKSPACE, "workspace smaller than required");
  int sms = 0;
  const pkv_status st = device_state(&sms, &p.err);
  if (st != PKV_OK) return st;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.plan = reinterpret_cast<SeqPlan*>(ws + lay.plan);
  p.lse = reinterpret_cast<float*>(ws + lay.lse);
  p.part = reinterpret_cast<float2*>(ws + lay.part);
  p.scale_log2 = (f8 ? scale * k_scale : scale) * 1.4426950408889634f;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  plan_scores_kernel<<<1, 1024, 0, s>>>(p);
  if (f8)
    launch<__nv_bfloat16, __nv_fp8_e4m3, 128>(p, sms, s);
  else if (dtype == PKV_DTYPE_BF16)
    D == 128 ? launch<__nv_bfloat16, __nv_bfloat16, 128>(p, sms, s) : launch<__nv_bfloat16, __nv_bfloat16, 64>(p, sms, s);
  else
    D == 128 ? launch<float, float, 128>(p, sms, s) : launch<float, float, 64>(p, sms, s);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_error(e, "paged_attention_scores launch");
  return PKV_OK;
}

}  // namespace
}  // namespace pkv

extern "C" {

size_t paged_attention_scores_workspace_size(int32_t num_seqs, int64_t num_tokens, int32_t num_q_heads,
                                             int32_t num_kv_heads, int64_t max_context) {
  if (num_seqs < 0 || num_tokens < 0 || num_kv_heads <= 0 || num_q_heads <= 0 || max_context < 0) return 0;
  return pkv::layout(num_seqs, num_tokens, num_q_heads, max_context).total;
}

size_t paged_attention_scores_workspace_min(int32_t num_seqs, int64_t num_tokens, int32_t num_q_heads,
                                            int32_t num_kv_heads, int64_t max_context) {
  return paged_attention_scores_workspace_size(num_seqs, num_tokens, num_q_heads, num_kv_heads, max_context);
}

pkv_status paged_attention_scores(const void* q, const void* k_cache, const int32_t* block_tables,
                                  const int32_t* context_lens, const int32_t* query_start_loc,
                                  const int32_t* score_rows, const float* scores, float* scores_out,
                                  int32_t num_seqs, int64_t num_tokens, int32_t num_q_heads, int32_t num_kv_heads,
                                  int32_t head_dim, int64_t num_blocks, int32_t block_size,
                                  int32_t max_blocks_per_seq, int32_t num_rows, int32_t max_len,
                                  int32_t max_query_len, float scale, int32_t causal, float decay, void* workspace,
                                  size_t workspace_bytes, pkv_dtype dtype, void* stream) {
  (void)max_query_len;
  pkv::ScoreParams p{q, k_cache, block_tables, context_lens, query_start_loc, score_rows, scores, scores_out,
                     nullptr, nullptr, nullptr, num_tokens, num_blocks, num_seqs, num_q_heads, num_kv_heads, 0,
                     block_size, max_blocks_per_seq, num_rows, max_len, causal ? 1 : 0, 0.f, decay, nullptr};
  return pkv::scores_impl(p, head_dim, false, 1.f, scale, workspace, workspace_bytes, dtype, stream);
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
  (void)max_query_len;
  pkv::ScoreParams p{q, k_cache, block_tables, context_lens, query_start_loc, score_rows, scores, scores_out,
                     nullptr, nullptr, nullptr, num_tokens, num_blocks, num_seqs, num_q_heads, num_kv_heads, 0,
                     block_size, max_blocks_per_seq, num_rows, max_len, causal ? 1 : 0, 0.f, decay, nullptr};
  return pkv::scores_impl(p, head_dim, true, k_scale, scale, workspace, workspace_bytes, PKV_DTYPE_BF16, stream);
}

}  // extern "C"
