// Compaction of a paged KV cache to its kept tokens (paged_kv_compact,
// declared in paged_kv_budget.h).
//
// Kept token r of a (sequence, kv head) moves from position kept[r] to
// position r of the sequence's cache, in K, V and the running scores.  The
// positions ascend, so kept[r] >= r: in place, a row's new position is never
// the old position of a LATER kept row, and the only hazard is to overwrite
// position r before the earlier row that lives there has been read.  So one
// block walks the rows of its (sequence, head, slice) in order, a round of
// them at a time: load the round into registers, barrier, store it.  Loads of
// later rounds may run ahead of the stores freely.
//
// The rows of one head are independent of the other heads', K of V, and
// every 16-byte column slice of the others: the grid is
// (sequences x heads) x (K slices + V slices + scores).
//
// HBM-bound: every kept row is read and written once; rows that stay where
// they are (the kept prefix) are neither read nor written.
#include <cuda_runtime.h>
#include <stdint.h>

#include "paged_kv_budget.h"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 4;  // 16-byte vectors a thread holds per round

struct CompactParams {
  uint8_t* kc;
  uint8_t* vc;
  const int32_t* tables;
  const int32_t* dst_tables;
  const int32_t* kept;
  const int32_t* rows;
  float* scores;
  int64_t num_blocks;
  int Hkv, bs, max_blocks, budget, num_rows, max_len;
  int row_bytes;     // head_dim * element size
  int slice_vecs;    // 16-byte vectors of a column slice
  int slices;        // column slices of a row
  int* err;
};

__global__ void __launch_bounds__(kThreads) compact_kernel(const CompactParams p) {
  const int per = 2 * p.slices + (p.scores ? 1 : 0);
  const int sh = blockIdx.x / per, part = blockIdx.x - sh * per;
  const int s = sh / p.Hkv, h = sh - s * p.Hkv;
  const int32_t* kept = p.kept + (int64_t)sh * p.budget;
  bool bad_block = false, bad_order = false;

  if (part == 2 * p.slices) {  // the running scores
    const int row = p.rows ? p.rows[s] : s;
    if (row < 0 || row >= p.num_rows) {
      if (row >= 0 && threadIdx.x == 0) raise_error(p.err, PKV_DEVERR_BAD_SEQUENCE);
      return;
    }
    float* sc = p.scores + ((int64_t)row * p.Hkv + h) * p.max_len;
    for (int base = 0; base < p.budget && kept[base] >= 0; base += kThreads * kVecs) {
      float x[kVecs];
      bool live[kVecs];
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        const int r = base + i * kThreads + threadIdx.x;
        const int src = r < p.budget ? kept[r] : -1;
        live[i] = src >= 0 && r < p.max_len && src != r;
        x[i] = 0.f;
        if (live[i]) {
          if (src < p.max_len)
            x[i] = sc[src];
          else
            bad_block = true;
        }
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
        if (live[i]) sc[base + i * kThreads + threadIdx.x] = x[i];
    }
    if (bad_block) raise_error(p.err, PKV_DEVERR_BLOCK_OUT_OF_RANGE);
    return;
  }

  uint8_t* pool = part < p.slices ? p.kc : p.vc;
  const int slice = part < p.slices ? part : part - p.slices;
  const int32_t* bt = p.tables + (int64_t)s * p.max_blocks;
  const int32_t* dt = (p.dst_tables ? p.dst_tables : p.tables) + (int64_t)s * p.max_blocks;
  const int rpr = kThreads / p.slice_vecs;  // rows per pass of the block
  const int my_row = threadIdx.x / p.slice_vecs, my_vec = threadIdx.x - my_row * p.slice_vecs;
  const bool idle = my_row >= rpr;
  const int64_t col = (int64_t)h * p.row_bytes + (slice * p.slice_vecs + my_vec) * 16;
  const bool in_row = (slice * p.slice_vecs + my_vec) * 16 < p.row_bytes;
  const int64_t token_bytes = (int64_t)p.Hkv * p.row_bytes;
  for (int base = 0; base < p.budget && kept[base] >= 0; base += rpr * kVecs) {
    int4 x[kVecs];
    uint8_t* to[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int r = base + i * rpr + my_row;
      const int src = !idle && in_row && r < p.budget ? kept[r] : -1;
      x[i] = make_int4(0, 0, 0, 0);
      to[i] = nullptr;
      if (src >= 0) {
        if (r > 0 && kept[r - 1] >= src) bad_order = true;
        const int sb = src / p.bs, db = r / p.bs;
        const int64_t sblk = sb < p.max_blocks ? bt[sb] : -1;
        const int64_t dblk = db < p.max_blocks ? dt[db] : -1;
        const bool s_ok = sblk >= 0 && sblk < p.num_blocks, d_ok = dblk >= 0 && dblk < p.num_blocks;
        bad_block |= !s_ok || !d_ok;
        uint8_t* from = pool + (sblk * p.bs + (src - sb * p.bs)) * token_bytes + col;
        uint8_t* dst = pool + (dblk * p.bs + (r - db * p.bs)) * token_bytes + col;
        if (d_ok && !(s_ok && from == dst)) {
          to[i] = dst;
          if (s_ok) x[i] = *reinterpret_cast<const int4*>(from);
        }
      }
    }
    __syncthreads();  // every row of this round is read
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      if (to[i]) *reinterpret_cast<int4*>(to[i]) = x[i];
  }
  if (bad_block) raise_error(p.err, PKV_DEVERR_BLOCK_OUT_OF_RANGE);
  if (bad_order) raise_error(p.err, PKV_DEVERR_BAD_SEQUENCE);
}

pkv_status fail(pkv_status st, const char* msg) {
  set_last_error(msg);
  return st;
}

}  // namespace
}  // namespace pkv

extern "C" pkv_status paged_kv_compact(void* k_cache, void* v_cache, const int32_t* block_tables,
                                       const int32_t* dst_block_tables, const int32_t* kept,
                                       const int32_t* score_rows, float* scores, int32_t num_seqs,
                                       int32_t num_kv_heads, int32_t head_dim, int64_t num_blocks,
                                       int32_t block_size, int32_t max_blocks_per_seq, int32_t budget,
                                       int32_t num_rows, int32_t max_len, pkv_dtype dtype, void* stream) {
  using namespace pkv;
  set_last_error("");
  if (dtype != PKV_DTYPE_BF16 && dtype != PKV_DTYPE_F32 && dtype != PKV_DTYPE_FP8_E4M3)
    return fail(PKV_ERR_UNSUPPORTED, "dtype");
  if (num_seqs < 0 || num_kv_heads <= 0 || head_dim <= 0 || num_blocks <= 0 || block_size <= 0 ||
      max_blocks_per_seq <= 0 || budget <= 0)
    return fail(PKV_ERR_INVALID_ARG, "sizes must be positive (num_seqs >= 0)");
  if (scores && (num_rows <= 0 || max_len <= 0)) return fail(PKV_ERR_INVALID_ARG, "scores without rows or length");
  const int es = dtype == PKV_DTYPE_BF16 ? 2 : dtype == PKV_DTYPE_F32 ? 4 : 1;
  const int64_t row_bytes = (int64_t)head_dim * es;
  if (row_bytes % 16 != 0) return fail(PKV_ERR_UNSUPPORTED, "head_dim * element size not a multiple of 16");
  if (row_bytes > 4096) return fail(PKV_ERR_UNSUPPORTED, "head_dim * element size above 4096");
  if (num_kv_heads > 1 << 16) return fail(PKV_ERR_UNSUPPORTED, "num_kv_heads too large");
  if (num_seqs > kMaxPlanSeqs) return fail(PKV_ERR_UNSUPPORTED, "too many sequences per call");
  if (num_blocks > ((int64_t)1 << 31) - 1) return fail(PKV_ERR_UNSUPPORTED, "num_blocks exceeds int32");
  if ((int64_t)max_blocks_per_seq * block_size > (int64_t)1 << 30 || budget > 1 << 30)
    return fail(PKV_ERR_UNSUPPORTED, "context too long");
  if (num_seqs == 0) return PKV_OK;
  if (!k_cache || !v_cache || !block_tables || !kept) return fail(PKV_ERR_INVALID_ARG, "null pointer");
  if ((reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache)) & 15u)
    return fail(PKV_ERR_INVALID_ARG, "caches must be 16-byte aligned");
  CompactParams p{};
  int sms = 0;
  const pkv_status st = device_state(&sms, &p.err);
  if (st != PKV_OK) return st;
  p.kc = static_cast<uint8_t*>(k_cache);
  p.vc = static_cast<uint8_t*>(v_cache);
  p.tables = block_tables;
  p.dst_tables = dst_block_tables;
  p.kept = kept;
  p.rows = score_rows;
  p.scores = scores;
  p.num_blocks = num_blocks;
  p.Hkv = num_kv_heads;
  p.bs = block_size;
  p.max_blocks = max_blocks_per_seq;
  p.budget = budget;
  p.num_rows = num_rows;
  p.max_len = max_len;
  p.row_bytes = (int)row_bytes;
  p.slices = 1;
  p.slice_vecs = (int)(row_bytes / 16);
  const int64_t grid = (int64_t)num_seqs * num_kv_heads * (2 * p.slices + (scores ? 1 : 0));
  if (grid > ((int64_t)1 << 31) - 1) return fail(PKV_ERR_UNSUPPORTED, "too many sequences and heads");
  compact_kernel<<<(unsigned)grid, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_error(e, "paged_kv_compact launch");
  return PKV_OK;
}
