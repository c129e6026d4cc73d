// Compaction of a paged KV cache to its kept tokens (paged_kv_compact,
// declared in paged_kv_budget.h).
//
// Kept token r of a (sequence, kv head) moves from position kept[r] to
// position r of the sequence's cache, in K, V and the running scores.  The
// positions ascend, so kept[r] >= r: in place, a row's new position is never
// the old position of a LATER kept row, and the only hazard is to overwrite
// position r before the earlier row that lives there has been read.  So the
// rows are walked in order, a round of them at a time, loads ahead of stores;
// and before the stores of a round, which reach up to position y, the rounds
// that hold a row from below y must have been loaded by everyone.  Which round
// that is, is known from the kept positions; a barrier is passed only when
// the last one did not cover it.  With an eighth of the tokens kept, a round's
// rows come from eight times as far, and few barriers are left (one a round
// instead: 73 us for 4 sequences of 131072 tokens in FP8, 64 us this way).
//
// The heads' rows are independent of each other, and the scores of the rows: a
// (sequence, head)'s rows, K and V together (one address computation), are
// one cluster's work and its scores another's.  With few of those a cluster
// has several blocks, which share each round (a block its rows in order, the
// blocks in order) and pass cluster barriers.
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

constexpr int kMaxThreads = 256;
constexpr int kVecs = 4;  // 16-byte vectors of one K and one V row (scores: values) a thread holds per round

struct CompactParams {
  uint8_t* kc;
  uint8_t* vc;
  const int32_t* tables;
  const int32_t* dst_tables;
  const int32_t* kept;
  const int32_t* rows;
  float* scores;
  int64_t num_blocks;
  int Hkv, bs, bs_log, max_blocks, budget, num_rows, max_len;  // bs_log < 0: not a power of two
  int row_bytes;  // head_dim * element size
  int cluster;    // blocks of a cluster
  int pairs;      // (sequence, head)s
  int* err;
};

// Threads that share a row of `vecs` 16-byte vectors, at most kVecs each.
__host__ __device__ constexpr int row_team(int vecs) { return (vecs + kVecs - 1) / kVecs; }

// Every thread of the cluster has performed its loads so far; stores of any
// of them may follow.
__device__ __forceinline__ void load_barrier(int cluster) {
  if (cluster > 1)
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  else
    __syncthreads();
}

// What a thread moves: Mover::Slot holds its part of `kTokens` kept tokens on
// their way.  locate() looks up where token i of them (kept token r, from
// position src; src < 0: none) comes from and goes to, load() starts it,
// store() ends it; each is done a round ahead of the next, so that none waits
// for the reads of the one before.
//
// Rows: up to four 16-byte vectors of one token's K and V rows each, `apart`
// bytes from one another so that the threads of a row read whole sectors side
// by side.
struct RowMover {
  static constexpr int kTokens = 1;
  struct Slot {
    int4 k[kVecs], v[kVecs];
    int64_t to;  // byte offset in the pools; < 0: nothing to store
  };
  uint8_t* kc;
  uint8_t* vc;
  const int32_t* bt;
  const int32_t* dt;
  int64_t col, token_bytes, num_blocks;
  int bs, bs_log, max_blocks, apart, vecs;
  bool bad;

  struct Place {
    int src, r, sblk, dblk;
  };
  __device__ __forceinline__ void locate(Place& l, int, int r, int src) {
    l.src = src;
    if (src < 0) return;
    l.r = r;
    const int sb = bs_log >= 0 ? src >> bs_log : src / bs, db = bs_log >= 0 ? r >> bs_log : r / bs;
    l.sblk = sb < max_blocks ? __ldg(bt + sb) : -1;
    l.dblk = db < max_blocks ? __ldg(dt + db) : -1;
  }
  __device__ __forceinline__ void load(Slot& v, const Place& l) {
    v.to = -1;
    if (l.src < 0) return;
    const int so = bs_log >= 0 ? l.src & (bs - 1) : l.src % bs, dof = bs_log >= 0 ? l.r & (bs - 1) : l.r % bs;
    const bool s_ok = l.sblk >= 0 && l.sblk < num_blocks, d_ok = l.dblk >= 0 && l.dblk < num_blocks;
    bad |= !s_ok || !d_ok;
    const int64_t from = ((int64_t)l.sblk * bs + so) * token_bytes + col;
    const int64_t dst = ((int64_t)l.dblk * bs + dof) * token_bytes + col;
    if (d_ok && !(s_ok && from == dst)) {
      v.to = dst;
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        v.k[i] = v.v[i] = make_int4(0, 0, 0, 0);
        if (s_ok && i < vecs) {
          v.k[i] = *reinterpret_cast<const int4*>(kc + from + i * apart);
          v.v[i] = *reinterpret_cast<const int4*>(vc + from + i * apart);
        }
      }
    }
  }
  __device__ __forceinline__ void store(const Slot& v) {
    if (v.to < 0) return;
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      if (i < vecs) {
        *reinterpret_cast<int4*>(kc + v.to + i * apart) = v.k[i];
        *reinterpret_cast<int4*>(vc + v.to + i * apart) = v.v[i];
      }
  }
};

struct ScoreMover {
  static constexpr int kTokens = kVecs;
  struct Slot {
    float x[kVecs];
    int to[kVecs];  // < 0: nothing to store
  };
  float* sc;
  int max_len;
  bool bad;

  struct Place {
    int src[kVecs], r[kVecs];
  };
  __device__ __forceinline__ void locate(Place& l, int i, int r, int src) {
    l.src[i] = src;
    l.r[i] = r;
  }
  __device__ __forceinline__ void load(Slot& v, const Place& l) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      v.to[i] = -1;
      if (l.src[i] < 0) continue;
      const bool past = l.src[i] >= max_len;
      bad |= past;
      if (l.src[i] == l.r[i] || l.r[i] >= max_len) continue;
      v.to[i] = l.r[i];
      v.x[i] = past ? 0.f : sc[l.src[i]];
    }
  }
  __device__ __forceinline__ void store(const Slot& v) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      if (v.to[i] >= 0) sc[v.to[i]] = v.x[i];
  }
};

// The rounds of one (sequence, head)'s rows or scores.  A round is `per` tokens for each
// block of the cluster; this thread moves tokens base + i * lanes + mine of
// its block's (mine < 0: it moves none, but keeps the barriers).
template <typename Mover>
__device__ __forceinline__ bool move_rounds(Mover& m, const int32_t* kept, int budget, int cluster, int block, int lanes,
                                            int mine) {
  typedef typename Mover::Slot Slot;
  constexpr int N = Mover::kTokens;
  const int per = lanes * N, round = per * cluster;
  bool bad_order = false;
  auto positions = [&](int base, int (&src)[N]) {  // of the round at base; -1 past the kept ones
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int r = base + block * per + i * lanes + mine;
      src[i] = mine >= 0 && r < budget ? __ldg(kept + r) : -1;
      if (src[i] >= 0 && r > 0 && __ldg(kept + r - 1) >= src[i]) bad_order = true;
    }
  };
  auto locate = [&](int base, const int (&src)[N], typename Mover::Place& l) {
#pragma unroll
    for (int i = 0; i < N; ++i) m.locate(l, i, base + block * per + i * lanes + mine, src[i]);
  };
  // every thread of the cluster sees the same rounds: the kept ones end at the first -1
  int src[N];
  typename Mover::Place place;
  Slot now, next;
  if (__ldg(kept) < 0) return false;
  positions(0, src);
  locate(0, src, place);
  positions(round, src);
  m.load(now, place);
  locate(round, src, place);
  positions(2 * round, src);
  int needed = 0;    // the last round that holds a row from below where this one's stores reach
  int covered = -1;  // the last round whose loads a barrier has covered
  int k = 0, base = 0;
  // round k, held in `cur`: the next one's loads, the barrier if it is needed,
  // the stores.  The two slots change places by unrolling: copying one to the
  // other would wait for the loads that are under way.
  auto turn = [&](Slot& cur, Slot& other) {
    const bool more = base + round < budget && __ldg(kept + base + round) >= 0;
    if (more) {
      m.load(other, place);
      locate(base + 2 * round, src, place);
      positions(base + 3 * round, src);
    }
    while (needed < k && __ldg(kept + (needed + 1) * round) < base + round) ++needed;
    if (needed > covered) {
      load_barrier(cluster);
      covered = k + (more ? 1 : 0);
    }
    m.store(cur);
    ++k;
    base += round;
    return more;
  };
  while (turn(now, next) && turn(next, now)) {
  }
  return bad_order;
}

__global__ void __launch_bounds__(kMaxThreads, 2) compact_kernel(const CompactParams p) {
  const int block = p.cluster == 1 ? 0 : blockIdx.x % p.cluster;
  const int work = p.cluster == 1 ? blockIdx.x : blockIdx.x / p.cluster;
  const int threads = blockDim.x;
  // the rows' clusters first: taking turns with the scores' short ones, a part of
  // them was left for a second wave of blocks (the long FP8 case: 72 us, not 64)
  const bool rows = work < p.pairs;
  const int sh = rows ? work : work - p.pairs;
  const int s = sh / p.Hkv, h = sh - s * p.Hkv;
  const int32_t* kept = p.kept + (int64_t)sh * p.budget;
  if (!rows) {  // the running scores
    const int row = p.rows ? p.rows[s] : s;
    if (row < 0 || row >= p.num_rows) {
      if (row >= 0 && threadIdx.x == 0) raise_error(p.err, PKV_DEVERR_BAD_SEQUENCE);
      return;
    }
    ScoreMover m{p.scores + ((int64_t)row * p.Hkv + h) * p.max_len, p.max_len, false};
    move_rounds(m, kept, p.budget, p.cluster, block, threads, threadIdx.x);
    if (m.bad) raise_error(p.err, PKV_DEVERR_BLOCK_OUT_OF_RANGE);
    return;
  }
  const int vecs = p.row_bytes / 16, team = row_team(vecs), lanes = threads / team;
  const int mine = threadIdx.x / team, member = threadIdx.x - mine * team;
  const int32_t* bt = p.tables + (int64_t)s * p.max_blocks;
  RowMover m{p.kc,
             p.vc,
             bt,
             p.dst_tables ? p.dst_tables + (int64_t)s * p.max_blocks : bt,
             (int64_t)h * p.row_bytes + member * 16,
             (int64_t)p.Hkv * p.row_bytes,
             p.num_blocks,
             p.bs,
             p.bs_log,
             p.max_blocks,
             team * 16,
             (vecs - member + team - 1) / team,
             false};
  const bool bad_order = move_rounds(m, kept, p.budget, p.cluster, block, lanes, mine < lanes ? mine : -1);
  if (m.bad) raise_error(p.err, PKV_DEVERR_BLOCK_OUT_OF_RANGE);
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
  p.bs_log = -1;
  for (int k = 0; k < 31; ++k)
    if (block_size == 1 << k) p.bs_log = k;
  p.max_blocks = max_blocks_per_seq;
  p.budget = budget;
  p.num_rows = num_rows;
  p.max_len = max_len;
  p.row_bytes = (int)row_bytes;
  // Enough (sequence, head)s: one block of 128 threads each, so that about as
  // many are resident as there are (64 x 8 rows of 512 kept tokens).  Few: up
  // to 8 blocks of 256 threads, while each has rounds to share.
  const int64_t pairs = (int64_t)num_seqs * num_kv_heads, units = pairs * (scores ? 2 : 1);
  const int team = row_team((int)(row_bytes / 16));
  int threads = 128, cluster = 1;
  if (pairs < 2 * sms || team > threads) threads = 256;
  while (cluster < 8 && pairs * cluster < 2 * sms && cluster * 2 * (threads / team) <= budget) cluster *= 2;
  p.cluster = cluster;
  p.pairs = (int)pairs;
  if (units * cluster > ((int64_t)1 << 31) - 1) return fail(PKV_ERR_UNSUPPORTED, "too many sequences and heads");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * cluster));
  cfg.blockDim = dim3(threads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, compact_kernel, p);
  if (e != cudaSuccess) return cuda_error(e, "paged_kv_compact launch");
  return PKV_OK;
}
