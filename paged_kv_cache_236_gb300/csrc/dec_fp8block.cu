// Attention of few rows per kv head (decode, short verify windows) over pools of
// E4M3 codes with a scale for each block and kv head: tcgen05.mma on the codes
// themselves (paged_attention_forward_fp8block).
//
// With codes ck, cv and block scales sk, sv, for rows r of one kv head:
//   x[r][j] = scale log2(e) (q_r . ck_j) sk(j)          (log2 units)
//   out_r   = sum_j 2^(x - m) sv(j) cv_j / sum_j 2^(x - m)
//
// The tensor cores multiply 8-bit operands at twice the 16-bit rate, but the
// point here is that the pools' tiles are operands as they land: converted to
// 16 bits first, as the kernel for pools of one scale does, a tile's chain
// of loads, conversion and MMAs sets the pace, at a third of the HBM rate.  So
// the other operand is split into 8-bit terms instead, which cost columns of
// an MMA whose columns are mostly unused anyway:
//   q    = 2^e (q1 + q2), E4M3 each, with e from the row's largest |q|, which
//          becomes 2^7 to 2^8: 8 significant bits, bf16's own, but for what is
//          below 2^-10, half of E4M3's least step: 2^-17 of the largest value;
//   w    = 2^(x - m) sv 2^11 = w1 + w2 + w3, E5M2 each: the top bytes of an fp16
//          value and of what is left of it, twice; 9 bits, down to 2^-16 (a
//          row's largest w is 2^11 to 2^15: E4M3's range would lose the many small
//          weights beside a large one).
// S^T [128 keys x 2 NR] = K [128 x 128 d] . [q1; q2]^T      (A K-major)
// O^T [128 d x 3 NR]   += V^T [128 d x 128 keys] . [w1; w2; w3]^T   (A MN-major)
// so a thread holds a key's logits (the sum of two columns), and a thread an
// output column (of three).  sk(j) multiplies a thread's logits; sv(j) moves
// its exponent, and the running reference m is one of x + log2 sv, so that w
// stays within its range whatever the blocks' scales are; the denominator takes
// w / (2^11 sv).
//
// Roles (416 threads, one CTA per SM, persistent, items from an atomic counter
// in the planner's largest-first order), as in the bf16 kernel:
//   warp 0    K producer: per 128-key tile one {128 bytes, 1, block_size, 1} box
//             per block (128-byte swizzle), the tile's scales and metadata;
//   warp 11   V producer;
//   warps 1,12 issue the MMAs, S and P.V (warp 1 also allocates TMEM);
//   warps 2-5 softmax (thread = key = TMEM lane);
//   warps 6-9 epilogue (thread = output column = TMEM lane of O^T);
//   warp 10   item fetch, and the split of the item's q rows.
// HBM-bound where contexts are long: 4 x 131072 keys (1.07 GB of codes, 2 MB of
// scales) 207 us with the planner's 10, 5.5 TB/s while it streams; the decode batch (303 MB in
// short items) 76 us, of which the planner, the start and the last items' merges are
// a third.  A tile's softmax takes about as long as its bytes.
// Shared memory: 6 stages of K and V codes (192 KB).  TMEM: S^T and O^T
// double-buffered.  Waits are bounded, and end as in the bf16 kernel.
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <limits.h>
#include <math_constants.h>

#include "block_scales.cuh"
#include "dec_rows.cuh"
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_tc.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 416;
constexpr int kStages = 6;
constexpr int kKeys = kMmaTileKeys;       // 128 keys per tile
constexpr int kTileBytes = kKeys * 128;   // K or V codes: 16 KB
constexpr int kStageBytes = 2 * kTileBytes;
constexpr int kFetchLeadTiles = 4;        // the next item is fetched when this many tiles are left to load
constexpr float kRescaleThreshold = 4.0f;  // log2 units
constexpr int kWeightExp = 11;            // weights are 2^11 times their value, at most 2^15
constexpr int kMetaDone = 2, kMetaLast = 1, kMetaFirst = 4;
constexpr uint32_t kTmemCols = 256;

// N of the MMAs: q's and the weights' terms of NR rows
constexpr int round16(int x) { return (x + 15) / 16 * 16; }
template <int NR>
struct Lay {
  static constexpr int kNQ = round16(2 * NR), kNP = round16(3 * NR);
  static constexpr uint32_t kSCol = 0, kOCol = 64;  // buffer b at + b * kNQ, + b * kNP
  static constexpr int kQOff = kStages * kStageBytes;
  static constexpr int kPOff = kQOff + 2 * kNQ * 128;
  static constexpr int kMetaOff = kPOff + 2 * kNP * 128;
  static constexpr int kScaleOff = kMetaOff + kStages * 64;           // [stage][16] float4
  static constexpr int kRedOff = kScaleOff + kStages * 256;
  static constexpr int kSlotOff = kRedOff + 2 * 4 * NR * 4;
  static constexpr int kISlotOff = kSlotOff + 2 * 256;
  static constexpr int kQsOff = kISlotOff + 2 * 448;
  static constexpr int kBarOff = kQsOff + 2 * NR * 4;
  static constexpr int kNumBars = 3 * kStages + 6 + 8 + 4 + 4 + 1;
  static constexpr int kSmem = kBarOff + kNumBars * 8 + 16 + 1024;
  static constexpr uint32_t kIdescS = idesc_f8(128, kNQ, kE4m3, kE4m3, false, false);
  static constexpr uint32_t kIdescO = idesc_f8(128, kNP, kE4m3, kE5m2, true, false);
  static_assert(2 * kNQ <= 64 && 64 + 2 * kNP <= (int)kTmemCols, "TMEM columns");
  static_assert(kSmem <= 232448, "shared memory per CTA");
};

struct alignas(16) Meta {
  int item, kbase, flags, seq;
  int kvh, row0, nrows, ke;
  int part, grp, L, n;
  int qstart, qbuf, pad1, pad2;
};
static_assert(sizeof(Meta) == 64, "meta slot");

struct Bars {
  // kv_empty[st] is the P.V of the stage's tile done: its codes and its P read
  uint64_t k_full[kStages], v_full[kStages], kv_empty[kStages];
  uint64_t s_full[2], s_free[2], p_full[2];
  uint64_t o_full[2], o_empty[2], ml_full[2], ml_empty[2];
  uint64_t islot_full[2], islot_free[2];
  uint64_t q_full[2], q_empty[2];  // an item's q terms written; its last S issued and its row scales read
  uint64_t fetch_go;
};
static_assert(sizeof(Bars) == Lay<4>::kNumBars * 8, "barrier block");

// An item as the fetch warp hands it to the producers: L counts places, the
// keys without those from `at` on that a window leaves out (len of them).
struct alignas(16) ItemSlot {
  WorkItem it;
  int idx, L, qstart, n;
  int done, nblk, at, len;
  int phys[32];       // the first 32 blocks
  float2 scales[32];  // K's and V's of them
};
static_assert(sizeof(ItemSlot) == 448, "item slot");

struct alignas(16) EpSlot {
  Meta mt;
  float m[16], l[16];
  int done;
  int pad[15];
};
static_assert(sizeof(EpSlot) == 256, "epilogue slot");

template <int N>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&v)[N]) {
  if constexpr (N == 8) {
    tmem_ld8(taddr, v);
  } else if constexpr (N == 16) {
    tmem_ld16(taddr, v);
  } else if constexpr (N == 32) {
    tmem_ld32(taddr, v);
  } else if constexpr (N == 12) {
    tmem_ld8(taddr, v);
    tmem_ld4(taddr + 8, v + 8);
  } else if constexpr (N == 24) {
    tmem_ld16(taddr, v);
    tmem_ld8(taddr + 16, v + 16);
  } else {
    static_assert(N == 48, "columns");
    tmem_ld32(taddr, v);
    tmem_ld16(taddr + 32, v + 32);
  }
}
template <int N>
__device__ __forceinline__ void tmem_st_cols(uint32_t taddr, const uint32_t (&v)[N]) {
  if constexpr (N == 12) {
    tmem_st8(taddr, v);
    tmem_st4(taddr + 8, v + 8);
  } else if constexpr (N == 24) {
    tmem_st16(taddr, v);
    tmem_st8(taddr + 16, v + 16);
  } else {
    static_assert(N == 48, "columns");
    tmem_st32(taddr, v);
    tmem_st16(taddr + 32, v + 32);
  }
}

// NR: rows per item (4, 8 or 16)
template <int NR>
__global__ void __launch_bounds__(kThreads, 1) dec_fp8block_kernel(const AttnParams p,
                                                                   const __grid_constant__ CUtensorMap kmap,
                                                                   const __grid_constant__ CUtensorMap vmap) {
  using Y = Lay<NR>;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Bars* bars = reinterpret_cast<Bars*>(smem + Y::kBarOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Y::kBarOff + Y::kNumBars * 8);
  Meta* meta = reinterpret_cast<Meta*>(smem + Y::kMetaOff);
  Scales* tile_scales = reinterpret_cast<Scales*>(smem + Y::kScaleOff);  // [stage][16]
  float* red = reinterpret_cast<float*>(smem + Y::kRedOff);              // [2][4 warps][NR rows]
  float* row_scales = reinterpret_cast<float*>(smem + Y::kQsOff);        // [2][NR], times the logit scale
  ItemSlot* islots = reinterpret_cast<ItemSlot*>(smem + Y::kISlotOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WaitCtl wc{p.err, wait_limit(p.wait_ns)};

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->v_full[s], 1);
      mbar_init(&bars->kv_empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars->s_full[b], 1);
      mbar_init(&bars->s_free[b], 128);
      mbar_init(&bars->p_full[b], 128);
      mbar_init(&bars->o_full[b], 1);
      mbar_init(&bars->o_empty[b], 128);
      mbar_init(&bars->ml_full[b], 128);
      mbar_init(&bars->ml_empty[b], 128);
      mbar_init(&bars->islot_full[b], 32);
      mbar_init(&bars->islot_free[b], 2);  // both producers read the slot
      mbar_init(&bars->q_full[b], 32);
      mbar_init(&bars->q_empty[b], 1 + 4);  // the S issuer's commit, the four softmax warps
    }
    mbar_init(&bars->fetch_go, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // as in the bf16 kernel: beside the many-row kernel the plan is complete at launch
  if (!p.no_wait) pdl_wait();
  const int n_items = __ldcg(&p.header->n_dec);
  const uint32_t tmem = *tmem_slot;
  const uint32_t smem_base = smem_u32(smem);
  const int nb = kKeys / p.bs;  // blocks per tile

  // block of table row `bt` that holds the places from `place`; num_blocks (the box
  // reads as zeros) past the end and for ids out of range
  auto block_of = [&](const int32_t* bt, int nblk, int at, int len, int place) -> int {
    const int lb = (place < at ? place : place + len) / p.bs;
    if (lb >= nblk) return (int)p.num_blocks;
    const int b = __ldg(bt + lb);
    if (b >= 0 && (int64_t)b < p.num_blocks) return b;
    raise_error(p.err, PKV_DEVERR_BLOCK_OUT_OF_RANGE);
    return (int)p.num_blocks;
  };

  if (warp == 0 || warp == 11) {
    // ================================================================ K / V producers
    const bool vprod = warp == 11;
    if (lane == 0) prefetch_tensormap(vprod ? &vmap : &kmap);
    uint64_t* fullb = vprod ? bars->v_full : bars->k_full;
    int g = 0;
    // leaving: the copies of the tiles issued last land first, whoever still waits for them
    auto drain = [&]() {
      for (int j = max(0, g - kStages); j < g; ++j)
        __all_sync(0xffffffffu, mbar_wait(&fullb[j % kStages], (j / kStages) & 1, wc));
    };
    for (int c = 0;; ++c) {
      const int qb = c & 1;
      if (!wait_all(&bars->islot_full[qb], (c >> 1) & 1, wc)) {
        drain();
        break;
      }
      const ItemSlot& sl = islots[qb];
      const bool done = sl.done != 0;
      const WorkItem it = sl.it;
      const int idx = sl.idx, L = sl.L, qstart = sl.qstart, n = sl.n, nblk = sl.nblk, at = sl.at, len = sl.len;
      // Block ids and scales are held 32 at a time, a lane to a block: those of the
      // item's next 32 / nb tiles.  The next 32 are read while these are used, so that
      // no tile waits for a read of its own.
      int phys = sl.phys[lane];
      Scales sc = make_scales<kWeightExp>(sl.scales[lane]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->islot_free[qb]);
      if (done) {
        if (vprod) {
          drain();
          break;
        }
        const int st = g % kStages;
        if (!wait_all(&bars->kv_empty[st], ((g / kStages) & 1) ^ 1, wc)) {
          drain();
          break;
        }
        drain();  // (before the arrival below, another phase of a barrier waited for)
        if (lane == 0) {
          meta[st].item = -1;
          meta[st].flags = kMetaDone;
          mbar_arrive(&bars->k_full[st]);
        }
        break;
      }
      const int32_t* bt = p.block_tables + (int64_t)it.seq * p.max_blocks;
      const int group = 32 / nb;  // tiles that 32 blocks make
      const int my_tile = lane / nb, my_block = lane % nb;
      int next_phys = (int)p.num_blocks;
      float2 next_sc = make_float2(1.f, 1.f);
      bool ok = true;
      int tile = 0;  // of the group
      for (int kbase = it.kb; kbase < it.ke; kbase += kKeys, ++g) {
        const int st = g % kStages;
        const bool first = kbase == it.kb;
        if (tile == 0) {
          const int place = kbase + group * kKeys + lane * p.bs;
          next_phys = place < it.ke ? block_of(bt, nblk, at, len, place) : (int)p.num_blocks;
        } else if (tile == 1 && !vprod) {
          next_sc = make_float2(1.f, 1.f);
          if (next_phys < p.num_blocks) {
            const int64_t i = (int64_t)next_phys * p.Hkv + it.kvh;
            next_sc = make_float2(__ldg(p.k_scales + i), __ldg(p.v_scales + i));
          }
        }
        if (!wait_all(&bars->kv_empty[st], ((g / kStages) & 1) ^ 1, wc)) {
          ok = false;
          break;
        }
        if (!vprod && lane == 0 && it.ke - kbase <= kFetchLeadTiles * kKeys &&
            (first || it.ke - (kbase - kKeys) > kFetchLeadTiles * kKeys))
          mbar_arrive(&bars->fetch_go);  // once per item: the next one may be taken now
        // testing only: this tile is never loaded, so the waits for it run out
        if (vprod || p.fault_tile != g + 1 || blockIdx.x != 0) {
          uint8_t* dst = smem + st * kStageBytes + (vprod ? kTileBytes : 0);
          if (!vprod) {
            if (my_tile == tile) tile_scales[st * 16 + my_block] = sc;
            if (lane == 0) {
              Meta& m = meta[st];
              m.item = idx;
              m.kbase = kbase;
              m.flags = ((kbase + kKeys >= it.ke) ? kMetaLast : 0) | (first ? kMetaFirst : 0);
              m.seq = it.seq;
              m.kvh = it.kvh;
              m.row0 = it.row0;
              m.nrows = it.nrows;
              m.ke = it.ke;
              m.part = it.part;
              m.grp = it.grp;
              m.L = L;
              m.n = n;
              m.qstart = qstart;
              m.qbuf = qb;
            }
            __syncwarp();
          }
          if (lane == 0) mbar_arrive_expect_tx(&fullb[st], kTileBytes);
          __syncwarp();
          if (my_tile == tile)
            tma_load_4d(dst + my_block * p.bs * 128, vprod ? &vmap : &kmap, &fullb[st], 0, it.kvh, 0, phys);
        }
        if (++tile == group) {
          tile = 0;
          phys = next_phys;
          sc = make_scales<kWeightExp>(next_sc);
        }
      }
      if (!ok) {
        drain();
        break;
      }
    }
  } else if (warp == 10) {
    // ================================================================ item fetch, q terms
    for (int c = 0;; ++c) {
      const int qb = c & 1;
      if (c >= 1 && !wait_all(&bars->fetch_go, (c - 1) & 1, wc)) break;
      if (c >= 2 && !wait_all(&bars->islot_free[qb], ((c - 2) >> 1) & 1, wc)) break;
      int idx = 0;
      if (lane == 0) idx = atomicAdd(p.counter, 1);
      idx = __shfl_sync(0xffffffffu, idx, 0);
      ItemSlot& sl = islots[qb];
      if (idx >= n_items) {
        if (lane == 0) sl.done = 1;
        mbar_arrive(&bars->islot_full[qb]);  // every lane: count 32
        break;
      }
      WorkItem it;
      {
        const int4* src = reinterpret_cast<const int4*>(p.items + idx);
        const int4 a = __ldcg(src), b = __ldcg(src + 1);
        it.seq = a.x; it.kvh = a.y; it.row0 = a.z; it.nrows = a.w;
        it.kb = b.x; it.ke = b.y; it.part = b.z; it.grp = b.w;
      }
      const int L = p.context_lens[it.seq];
      const int qstart = p.query_start_loc[it.seq];
      const int n = p.query_start_loc[it.seq + 1] - qstart;
      const int nblk = (L + p.bs - 1) / p.bs;
      // this lane's element pairs of the item's q rows, on their way while the block ids are read
      const __nv_bfloat16* q0 =
          static_cast<const __nv_bfloat16*>(p.q) + ((int64_t)qstart * p.Hq + (int64_t)it.kvh * p.G) * 128;
      uint2 raw[NR];
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        raw[r] = make_uint2(0, 0);
        if (r < it.nrows) {
          const int row = it.row0 + r, tok = row / p.G, gh = row - tok * p.G;
          raw[r] = __ldg(reinterpret_cast<const uint2*>(q0 + ((int64_t)tok * p.Hq + gh) * 128) + lane);
        }
      }
      int at = 0, len = 0;
      if (p.window > 0) {
        const Hole hole(L, n, it.row0 / p.G, p.window, p.num_sink, p.bs);
        at = hole.at;
        len = hole.len;
      }
      const int32_t* bt = p.block_tables + (int64_t)it.seq * p.max_blocks;
      const int place = it.kb + lane * p.bs;
      const int phys = place < it.ke ? block_of(bt, nblk, at, len, place) : (int)p.num_blocks;
      sl.phys[lane] = phys;
      float2 sc = make_float2(1.f, 1.f);
      if (phys < p.num_blocks) {
        const int64_t i = (int64_t)phys * p.Hkv + it.kvh;
        sc = make_float2(__ldg(p.k_scales + i), __ldg(p.v_scales + i));
      }
      sl.scales[lane] = sc;
      if (lane == 0) {
        sl.it = it;
        sl.idx = idx;
        sl.L = L - len;
        sl.qstart = qstart;
        sl.n = n;
        sl.nblk = nblk;
        sl.at = at;
        sl.len = len;
        sl.done = 0;
      }
      mbar_arrive(&bars->islot_full[qb]);  // every lane, after its own writes
      // item c-2's q terms are no longer read
      if (c >= 2 && !wait_all(&bars->q_empty[qb], ((c - 2) >> 1) & 1, wc)) break;
      uint8_t* qd = smem + Y::kQOff + qb * Y::kNQ * 128;
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float x[4] = {bf16_lo(raw[r].x), bf16_hi(raw[r].x), bf16_lo(raw[r].y), bf16_hi(raw[r].y)};
        float top = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        // the row's power of two: its largest |q| becomes 128 to 256 (E4M3 ends at 448)
        const int e = min(max((int)(__float_as_uint(top) >> 23) - 127 - 7, -126), 120);
        const float down = __uint_as_float((uint32_t)(127 - e) << 23);
        uint32_t hi = 0, lo = 0;
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          uint32_t t, u;
          split_e4m3(x[i] * down, x[i + 1] * down, t, u);
          hi |= t << (8 * i);
          lo |= u << (8 * i);
        }
        // rows r and NR + r, columns 4 lane ..: 16-byte chunk lane / 4, swizzled
        const int c1 = (lane >> 2) ^ (r & 7), c2 = (lane >> 2) ^ ((NR + r) & 7);
        *reinterpret_cast<uint32_t*>(qd + r * 128 + (c1 << 4) + (lane & 3) * 4) = hi;
        *reinterpret_cast<uint32_t*>(qd + (NR + r) * 128 + (c2 << 4) + (lane & 3) * 4) = lo;
        if (lane == r) row_scales[qb * NR + r] = __uint_as_float((uint32_t)(127 + e) << 23) * p.scale_log2;
      }
      fence_proxy_async_smem();
      mbar_arrive(&bars->q_full[qb]);
    }
  } else if (warp == 1) {
    // ================================================================ S issuer
    // The issuing warps stay together and only the issue itself is one lane's, so
    // that descriptors and counters are warp-uniform.  Waits are taken several at
    // a time (one that is over takes 110 cycles), and S and P.V have a warp each:
    // an MMA takes a warp 70 cycles to issue, and the eight of a tile with their
    // waits and commits took one warp 1600, as long as a tile comes from HBM.
    const bool issues = lane == 0;
    const uint64_t dk0 = desc_k(smem_base), dq0 = desc_k(smem_base + Y::kQOff);
    int g = 0, it_cnt = -1;
    for (;; ++g) {
      const int st = g % kStages, b = g & 1;
      uint64_t* const kf = &bars->k_full[st];
      const uint32_t kph = (g / kStages) & 1, sph = ((g >> 1) & 1) ^ 1;
      // K(g) landed, S buffer b read
      if (!__all_sync(0xffffffffu, mbar_test_wait3(kf, kph, &bars->s_free[b], sph, kf, kph)) &&
          (!wait_all(kf, kph, wc) || (!(meta[st].flags & kMetaDone) && !wait_all(&bars->s_free[b], sph, wc))))
        break;
      const int flags = meta[st].flags;
      if (flags & kMetaDone) break;
      if (flags & kMetaFirst) {
        ++it_cnt;
        if (!wait_all(&bars->q_full[it_cnt & 1], (it_cnt >> 1) & 1, wc)) break;
      }
      tc_fence_after();
      const uint64_t dk = desc_add(dk0, st * kStageBytes);
      const uint64_t dq = desc_add(dq0, (it_cnt & 1) * Y::kNQ * 128);
      const uint32_t d = tmem + Y::kSCol + b * Y::kNQ;
      if (issues) {
#pragma unroll
        for (int kk = 0; kk < 128 / 32; ++kk)
          umma_f8(d, desc_add(dk, kk * 32), desc_add(dq, kk * 32), Y::kIdescS, kk > 0 ? 1u : 0u);
        umma_commit(&bars->s_full[b]);
        if (flags & kMetaLast) umma_commit(&bars->q_empty[it_cnt & 1]);
      }
      __syncwarp();
    }
    // leaving: the MMAs already issued finish before TMEM is freed
    if (g > 0) wait_all(&bars->s_full[(g - 1) & 1], ((g - 1) >> 1) & 1, wc);
  } else if (warp == 12) {
    // ================================================================ P.V issuer
    const bool issues = lane == 0;
    const uint64_t dv0 = desc_mn(smem_base + kTileBytes), dp0 = desc_k(smem_base + Y::kPOff);
    int g = 0, it_cnt = -1;
    for (;; ++g) {
      const int st = g % kStages, b = g & 1;
      const uint32_t sph = (g / kStages) & 1, pph = (g >> 1) & 1;
      // the tile's metadata (with its K)
      if (!wait_all(&bars->k_full[st], sph, wc)) break;
      const int flags = meta[st].flags;
      if (flags & kMetaDone) break;
      const bool first = flags & kMetaFirst;
      if (first) ++it_cnt;
      const int ob = it_cnt & 1;
      // P and V there, and, on an item's first tile, O^T[ob], which is about to be
      // overwritten, read by the epilogue of the item before last
      uint64_t *const pf = &bars->p_full[b], *const vf = &bars->v_full[st];
      uint64_t* const of = first ? &bars->o_empty[ob] : vf;
      const uint32_t oph = first ? ((it_cnt >> 1) & 1) ^ 1 : sph;
      if (!__all_sync(0xffffffffu, mbar_test_wait3(pf, pph, vf, sph, of, oph)) &&
          (!wait_all(of, oph, wc) || !wait_all(pf, pph, wc) || !wait_all(vf, sph, wc)))
        break;
      tc_fence_after();
      const uint64_t dv = desc_add(dv0, st * kStageBytes);
      const uint64_t dp = desc_add(dp0, b * Y::kNP * 128);
      const uint32_t d = tmem + Y::kOCol + ob * Y::kNP, more = first ? 0u : 1u;
      if (issues) {
#pragma unroll
        for (int kk = 0; kk < kKeys / 32; ++kk)  // 32 keys: 4 KB of V's rows, 32 bytes of the weights'
          umma_f8(d, desc_add(dv, kk * 4096), desc_add(dp, kk * 32), Y::kIdescO, kk == 0 ? more : 1u);
        umma_commit(&bars->kv_empty[st]);
        if (flags & kMetaLast) umma_commit(&bars->o_full[ob]);
      }
      __syncwarp();
    }
    if (g > 0) wait_all(&bars->kv_empty[(g - 1) % kStages], ((g - 1) / kStages) & 1, wc);
  } else {
    // ================================================================ softmax / epilogue
    constexpr int kLog = NR == 4 ? 2 : NR == 8 ? 3 : 4;
    const int q4 = warp & 3;
    const int t = q4 * 32 + lane;  // key of the tile (S^T lane) / output column (O^T lane)
    const uint32_t lane_base = tmem + ((uint32_t)(q4 * 32) << 16);
    EpSlot* slots = reinterpret_cast<EpSlot*>(smem + Y::kSlotOff);
    if (warp < 6) {
      // ---------------------------------------------------------- softmax
      // Failures of waits are carried in `pending` (warp-uniform) to the next
      // agreement barrier (barrier 1 over the 4 softmax warps), where all four
      // warps go on or leave.
      // The weights are made with the reference as it stands, and the barrier
      // that ends the tile tells whether a key of any warp exceeded it by the
      // threshold; only then are the tile's row maxima found and exchanged and
      // the weights made again (the first tile of an item, and few others): maxima in
      // every tile are a chain of shuffles and a barrier ahead of the exponentials.
      const int my_row = lane >> (5 - kLog);  // row this lane holds after a reduction
      const bool row_writer = (lane & ((1 << (5 - kLog)) - 1)) == 0;
      const int my_block = t / p.bs;
      float m_ref[NR], lsum[NR];
      // a row's scale times the logit scale: in registers where they do (read in every
      // tile from shared memory: 224 us against 207 for 4 x 131072 keys)
      constexpr bool kHeld = NR <= 8;
      float unit[kHeld ? NR : 1];
      int ends[NR];  // keys a row may see end here (and its window starts p.window keys earlier)
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        m_ref[r] = -CUDART_INF_F;
        lsum[r] = 0.f;
        ends[r] = 0;
      }
      const int window = p.window > 0 ? p.window : 1 << 30;
      Meta mt{};
      int it_cnt = -1;
      bool pending = false;
      for (int g = 0;; ++g) {
        const int st = g % kStages;
        const int b = g & 1;
        float* redb = red + b * 4 * NR;  // [4 warps][NR], double-buffered by tile
        uint64_t* const kf = &bars->k_full[st];
        const uint32_t kph = (g / kStages) & 1, ph = (g >> 1) & 1;
        // the tile's metadata (with its K), its S, and the P buffer free (P.V of
        // tile g-2 done): all three at once where they are there
        uint64_t* const ef = g < 2 ? kf : &bars->kv_empty[(g - 2) % kStages];
        const uint32_t eph = g < 2 ? kph : ((g - 2) / kStages) & 1;
        bool fail = pending;
        if (!fail && !__all_sync(0xffffffffu, mbar_test_wait3(kf, kph, &bars->s_full[b], ph, ef, eph))) {
          fail = !wait_all(kf, kph, wc);
          if (!fail && !(meta[st].flags & kMetaDone))
            fail = !wait_all(&bars->s_full[b], ph, wc) || !wait_all(ef, eph, wc);
        }
        const int flags = fail ? 0 : meta[st].flags;
        const bool done = (flags & kMetaDone) != 0;
        if (!fail && !done && (flags & kMetaFirst)) {
          mt = meta[st];
          ++it_cnt;
          fail = !wait_all(&bars->q_full[mt.qbuf], (it_cnt >> 1) & 1, wc);
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            m_ref[r] = -CUDART_INF_F;
            lsum[r] = 0.f;
            const int tok = (mt.row0 + r) / p.G;
            if constexpr (kHeld) unit[r] = row_scales[mt.qbuf * NR + r];
            ends[r] = r < mt.nrows ? (p.causal ? mt.L - mt.n + tok + 1 : mt.L) : 0;
          }
        }
        const bool ok = !fail && !done;
        const int kbase = ok ? meta[st].kbase : 0;
        const int key = kbase + t;
        Scales sc{1.f, 0.f, 1.f, 0.f};
        float v[NR], w[NR];  // log2 of the weights (V's scale in them); the weights
        bool exceeds = false;
        uint8_t* pbuf = smem + Y::kPOff + b * Y::kNP * 128 + (t & 15);
        const int chunk = t >> 4;
        auto at = [&](int row) { return pbuf + row * 128 + ((chunk ^ (row & 7)) << 4); };
        // the weights and their three terms in this tile's P buffer: row i NR + r, column t, 128-byte swizzle
        auto make_weights = [&]() {
#pragma unroll
          for (int r = 0; r < NR; r += 2) {
            auto m_use = [&](int i) { return (m_ref[i] == -CUDART_INF_F ? 0.f : m_ref[i]) - kWeightExp; };
            w[r] = fast_exp2(v[r] - m_use(r));
            w[r + 1] = fast_exp2(v[r + 1] - m_use(r + 1));
            const __half2 h = __floats2half2_rn(w[r], w[r + 1]);
            const uint32_t b0 = *reinterpret_cast<const uint32_t*>(&h), t0 = b0 & 0xFF00FF00u;
            const __half2 h1 = __hsub2(h, *reinterpret_cast<const __half2*>(&t0));  // exact
            const uint32_t b1 = *reinterpret_cast<const uint32_t*>(&h1), t1 = b1 & 0xFF00FF00u;
            const __half2 h2 = __hsub2(h1, *reinterpret_cast<const __half2*>(&t1));
            const uint32_t b2 = *reinterpret_cast<const uint32_t*>(&h2) + 0x00800080u;  // to nearest
            *at(r) = (uint8_t)(b0 >> 8);
            *at(r + 1) = (uint8_t)(b0 >> 24);
            *at(NR + r) = (uint8_t)(b1 >> 8);
            *at(NR + r + 1) = (uint8_t)(b1 >> 24);
            *at(2 * NR + r) = (uint8_t)(b2 >> 8);
            *at(2 * NR + r + 1) = (uint8_t)(b2 >> 24);
          }
        };
        if (ok) {
          uint32_t sraw[2 * NR];
          tc_fence_after();
          tmem_ld_cols<2 * NR>(lane_base + Y::kSCol + b * Y::kNQ, sraw);
          sc = tile_scales[st * 16 + my_block];
          tmem_wait_ld();
          tc_fence_before();
          mbar_arrive(&bars->s_free[b]);
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            const bool seen = key < min(ends[r], mt.ke) && (key >= ends[r] - window || key < p.num_sink);
            const float s = (__uint_as_float(sraw[r]) + __uint_as_float(sraw[NR + r])) * sc.k;
            const float u = kHeld ? unit[kHeld ? r : 0] : row_scales[mt.qbuf * NR + r];  // (log2 units)
            v[r] = seen ? fmaf(s, u, sc.log_v) : -CUDART_INF_F;
            exceeds |= v[r] > m_ref[r] + kRescaleThreshold;  // false while both are -inf
          }
          if (flags & kMetaLast) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->q_empty[mt.qbuf]);
          }
          if (!(flags & kMetaFirst)) make_weights();
        }
        bool any_rescale = false;
        float alpha[NR];
        if (barrier_any(1, 128, exceeds || !ok)) {
          // leave, or raise the reference
          if (barrier_any(1, 128, !ok)) {
            // leaving: at the end of the work (nobody failed), tell the epilogue
            if (!barrier_any(1, 128, fail)) {
              const int ob = (it_cnt + 1) & 1;
              if (wait_all(&bars->ml_empty[ob], (((it_cnt + 1) >> 1) & 1) ^ 1, wc)) {
                if (t == 0) slots[ob].done = 1;
                mbar_arrive(&bars->ml_full[ob]);
              }
            }
            break;
          }
          float a[NR];
#pragma unroll
          for (int r = 0; r < NR; ++r) a[r] = v[r];
          const float wmax = xreduce<NR>(a, lane, MaxOp());
          if (row_writer) redb[q4 * NR + my_row] = wmax;
          named_barrier(1, 128);
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            const float mx = fmaxf(fmaxf(redb[r], redb[NR + r]), fmaxf(redb[2 * NR + r], redb[3 * NR + r]));
            alpha[r] = 1.f;
            if (mx > m_ref[r] + kRescaleThreshold) {
              alpha[r] = fast_exp2(m_ref[r] - mx);  // 0 when m_ref is -inf
              any_rescale |= m_ref[r] != -CUDART_INF_F;
              m_ref[r] = mx;
              lsum[r] *= alpha[r];
            }
          }
          any_rescale = any_rescale && !(flags & kMetaFirst);
          make_weights();
        } else if (flags & kMetaFirst) {
          make_weights();  // (none of the tile's keys is seen by any row)
        }
#pragma unroll
        for (int r = 0; r < NR; ++r) lsum[r] = fmaf(w[r], sc.inv_v, lsum[r]);
        pending = false;
        if (any_rescale) {
          // O^T must hold every earlier tile's P.V before it is scaled; thread t
          // owns O^T row t (output column t), whose columns i NR + r belong to row r
          pending = !wait_all(&bars->kv_empty[(g - 1) % kStages], ((g - 1) / kStages) & 1, wc);
          if (!pending) {
            tc_fence_after();
            const uint32_t ocol = lane_base + Y::kOCol + (it_cnt & 1) * Y::kNP;
            uint32_t o[3 * NR];
            tmem_ld_cols<3 * NR>(ocol, o);
            tmem_wait_ld();
#pragma unroll
            for (int r = 0; r < 3 * NR; ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) * alpha[r % NR]);
            tmem_st_cols<3 * NR>(ocol, o);
            tmem_wait_st();
          }
        }
        // a tile that holds keys before every row's window (row 0's comes first)
        const int lo = ends[0] - window;
        const bool early = kbase < lo && kbase + kKeys > p.num_sink;
        if ((kbase + kKeys > mt.L || early) && !pending) {
          // keys at or past the sequence's end hold arbitrary codes, as those before
          // the windows may: zero their V rows (after the tile has landed) so that
          // 0 * V stays 0
          pending = !wait_all(&bars->v_full[st], (g / kStages) & 1, wc);
          if (!pending && (key >= mt.L || (key < lo && key >= p.num_sink))) {
            uint4* v0 = reinterpret_cast<uint4*>(smem + st * kStageBytes + kTileBytes + t * 128);
#pragma unroll
            for (int c = 0; c < 8; ++c) v0[c] = make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(&bars->p_full[b]);

        if (!(flags & kMetaLast)) continue;
        // ---- item end: row sums over the 128 key-threads, handed to the epilogue
        float* reds = red + (b ^ 1) * 4 * NR;  // the other buffer of this tile pair
        {
          float c[NR];
#pragma unroll
          for (int r = 0; r < NR; ++r) c[r] = lsum[r];
          const float wsum = xreduce<NR>(c, lane, AddOp());
          if (row_writer) reds[q4 * NR + my_row] = wsum;
        }
        if (barrier_any(1, 128, pending)) break;
        const int ob = it_cnt & 1;
        pending = !wait_all(&bars->ml_empty[ob], ((it_cnt >> 1) & 1) ^ 1, wc);
        if (!pending) {
          EpSlot& es = slots[ob];
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            if (t == r) {
              es.m[r] = m_ref[r];
              es.l[r] = (reds[r] + reds[NR + r]) + (reds[2 * NR + r] + reds[3 * NR + r]);
            }
          }
          if (t == 0) {
            es.mt = mt;
            es.done = 0;
          }
        }
        // reds[] is rewritten two tiles from now; the slot is complete
        if (barrier_any(1, 128, pending)) break;
        mbar_arrive(&bars->ml_full[ob]);
      }
    } else {
      // ---------------------------------------------------------- epilogue
      // Over the 4 epilogue warps, barrier 3: agreement after each wait that
      // decides what they do next; barrier 2: the split tickets' ordering.
      const int d = t;
      int* flag_last = reinterpret_cast<int*>(tmem_slot + 1);
      bool pending = false;
      auto out_row = [&](int seq_q, int kvh, int row) {
        const int tok = row / p.G, gh = row - tok * p.G;
        return static_cast<__nv_bfloat16*>(p.out) + ((int64_t)(seq_q + tok) * p.Hq + (int64_t)kvh * p.G + gh) * 128;
      };
      for (int it_cnt = 0;; ++it_cnt) {
        const int ob = it_cnt & 1;
        const bool fail = pending || !wait_all(&bars->ml_full[ob], (it_cnt >> 1) & 1, wc);
        if (barrier_any(3, 128, fail)) break;
        const EpSlot& es = slots[ob];
        if (es.done) break;
        const Meta mt = es.mt;
        float mrow[NR], lrow[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          mrow[r] = es.m[r];
          lrow[r] = es.l[r];
        }
        mbar_arrive(&bars->ml_empty[ob]);
        pending = !wait_all(&bars->o_full[ob], (it_cnt >> 1) & 1, wc);
        float acc[NR];
        if (!pending) {
          uint32_t o[3 * NR];
          tc_fence_after();
          tmem_ld_cols<3 * NR>(lane_base + Y::kOCol + ob * Y::kNP, o);
          tmem_wait_ld();
          tc_fence_before();
          mbar_arrive(&bars->o_empty[ob]);
          // smallest terms first; p.v_scale undoes the weights' factor
#pragma unroll
          for (int r = 0; r < NR; ++r)
            acc[r] = ((__uint_as_float(o[2 * NR + r]) + __uint_as_float(o[NR + r])) + __uint_as_float(o[r])) * p.v_scale;
        }
        if (mt.part < 0) {
          if (pending) continue;  // leaves at the next agreement
#pragma unroll
          for (int r = 0; r < NR; ++r)
            if (r < mt.nrows) out_row(mt.qstart, mt.kvh, mt.row0 + r)[d] = __float2bfloat16_rn(acc[r] / lrow[r]);
          continue;
        }
        if (!pending) {
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            if (r < mt.nrows) {
              p.part_acc[(int64_t)(mt.part + r) * 128 + d] = acc[r];
              if (d == r) p.part_ml[mt.part + r] = make_float2(mrow[r], lrow[r]);
            }
          }
        }
        // The split that completes its merge group combines the group's partial
        // rows: m = max m_p, l = sum l_p 2^(m_p - m), O = sum acc_p 2^(m_p - m) / l.
        // Release: the barrier orders every thread's partial writes before
        // thread 0's fence and ticket; acquire: thread 0's fence after the
        // ticket, then the barrier, before anyone reads other splits' rows.
        if (barrier_any(3, 128, pending)) break;
        if (d == 0) {
          __threadfence();
          *flag_last = atomicAdd(p.tickets + mt.grp, 1);
        }
        named_barrier(2, 128);
        const MergeGroup gr = load_group(p.groups + mt.grp);
        if (*flag_last == gr.nsplit - 1) {
          if (d == 0) __threadfence();
          named_barrier(2, 128);
          for (int r = 0; r < gr.nrows; ++r) {
            float M = -CUDART_INF_F;
#pragma unroll 8
            for (int k = 0; k < gr.nsplit; ++k)
              M = fmaxf(M, __ldcg(&p.part_ml[gr.part_base + k * gr.nrows + r]).x);
            const float Mu = M == -CUDART_INF_F ? 0.f : M;
            float lt = 0.f, sum = 0.f;
#pragma unroll 8
            for (int k = 0; k < gr.nsplit; ++k) {
              const int slot = gr.part_base + k * gr.nrows + r;
              const float2 ml = __ldcg(&p.part_ml[slot]);
              const float wt = fast_exp2(ml.x - Mu);
              lt = fmaf(wt, ml.y, lt);
              sum = fmaf(wt, __ldcg(&p.part_acc[(int64_t)slot * 128 + d]), sum);
            }
            out_row(mt.qstart, gr.kvh, gr.row0 + r)[d] = __float2bfloat16_rn(sum / lt);
          }
        }
        named_barrier(2, 128);  // the flag is rewritten by the next split item
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
  // as in the bf16 kernel: this grid's completion implies the many-row kernel's
  if (p.no_wait && threadIdx.x == 0) pdl_wait();
}

template <int NR>
cudaError_t launch_t(const AttnParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap, int grid, cudaStream_t s) {
  static unsigned long long done_mask = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!(__atomic_load_n(&done_mask, __ATOMIC_ACQUIRE) & (1ull << dev))) {
    e = cudaFuncSetAttribute(dec_fp8block_kernel<NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<NR>::kSmem);
    if (e != cudaSuccess) return e;
    __atomic_fetch_or(&done_mask, 1ull << dev, __ATOMIC_RELEASE);
  }
  AttnParams q = p;
  q.v_scale = 1.f / (1 << kWeightExp);
  e = launch_pdl(dec_fp8block_kernel<NR>, dim3(grid), dim3(kThreads), Lay<NR>::kSmem, s, q, kmap, vmap);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_dec_fp8block(const AttnParams& p, int unit_rows, const CUtensorMap& kmap, const CUtensorMap& vmap,
                                int grid, cudaStream_t s) {
  if (unit_rows == 4) return launch_t<4>(p, kmap, vmap, grid, s);
  if (unit_rows == 8) return launch_t<8>(p, kmap, vmap, grid, s);
  return launch_t<16>(p, kmap, vmap, grid, s);
}

}  // namespace pkv
