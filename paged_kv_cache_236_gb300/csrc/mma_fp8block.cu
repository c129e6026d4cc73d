// Attention of many rows per kv head (prompt chunks, wide verify windows) over
// pools of E4M3 codes with a scale for each block and kv head: tcgen05.mma with
// TMEM accumulators (paged_attention_forward_fp8block).
//
// With codes ck, cv and block scales sk, sv, for rows r of one kv head:
//   x[r][j] = scale log2(e) (q_r . ck_j) sk(j)          (log2 units)
//   out_r   = sum_j 2^(x - m) sv(j) cv_j / sum_j 2^(x - m)
// for items of up to 128 rows, 128 keys a tile, otherwise as the bf16 kernel does
// it (mma_attn.cu: tiles, two issuing threads, epilogue, splits, waits).  What
// differs:
//   Q K^T  multiplies K's codes as they land.  A row of q is 2^e (q1 + q2), E4M3
//          each (e from the row's largest |q|: bf16's 8 bits, off by at most 2^-17
//          of that largest value), two chains of four MMAs of K = 32 into the same
//          accumulator: as long as eight of K = 16 in bf16.  Three warps split
//          the Q tile in place.
//   P V    takes fp16: V's codes are converted (exactly) by four warps, which zero
//          the rows that no row of the item sees.  The weights carry V's scale:
//          w = 2^(x + log2 sv - m + 7), with m a running reference of x + log2 sv
//          (raised when a tile exceeds it by 8: w <= 2^15), fp16 with 11 bits down
//          to 2^-21 of the row's largest; the denominator takes w / (2^7 sv).
//          8-bit weights would take three terms each here, where the softmax
//          warps' instructions are what is scarce.
// Scales are applied by runs of 8 columns (no block is shorter).
//
// A tile of 128 x 128 takes about 2700 cycles (MMAs 1100 of them; the softmax
// warps' chain: 200 for its waits, 600 for the maxima, 1400 for the weights, 100 to
// 700 to hand them on), so that operations bound it and not bytes: chunks of 512 on up to 2048
// (86 GFLOP) 150 us, 574 TFLOP/s; the verify batch (5 tokens of 8 heads on 8192
// keys, 40 of a tile's 128 rows used) 192 us, 2.8 TB/s of codes.
//
// Roles (640 threads, one CTA per SM, persistent):
//   warp 0     the thread issuing P.V;
//   warp 1     TMEM allocation, the thread issuing Q K^T;
//   warp 2     K producer: {128 bytes, 1, block_size, 1} boxes (128-byte
//              swizzle), ids two tiles ahead and scales one, into a ring of 8
//              tiles' scales (the softmax warps read them up to 5 tiles after the
//              K stage they came with is free);
//   warp 12    V producer: codes into a staging ring;
//   warps 16-19 V converters, one to each scheduler, since conversions and the
//              softmax warps' exponentials share a pipe;
//   warps 4-11 softmax / correction / epilogue, two threads per row;
//   warp 14    item fetch, Q and output stores;
//   warps 3,13,15 split the Q tile.
// Shared memory: 2 Q tiles (64 KB), 3 stages of K codes (48 KB), 2 of V codes
// (32 KB), 2 fp16 V tiles (64 KB).
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <limits.h>
#include <math_constants.h>

#include "block_scales.cuh"
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_tc.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 640;
constexpr int kKeys = kMmaTileKeys;                 // 128 keys per tile
constexpr int kKStages = 3, kVStages = 2;
constexpr int kCodeTile = kKeys * 128;              // K or V codes of a tile (16 KB)
constexpr int kHalfKV = kKeys * 128;                // one 64-column half of an fp16 V tile (16 KB)
constexpr int kTileBytes = 2 * kHalfKV;             // an fp16 V tile: 32 KB
constexpr int kScaleSlots = 8;
constexpr int kConverters = 128;                    // threads
constexpr int kSplitters = 96;                      // threads
constexpr int kWeightExp = 7;                       // weights are 2^7 times their value, at most 2^15
constexpr int kQBytes = kMmaRows * 128 * 2;         // 32 KB (two 16 KB halves)
// shared-memory carve-up (offsets from a 1024-byte aligned base)
constexpr int kQOff = 0;
constexpr int kKOff = kQOff + 2 * kQBytes;
constexpr int kCOff = kKOff + kKStages * kCodeTile;  // V codes
constexpr int kVOff = kCOff + kVStages * kCodeTile;
constexpr int kBarOff = kVOff + kVStages * kTileBytes;
constexpr int kNumBars = 10 + 2 * kKStages + 3 * kVStages + 8 + 1 + 2 + kScaleSlots;
constexpr int kSlotOff = (kBarOff + kNumBars * 8 + 16 + 15) & ~15;  // 2 item slots
constexpr int kRedOff = kSlotOff + 2 * 320;         // [2 tiles][2 halves][128 rows] row maxima / sums
// No alignment slack: the buffers need a 1024-byte aligned base, which the
// dynamic shared memory of a kernel without static shared memory has; the
// kernel checks and refuses to run otherwise.
constexpr int kRowScaleOff = kRedOff + 2 * 2 * 128 * 4;        // [2 Q tiles][128]
constexpr int kScaleOff = kRowScaleOff + 2 * 128 * 4;         // [kScaleSlots][16] float4
constexpr int kSmem = kScaleOff + kScaleSlots * 16 * 16;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSCol = 0;    // S buffer b at kSCol + 128 b
constexpr uint32_t kPCol = 256;  // P buffer b at kPCol + 64 b
constexpr uint32_t kOCol = 384;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
// Register split between warpgroups (setmaxnreg): warpgroups 0, 3 and 4 (MMA
// issuers, producers, item fetch, Q split, converters) give up registers that
// warpgroups 1 and 2 (softmax) take.  The sum must stay within what the block is launched with
// (kThreads x the kernel's register count); the launcher checks the count.
constexpr int kRegs = 96, kRegsLight = 56, kRegsSoftmax = 152;
static_assert(3 * 128 * kRegsLight + 2 * 128 * kRegsSoftmax <= kThreads * kRegs, "register split above the launch's");

constexpr uint32_t kIdescS = idesc_f8(128, kKeys, kE4m3, kE4m3, false, false);
// fp16 A and B: idesc_bf16 with the format fields 0
constexpr uint32_t kIdescO = idesc_bf16(128, 128, false, true) & ~((7u << 7) | (7u << 10));

// V as the B of P.V (MN-major): the two 64-column halves are kHalfKV apart,
// 8-key groups 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_v(uint32_t saddr) { return smem_desc(saddr, kHalfKV, 1024); }

struct Bars {
  uint64_t q_full[2], q_split[2], q_empty[2], slot_full[2], slot_free[2];
  uint64_t k_full[kKStages], k_empty[kKStages];
  uint64_t c_full[kVStages], c_empty[kVStages];  // V codes landed; converted
  uint64_t v_full[kVStages];                     // the fp16 V tile written
  // s_full[b], phase n: S of tile 2n+b complete; s_free[b]: the softmax
  // warps have read it.  pv_done[b], phase n: the P.V of tile 2n+b complete,
  // and with it every earlier P.V.
  uint64_t s_full[2], s_free[2], pv_done[2], p_full[2];
  uint64_t o_empty;
  // o_staged[b], phase n: the epilogue of item 2n+b has left its output tile
  // in Q buffer b (or written it directly)
  uint64_t o_staged[2];
  uint64_t sc_full[kScaleSlots];  // a tile's scales written
};

// An item's description, published by the item-fetching warp before its Q
// tile is loaded (slot_full), with the block ids of its first two key tiles and
// the scales of the first one's.  L counts places (Hole: at, len).
struct alignas(16) ItemSlot {
  WorkItem it;
  int L, qstart, n, done;
  int nblk, at, len, pad;
  int phys[32];
  float2 scales[16];
};
// readers of a slot: the 256 softmax threads, the two MMA-issuing threads, the
// K / V producers, the four converting and three splitting warps
constexpr int kSlotReaders = 256 + 2 + 2 + 4 + 3;

static_assert(sizeof(ItemSlot) == 320, "item slot");
static_assert(sizeof(Bars) == kNumBars * 8, "barrier block");
static_assert(kVStages == 2, "V stage t % 2 is released by the P.V barrier of tile t");
static_assert(kSmem <= 232448, "shared memory");
static_assert(kKOff % 1024 == 0 && kCOff % 1024 == 0 && kVOff % 1024 == 0, "swizzled tiles");
static_assert(kBarOff % 8 == 0 && kSlotOff % alignof(ItemSlot) == 0 && kRedOff % 16 == 0 && kScaleOff % 16 == 0,
              "alignment");

__device__ __forceinline__ uint32_t pack_half(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Rows row0 .. row1 - 1 (a multiple of 4) of a Q tile in place, by a warp, a row at a time (four
// on their way): 128 bf16 in two 64-column halves kHalf apart (16-byte chunk j at
// j ^ (r & 7) of the row) become 128 codes of q1 in the first and of q2 in the
// second, swizzled alike.  scales[r]: 2^e times the logit scale.
__device__ __forceinline__ void split_rows(uint8_t* tile, int row0, int row1, float* scales, float scale_log2,
                                           int lane) {
  // The least e: 2^e scale_log2 stays in [2^-84, 2^-83], so that its product with a K
  // scale (2^-60 or more) is not 0, which the masks' infinities must not meet.  Rows
  // below 2^(e + 7) lose low bits: 2^-10 2^e of each of 128 elements, times values of
  // K up to 448 * 2^60, is 2^-17 of a logit.
  const int least = max(-84 - min(ilogbf(scale_log2), 127), -126);
  // this lane's columns 4 lane .. + 3: 8 bytes of bf16, 4 codes
  const int from = (lane >> 4) * kHalf + (lane & 1) * 8, fc = (lane & 15) >> 1;
  const int to = (lane & 3) * 4, tc = lane >> 2;
#pragma unroll 1
  for (int r0 = row0; r0 < row1; r0 += 4) {
    uint2 raw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      raw[i] = *reinterpret_cast<const uint2*>(tile + (r0 + i) * 128 + from + ((fc ^ ((r0 + i) & 7)) << 4));
    __syncwarp();  // all of the rows is read before any of it is written
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t top2 = __vmaxu2(raw[i].x & 0x7FFF7FFFu, raw[i].y & 0x7FFF7FFFu);
      const int top = (int)__reduce_max_sync(0xffffffffu, max(top2 & 0xFFFFu, top2 >> 16));
      // the largest |q| becomes 128 to 256 (E4M3 ends at 448)
      const int e = min(max((top >> 7) - 127 - 7, least), 120);
      const float down = __uint_as_float((uint32_t)(127 - e) << 23);
      const float a[4] = {bf16_lo(raw[i].x) * down, bf16_hi(raw[i].x) * down, bf16_lo(raw[i].y) * down,
                          bf16_hi(raw[i].y) * down};
      uint32_t h[2], l[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) split_e4m3(a[2 * k], a[2 * k + 1], h[k], l[k]);
      uint8_t* dst = tile + (r0 + i) * 128 + to + ((tc ^ ((r0 + i) & 7)) << 4);
      *reinterpret_cast<uint32_t*>(dst) = h[0] | h[1] << 16;
      *reinterpret_cast<uint32_t*>(dst + kHalf) = l[0] | l[1] << 16;
      if (lane == i) scales[r0 + i] = __uint_as_float((uint32_t)(127 + e) << 23) * scale_log2;
    }
  }
}

// kRun: columns that surely share a block's scales, 8 or 16 (fewer loads and
// factors: 3 % of a verify batch).
template <int kRun>
__global__ void __launch_bounds__(kThreads, 1) mma_fp8block_kernel(const AttnParams p,
                                                                   const __grid_constant__ CUtensorMap qmap,
                                                                   const __grid_constant__ CUtensorMap kmap,
                                                                   const __grid_constant__ CUtensorMap vmap,
                                                                   const __grid_constant__ CUtensorMap omap) {
  constexpr int D = 128;
  constexpr int kOC = D / 2;  // output columns per softmax thread
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // uniform: every thread returns before any barrier
    if (threadIdx.x == 0) raise_error(p.err, PKV_DEVERR_INTERNAL);
    return;
  }
  Bars* bars = reinterpret_cast<Bars*>(smem + kBarOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kBarOff + kNumBars * 8);
  ItemSlot* slots = reinterpret_cast<ItemSlot*>(smem + kSlotOff);
  float* row_scales = reinterpret_cast<float*>(smem + kRowScaleOff);      // [2][128], times the logit scale
  Scales* tile_scales = reinterpret_cast<Scales*>(smem + kScaleOff);      // [kScaleSlots][16 runs of 8 keys]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WaitCtl wc{p.err, wait_limit(p.wait_ns)};

  if (threadIdx.x == 0) {
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars->q_full[b], 1);
      mbar_init(&bars->q_split[b], kSplitters);
      mbar_init(&bars->q_empty[b], 1);
      mbar_init(&bars->slot_full[b], 32);
      mbar_init(&bars->slot_free[b], kSlotReaders);
      mbar_init(&bars->s_full[b], 1);
      mbar_init(&bars->s_free[b], 256);
      mbar_init(&bars->pv_done[b], 1);
      mbar_init(&bars->p_full[b], 256);
    }
    for (int s = 0; s < kKStages; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->k_empty[s], 1);
    }
    for (int s = 0; s < kVStages; ++s) {
      mbar_init(&bars->c_full[s], 1);
      mbar_init(&bars->c_empty[s], kConverters);
      mbar_init(&bars->v_full[s], kConverters);
    }
    for (int s = 0; s < kScaleSlots; ++s) mbar_init(&bars->sc_full[s], 1);
    mbar_init(&bars->o_empty, 256);
    mbar_init(&bars->o_staged[0], 256);
    mbar_init(&bars->o_staged[1], 256);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();  // the plan and the K/V write are complete and visible from here on
  const int n_items = p.header->n_mma;
  // CTAs past the plan's mma_ctas leave their SMs to the decode kernel, which
  // may start once every CTA here has seen the plan (signalled just below)
  const bool active = blockIdx.x < p.header->mma_ctas;
  pdl_launch_dependents();
  const uint32_t tmem = *tmem_slot;
  const uint32_t smem_base = smem_u32(smem);

  // One counter g numbers the key tiles this CTA processes (across items): K
  // stage g % 3 (parity (g / 3) & 1), V stage g % 2 (parity (g / 2) & 1), S
  // and P buffer g % 2.  Item c of this CTA uses Q tile and slot c & 1
  // (parity (c >> 1) & 1); O's phases count items.
  const int nb = kKeys / p.bs;  // physical blocks per tile
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

  // The branches below are per warpgroup first (the register split is a
  // warpgroup-wide instruction), then per warp.
  if (!active) {
    // nothing: straight to the teardown
  } else if (warp < 4 || warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLight));
    if (warp == 14) {
      // ================================================================ item fetch, Q, output stores
      if (lane == 0) {
        prefetch_tensormap(&qmap);
        prefetch_tensormap(&omap);
      }
      // where the output tile staged in Q buffer b goes: token and head
      // coordinates of its TMA stores, token -1 when the epilogue wrote it itself
      int otok0 = -1, otok1 = -1, ohead0 = 0, ohead1 = 0;
      auto store_staged = [&](int ci) -> bool {  // item ci's output, once its epilogue is done
        const int b = ci & 1;
        if (!__all_sync(0xffffffffu, mbar_wait(&bars->o_staged[b], (ci >> 1) & 1, wc))) return false;
        const int tok = b ? otok1 : otok0, head = b ? ohead1 : ohead0;
        if (lane == 0 && tok >= 0) {
          tma_store_3d(&omap, smem + kQOff + b * kQBytes, 0, head, tok);
          tma_store_3d(&omap, smem + kQOff + b * kQBytes + kHalf, 64, head, tok);
          bulk_commit_group();
          bulk_wait_read_all();  // the buffer may take the next Q tile
        }
        __syncwarp();
        return true;
      };
      int c = 0, q_last = -1;  // the last item whose Q tile was loaded
      bool ok = true;
      for (;; ++c) {
        const int qb = c & 1;
        // Item c is taken from the queue once item c-2's last Q K^T is
        // complete (Q tile qb free) and every reader has taken item c-2's
        // description (slot qb free): while item c-2 ends, item c-1 waits
        // with its Q loaded.  Taking items no earlier keeps the queue's
        // largest-first order close to the order in which the SMs fall idle,
        // which is what keeps the tail short.
        if (!__all_sync(0xffffffffu, mbar_wait(&bars->q_empty[qb], ((c >> 1) & 1) ^ 1, wc) &&
                                         mbar_wait(&bars->slot_free[qb], ((c >> 1) & 1) ^ 1, wc))) {
          ok = false;
          break;
        }
        int idx = 0;
        if (lane == 0) idx = atomicAdd(p.counter, 1);
        idx = __shfl_sync(0xffffffffu, idx, 0);
        const bool done = idx >= n_items;
        ItemSlot& sl = slots[qb];
        WorkItem it{};
        int qstart = 0;
        if (done) {
          if (lane == 0) sl.done = 1;
        } else {
          it = p.items[idx];
          const int L = p.context_lens[it.seq];
          qstart = p.query_start_loc[it.seq];
          const int n = p.query_start_loc[it.seq + 1] - qstart;
          const int nblk = (L + p.bs - 1) / p.bs;
          int at = 0, len = 0;
          if (p.window > 0) {
            const Hole hole(L, n, it.row0 / p.G, p.window, p.num_sink, p.bs);
            at = hole.at;
            len = hole.len;
          }
          const int32_t* bt = p.block_tables + (int64_t)it.seq * p.max_blocks;
          const int tile = it.kb + (lane >> 4) * kKeys;
          int phys = (int)p.num_blocks;
          if ((lane & 15) < nb && tile < it.ke) phys = block_of(bt, nblk, at, len, tile + (lane & 15) * p.bs);
          sl.phys[lane] = phys;
          float2 sc = make_float2(1.f, 1.f);
          if (lane < nb && phys < p.num_blocks) {
            const int64_t i = (int64_t)phys * p.Hkv + it.kvh;
            sc = make_float2(__ldg(p.k_scales + i), __ldg(p.v_scales + i));
          }
          if (lane < 16) sl.scales[lane] = sc;
          if (lane == 0) {
            sl.it = it;
            sl.L = L - len;
            sl.qstart = qstart;
            sl.n = n;
            sl.nblk = nblk;
            sl.at = at;
            sl.len = len;
            sl.done = 0;
          }
        }
        mbar_arrive(&bars->slot_full[qb]);  // every lane, after its own writes (count 32)
        // Q tile qb: item c-2's output, staged there by its epilogue, read out
        if (c >= 2 && !store_staged(c - 2)) {
          ok = false;
          break;
        }
        if (done) {
          if (lane == 0) mbar_arrive(&bars->q_full[qb]);
          break;
        }
        // a full tile of whole tokens, not a split: its epilogue stages the output
        const int tok = (it.nrows == p.mma_unit_rows && it.part < 0) ? qstart + it.row0 / p.G : -1;
        if (qb) {
          otok1 = tok;
          ohead1 = it.kvh * p.G;
        } else {
          otok0 = tok;
          ohead0 = it.kvh * p.G;
        }
        if (lane == 0) {
          // the Q box: {64, G, floor(128 / G)} (whole tokens, up to 128 rows)
          mbar_arrive_expect_tx(&bars->q_full[qb], 2 * 128 * (kMmaRows / p.G) * p.G);
          const int tok0 = qstart + it.row0 / p.G;
          tma_load_3d(smem + kQOff + qb * kQBytes, &qmap, &bars->q_full[qb], 0, it.kvh * p.G, tok0);
          tma_load_3d(smem + kQOff + qb * kQBytes + kHalf, &qmap, &bars->q_full[qb], 64, it.kvh * p.G, tok0);
        }
        q_last = c;
      }
      if (ok && c >= 1) store_staged(c - 1);  // the last item's output
      // leaving early: the last Q tile's copy must have landed before the CTA exits
      if (!ok && q_last >= 0) __all_sync(0xffffffffu, mbar_wait(&bars->q_full[q_last & 1], (q_last >> 1) & 1, wc));
      if (lane == 0) bulk_wait_all();
    } else if (warp == 2 || warp == 12) {
      // ================================================================ K / V producers
      const bool is_v = warp == 12;
      const CUtensorMap* map = is_v ? &vmap : &kmap;
      if (lane == 0) prefetch_tensormap(map);
      const int run_block = (lane & 15) * 8 / p.bs;  // block of the tile's run of 8 keys that this lane writes the scales of
      const int nst = is_v ? kVStages : kKStages;
      uint8_t* const ring = smem + (is_v ? kCOff : kKOff);
      uint64_t* const fullb = is_v ? bars->c_full : bars->k_full;
      uint64_t* const emptyb = is_v ? bars->c_empty : bars->k_empty;
      int g = 0;
      bool ok = true;
      for (int c = 0; ok; ++c) {
        const int qb = c & 1;
        if (!__all_sync(0xffffffffu, mbar_wait(&bars->slot_full[qb], (c >> 1) & 1, wc))) {
          ok = false;
          break;
        }
        const ItemSlot& sl = slots[qb];
        const bool done = sl.done != 0;
        const int kb = sl.it.kb, ke = sl.it.ke, kvh = sl.it.kvh, nblk = sl.nblk, at = sl.at, len = sl.len;
        const int32_t* bt = p.block_tables + (int64_t)sl.it.seq * p.max_blocks;
        int phys = sl.phys[lane & 15], next = sl.phys[16 + (lane & 15)];
        float2 sc = sl.scales[lane & 15];
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->slot_free[qb]);
        if (done) break;
        for (int kbase = kb; kbase < ke; kbase += kKeys, ++g) {
          const int st = g % nst, ph = (g / nst) & 1;
          // the ids of the tile after the next, the scales of the next
          int after = (int)p.num_blocks;
          if (lane < nb && kbase + 2 * kKeys < ke) after = block_of(bt, nblk, at, len, kbase + 2 * kKeys + lane * p.bs);
          float2 nsc = make_float2(1.f, 1.f);
          if (!is_v && lane < nb && kbase + kKeys < ke && next < p.num_blocks) {
            const int64_t i = (int64_t)next * p.Hkv + kvh;
            nsc = make_float2(__ldg(p.k_scales + i), __ldg(p.v_scales + i));
          }
          // K stage g % 3 is free once Q K^T(g-3) is complete; V's codes once converted
          if (!__all_sync(0xffffffffu, mbar_wait(&emptyb[st], ph ^ 1, wc))) {
            ok = false;
            break;
          }
          if (!is_v) {
            // the slot's last reader was tile g-8's softmax: Q K^T(g-3) was issued after S(g-5) was read
            const float2 mine = make_float2(__shfl_sync(0xffffffffu, sc.x, run_block), __shfl_sync(0xffffffffu, sc.y, run_block));
            if (lane < 16) tile_scales[(g & (kScaleSlots - 1)) * 16 + lane] = make_scales<kWeightExp>(mine);
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->sc_full[g & (kScaleSlots - 1)]);
          }
          if (lane == 0) mbar_arrive_expect_tx(&fullb[st], kCodeTile);
          __syncwarp();
          // testing only: one CTA's K of tile fault_tile - 1 is never loaded, so the waits for it run out
          const bool skip = p.fault_tile == g + 1 && !is_v && blockIdx.x == 0;
          if (lane < nb && !skip) tma_load_4d(ring + st * kCodeTile + lane * p.bs * 128, map, &fullb[st], 0, kvh, 0, phys);
          phys = next;
          next = after;
          sc = nsc;
        }
      }
      // leaving: the copies of the tiles issued last land first, whoever still waits for them
      for (int j = max(0, g - nst); j < g; ++j) __all_sync(0xffffffffu, mbar_wait(&fullb[j % nst], (j / nst) & 1, wc));
    } else if (warp >= 16) {
      // ================================================================ V converters
      // Codes (rows of 128 bytes, chunk j at j ^ (key & 7)) become an fp16 tile of
      // two 64-column halves, swizzled alike; rows past the sequence's end, and
      // those before every row's window, become zeros whatever they hold.
      // A thread takes one chunk of every sixteenth key, so that its places within a
      // tile are 2048 bytes apart.
      const int t = (warp - 16) * 32 + lane;
      const int ch = t & 7, x = (t >> 3) & 7, row = (t >> 3) * 128;
      const int from = row + ((ch ^ x) << 4);
      const int to = (ch >> 2) * kHalfKV + row;
      const int to0 = to + (((2 * (ch & 3)) ^ x) << 4), to1 = to + (((2 * (ch & 3) + 1) ^ x) << 4);
      int g = 0;
      bool ok = true;
      for (int c = 0; ok; ++c) {
        const int qb = c & 1;
        if (!__all_sync(0xffffffffu, mbar_wait(&bars->slot_full[qb], (c >> 1) & 1, wc))) break;
        const ItemSlot& sl = slots[qb];
        const bool done = sl.done != 0;
        const int kb = sl.it.kb, ke = sl.it.ke, L = sl.L;
        const int lo = p.window > 0 ? L - sl.n + sl.it.row0 / p.G + 1 - p.window : INT_MIN;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->slot_free[qb]);
        if (done) break;
        for (int kbase = kb; kbase < ke; kbase += kKeys, ++g) {
          const int st = g % kVStages, ph = (g / kVStages) & 1;
          // the codes landed; the fp16 tile is free: P.V(g-2) is complete
          if (!__all_sync(0xffffffffu, mbar_wait(&bars->c_full[st], ph, wc) &&
                                           mbar_wait(&bars->pv_done[st], ph ^ 1, wc))) {
            ok = false;
            break;
          }
          const uint8_t* src = smem + kCOff + st * kCodeTile + from;
          uint8_t* dst = smem + kVOff + st * kTileBytes;
          const bool masked = kbase + kKeys > L || (kbase < lo && kbase + kKeys > p.num_sink);
#pragma unroll 1
          for (int i0 = 0; i0 < kKeys / 16; i0 += 4) {  // keys t / 8 + 16 i
            uint4 raw[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) raw[i] = *reinterpret_cast<const uint4*>(src + (i0 + i) * 2048);
            if (masked) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int k = kbase + (t >> 3) + 16 * (i0 + i);
                if (k >= L || (k < lo && k >= p.num_sink)) raw[i] = make_uint4(0, 0, 0, 0);
              }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t in[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
              uint32_t w[8];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                w[2 * e] = e4m3x2_to_f16x2(in[e] & 0xFFFFu);
                w[2 * e + 1] = e4m3x2_to_f16x2(in[e] >> 16);
              }
              *reinterpret_cast<uint4*>(dst + to0 + (i0 + i) * 2048) = make_uint4(w[0], w[1], w[2], w[3]);
              *reinterpret_cast<uint4*>(dst + to1 + (i0 + i) * 2048) = make_uint4(w[4], w[5], w[6], w[7]);
            }
          }
          fence_proxy_async_smem();  // generic-proxy writes, read by the tensor core
          mbar_arrive(&bars->v_full[st]);
          mbar_arrive(&bars->c_empty[st]);
        }
      }
    } else if (warp == 3 || warp == 13 || warp == 15) {
      // ================================================================ Q split
      const int part = warp == 3 ? 0 : warp == 13 ? 1 : 2;
      for (int c = 0;; ++c) {
        const int qb = c & 1;
        if (!__all_sync(0xffffffffu, mbar_wait(&bars->slot_full[qb], (c >> 1) & 1, wc))) break;
        const bool done = slots[qb].done != 0;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->slot_free[qb]);
        if (done) break;
        if (!__all_sync(0xffffffffu, mbar_wait(&bars->q_full[qb], (c >> 1) & 1, wc))) break;
        // rows 44 part .. (40 for the last)
        split_rows(smem + kQOff + qb * kQBytes, 44 * part, min(44 * part + 44, kMmaRows), row_scales + qb * kMmaRows,
                   p.scale_log2, lane);
        fence_proxy_async_smem();  // generic-proxy writes, read by the tensor core
        mbar_arrive(&bars->q_split[qb]);
      }
    } else if (warp == 1) {
      // ================================================================ Q K^T issuer
      if (lane == 0) {
        const uint64_t dq = desc_k(smem_base + kQOff);
        const uint64_t dk0 = desc_k(smem_base + kKOff);
        int gs = 0, s_item = -1, s_j = 0, s_nt = 0;
        bool ok = true;
        for (;;) {
          if (s_j == s_nt) {  // next item: its slot written, its Q tile split
            ++s_item;
            const int qb = s_item & 1;
            if (!mbar_wait(&bars->slot_full[qb], (s_item >> 1) & 1, wc)) {
              ok = false;
              break;
            }
            const bool done = slots[qb].done != 0;
            const int nt = (slots[qb].it.ke - slots[qb].it.kb + kKeys - 1) / kKeys;
            mbar_arrive(&bars->slot_free[qb]);
            if (done) break;
            if (!mbar_wait(&bars->q_split[qb], (s_item >> 1) & 1, wc)) {
              ok = false;
              break;
            }
            s_nt = nt;
            s_j = 0;
          }
          const int sb = gs & 1, st = gs % kKStages;
          // S buffer sb: the softmax warps have read S(gs-2) from it; K(gs) loaded
          const uint32_t kph = (gs / kKStages) & 1;
          if (!mbar_wait(&bars->s_free[sb], ((gs >> 1) & 1) ^ 1, wc) || !mbar_wait(&bars->k_full[st], kph, wc)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t dqb = desc_add(dq, (s_item & 1) * kQBytes);
          const uint64_t dk = desc_add(dk0, st * kCodeTile);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)  // q1's four steps of 32 columns, then q2's
            umma_f8(tmem + kSCol + 128 * sb, desc_add(dqb, (kk >> 2) * kHalf + (kk & 3) * 32),
                    desc_add(dk, (kk & 3) * 32), kIdescS, kk > 0 ? 1u : 0u);
          umma_commit(&bars->s_full[sb]);
          umma_commit(&bars->k_empty[st]);
          if (s_j == s_nt - 1) umma_commit(&bars->q_empty[s_item & 1]);  // Q no longer read by this item
          ++s_j;
          ++gs;
        }
        // leaving early: the S MMAs already issued finish before TMEM is freed
        if (!ok && gs > 0) mbar_wait(&bars->s_full[(gs - 1) & 1], ((gs - 1) >> 1) & 1, wc);
      }
      __syncwarp();
    } else if (warp == 0) {
      // ================================================================ P.V issuer
      if (lane == 0) {
        const uint64_t dv0 = desc_v(smem_base + kVOff);
        int gp = 0;
        bool ok = true;
        for (int c = 0; ok; ++c) {
          const int qb = c & 1;
          if (!mbar_wait(&bars->slot_full[qb], (c >> 1) & 1, wc)) {
            ok = false;
            break;
          }
          const bool done = slots[qb].done != 0;
          const int nt = (slots[qb].it.ke - slots[qb].it.kb + kKeys - 1) / kKeys;
          mbar_arrive(&bars->slot_free[qb]);
          if (done) break;
          // O is about to be overwritten: item c-1's epilogue must have read it
          if (!mbar_wait(&bars->o_empty, (c & 1) ^ 1, wc)) {
            ok = false;
            break;
          }
          for (int j = 0; j < nt; ++j, ++gp) {
            const int pb = gp & 1, vst = gp % kVStages;
            // P(gp) written, V(gp) converted
            const uint32_t vph = (gp / kVStages) & 1;
            if (!mbar_wait(&bars->p_full[pb], (gp >> 1) & 1, wc) || !mbar_wait(&bars->v_full[vst], vph, wc)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t dv = desc_add(dv0, vst * kTileBytes);
  #pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk)
              umma_bf16_ts(tmem + kOCol, tmem + kPCol + 64 * pb + kk * 8, desc_add(dv, kk * 2048), kIdescO,
                           (j == 0 && kk == 0) ? 0u : 1u);
            umma_commit(&bars->pv_done[pb]);  // P.V(gp) complete: frees P buffer and V stage gp % 2
          }
        }
        // leaving early: the P.V MMAs already issued finish before TMEM is freed
        if (!ok && gp > 0) mbar_wait(&bars->pv_done[(gp - 1) & 1], ((gp - 1) >> 1) & 1, wc);
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // ================================================================ softmax / epilogue
    const int q4 = warp & 3;
    const int h = (warp - 4) >> 2;  // key half of a tile (columns 64h .. 64h+63); output half 64h .. 64h+63
    const int r = q4 * 32 + lane;   // row of the tile == TMEM lane
    const int pair_bar = 1 + q4;    // warps (w, w+4) of one row quarter
    const uint32_t lane_base = tmem + ((uint32_t)(q4 * 32) << 16);
    float* red = reinterpret_cast<float*>(smem + kRedOff);
    // A failed wait (warp-uniform) ends the warp's work on the item at once;
    // it then takes the pair barriers the item still owes its partner
    // (ntiles + 2 per item in all), so the partner never waits for a warp
    // that left: the partner finishes the item, or gives up in turn when a
    // wait of its own runs out.  All 8 warps then agree at an OR-reducing
    // barrier (id 6)
    // that each reaches once at the end of every item: there they all go on
    // to the stores, or all leave.
    int g = 0;
    for (int c = 0;; ++c) {
      const int qb = c & 1;
      if (barrier_any(6, 256, !__all_sync(0xffffffffu, mbar_wait(&bars->slot_full[qb], (c >> 1) & 1, wc)))) break;
      const ItemSlot& sl = slots[qb];
      const bool done = sl.done != 0;
      const WorkItem it = sl.it;
      const int L = sl.L, qstart = sl.qstart, n = sl.n;
      mbar_arrive(&bars->slot_free[qb]);
      if (done) break;
      const bool valid = r < it.nrows;
      const int row = it.row0 + r;
      const int tok = row / p.G, gh = row - tok * p.G;
      // rows past the item's are left as they come: their logits are 0 (or NaN), in no other row's way
      const int vis = valid ? min(it.ke, p.causal ? L - n + tok + 1 : L) : INT_MAX;
      const bool idle = q4 * 32 >= it.nrows;  // none of the warp's rows is the item's
      if (barrier_any(6, 256, !__all_sync(0xffffffffu, mbar_wait(&bars->q_split[qb], (c >> 1) & 1, wc)))) break;
      // of this row's accumulator, in log2 units; times any K scale not 0 (split_rows)
      const float unit = valid ? row_scales[qb * kMmaRows + r] : 0.f;
      float m_ref = -CUDART_INF_F, l = 0.f;
      int owe = -1;  // after a failed wait: the pair barriers of the item not yet taken
      const int ntiles = (it.ke - it.kb + kKeys - 1) / kKeys;
      for (int j = 0; j < ntiles; ++j, ++g) {
        const int sb = g & 1;
        const int kt = it.kb + j * kKeys;  // first key of the tile
        const uint32_t s_half = lane_base + kSCol + 128 * sb + 64 * h, p_half = lane_base + kPCol + 64 * sb + 32 * h;
        // S(g), the P buffer free (the P.V of tile g-2, which read it, done), the
        // tile's scales; all three at once where they are there
        uint64_t* const scb = &bars->sc_full[g & (kScaleSlots - 1)];
        const uint32_t ph = (g >> 1) & 1, scph = (g / kScaleSlots) & 1;
        if (!__all_sync(0xffffffffu, mbar_test_wait3(&bars->s_full[sb], ph, &bars->pv_done[sb], ph ^ 1, scb, scph)) &&
            !__all_sync(0xffffffffu, mbar_wait(&bars->s_full[sb], ph, wc) && mbar_wait(&bars->pv_done[sb], ph ^ 1, wc) &&
                                         mbar_wait(scb, scph, wc))) {
          owe = (idle ? 0 : ntiles - j) + 2;
          break;
        }
        if (idle) {  // nothing to do but keep the tiles' pace (its partner is as idle: they meet at the item's end)
          mbar_arrive(&bars->s_free[sb]);
          mbar_arrive(&bars->p_full[sb]);
          continue;
        }
        tc_fence_after();
        // The keys of this half that the row sees, as bits: c < nvis and, with a
        // window, not nsink <= c < nlo.
        const int nvis = vis - (kt + 64 * h);
        const int nlo = p.window > 0 && valid ? L - n + tok + 1 - p.window - (kt + 64 * h) : 0;
        uint64_t seen = ~0ull;
        const bool masked = __any_sync(0xffffffffu, nvis < 64 || nlo > 0);
        if (masked) {
          auto below = [](int k) { return k <= 0 ? 0ull : k >= 64 ? ~0ull : (1ull << k) - 1; };  // bits c < k
          seen = below(nvis) & (below(p.num_sink - (kt + 64 * h)) | ~below(nlo));
        }
        const Scales* scales = tile_scales + (g & (kScaleSlots - 1)) * 16 + 8 * h;
        // S is read twice, 32 columns at a time, in loops: the code unrolled over a row's
        // 64 columns did not fit the instruction cache beside the other roles' code.
        auto columns = [&](int run, uint32_t (&z)[16]) {  // masked: columns 8 run .. + 15
          if (masked) {
            const uint32_t m = (uint32_t)(seen >> (8 * run));
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (!((m >> i) & 1)) z[i] = __float_as_uint(-CUDART_INF_F);
          }
        };
        // this half's max of x + log2 sv: factors are positive, so of each run the largest S
        float mloc = -CUDART_INF_F;
        auto max_of = [&](int run, uint32_t (&z)[16]) {
          columns(run, z);
          auto at = [&](int i) { return __uint_as_float(z[i]); };
          float t0 = fmax3(fmax3(at(0), at(1), at(2)), fmax3(at(3), at(4), at(5)), fmaxf(at(6), at(7)));
          float t1 = fmax3(fmax3(at(8), at(9), at(10)), fmax3(at(11), at(12), at(13)), fmaxf(at(14), at(15)));
          const Scales sc = scales[run];
          if constexpr (kRun == 8) {
            const Scales sd = scales[run + 1];
            mloc = fmax3(mloc, fmaf(t0, unit * sc.k, sc.log_v), fmaf(t1, unit * sd.k, sd.log_v));
          } else {
            mloc = fmaxf(mloc, fmaf(fmaxf(t0, t1), unit * sc.k, sc.log_v));
          }
        };
        // P of keys 64h .. 64h+63: 2^(x + log2 sv - m + 7), fp16 pairs (TMEM
        // columns 32h .. 32h+31 of P buffer sb); ps the sum of 2^(x - m)
        float ps = 0.f, nm = 0.f;
        auto exps_of = [&](int run, uint32_t (&z)[16]) {
          columns(run, z);
          uint32_t pk[8];
#pragma unroll
          for (int half = 0; half < 16 / kRun; ++half) {
            const Scales sc = scales[run + half];
            const float u = unit * sc.k, b = nm + sc.log_v;
            const f32x2 u2 = pk2(u, u), b2 = pk2(b, b);
            f32x2 sum = pk2(0.f, 0.f);
#pragma unroll
            for (int i = 4 * half; i < 4 * half + kRun / 2; ++i) {
              const float2 x = up2(fma2(pk2(__uint_as_float(z[2 * i]), __uint_as_float(z[2 * i + 1])), u2, b2));
              const float e0 = fast_exp2(x.x), e1 = fast_exp2(x.y);
              sum = add2(sum, pk2(e0, e1));
              pk[i] = pack_half(e0, e1);
            }
            const float2 s2 = up2(sum);
            ps = fmaf(s2.x + s2.y, sc.inv_v, ps);
          }
          tmem_st8(p_half + 4 * run, pk);
        };
        auto each = [&](auto&& use) {  // use(run, columns 8 run .. + 15 of this half's S)
          uint32_t a[16], b[16];
#pragma unroll 1
          for (int run = 0; run < 8; run += 4) {
            tmem_ld16(s_half + 8 * run, a);
            tmem_ld16(s_half + 8 * run + 16, b);
            tmem_wait_ld();
            use(run, a);
            use(run + 2, b);
          }
        };
        each(max_of);
        float* redm = red + sb * 256;
        redm[h * 128 + r] = mloc;
        named_barrier(pair_bar, 64);
        // the running reference rises where the row's max exceeds it by the threshold
        const float mx = fmaxf(mloc, redm[(h ^ 1) * 128 + r]);
        float alpha = 1.f;
        bool rescale = false;
        if (mx > m_ref + kRescaleThreshold) {  // false while both are -inf
          alpha = fast_exp2(m_ref - mx);       // 0 when m_ref is -inf
          rescale = m_ref != -CUDART_INF_F;
          m_ref = mx;
        }
        nm = (m_ref == -CUDART_INF_F ? 0.f : -m_ref) + kWeightExp;
        __syncwarp();
        each(exps_of);
        tc_fence_before();
        mbar_arrive(&bars->s_free[sb]);  // S buffer sb may take S(g+2)
        l = fmaf(l, alpha, ps);
        if (__any_sync(0xffffffffu, rescale)) {
          // O must hold every earlier tile's P.V before it is scaled; the TMEM
          // accesses are warp-wide, rows that keep their max scale by 1
          // P.V(g-1) complete
          if (!__all_sync(0xffffffffu, mbar_wait(&bars->pv_done[sb ^ 1], ((g - 1) >> 1) & 1, wc))) {
            owe = ntiles - j + 1;
            break;
          }
          tc_fence_after();
          const float f = rescale ? alpha : 1.f;
#pragma unroll 1
          for (int cc = 0; cc < kOC; cc += 16) {
            uint32_t o[16];
            tmem_ld16(lane_base + kOCol + kOC * h + cc, o);
            tmem_wait_ld();
#pragma unroll
            for (int t = 0; t < 16; ++t) o[t] = __float_as_uint(__uint_as_float(o[t]) * f);
            tmem_st16(lane_base + kOCol + kOC * h + cc, o);
          }
        }
        tmem_wait_st();  // P (and a rescaled O) written
        tc_fence_before();
        mbar_arrive(&bars->p_full[sb]);
      }
      // ---- epilogue: row sum of the pair, O (this thread's 64 output columns) / l.
      // The sums go through the max buffer the last tile did not use; the
      // second pair barrier keeps the next tile from overwriting them early.
      float ltot = 0.f;
      if (owe < 0) {
        float* reds = red + (g & 1) * 256;
        reds[h * 128 + r] = l;
        named_barrier(pair_bar, 64);
        ltot = l + reds[(h ^ 1) * 128 + r];
        named_barrier(pair_bar, 64);
        // P.V of the item's last tile (g-1) complete
        if (!__all_sync(0xffffffffu, mbar_wait(&bars->pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1, wc))) owe = 0;
      }
      for (int k = 0; k < owe; ++k) named_barrier(pair_bar, 64);
      if (barrier_any(6, 256, owe >= 0)) break;
      tc_fence_after();
      // a full tile of whole tokens leaves through TMA stores from Q buffer qb
      // (its Q K^T are complete), in the Q tile's layout: row r, 16-byte
      // chunk j at chunk j ^ (r & 7) of the row (128-byte swizzle); this
      // thread's columns are half h
      const bool staged = it.nrows == p.mma_unit_rows && it.part < 0;
      // a partial row keeps 2^-7 of its accumulator, a finished one its share of the row's sum
      const float inv = (1.f / (1 << kWeightExp)) / (it.part < 0 ? ltot : 1.f);
      __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(p.out) +
                            ((int64_t)(qstart + tok) * p.Hq + (int64_t)it.kvh * p.G + gh) * D + kOC * h;
      float* prow = p.part_acc + (int64_t)(it.part + r) * D + kOC * h;  // (the workspace is 256-byte aligned)
      uint8_t* srow = smem + kQOff + qb * kQBytes + h * kHalf + r * 128;
#pragma unroll 1
      for (int cc = 0; cc < kOC; cc += 16) {
        uint32_t o[16];
        __syncwarp();  // (the rows part below; TMEM loads are the whole warp's)
        tmem_ld16(lane_base + kOCol + kOC * h + cc, o);
        tmem_wait_ld();
        if (!valid) continue;
#pragma unroll
        for (int t = 0; t < 16; ++t) o[t] = __float_as_uint(__uint_as_float(o[t]) * inv);
        if (it.part >= 0) {
          st_global_v8(prow + cc, o);
          st_global_v8(prow + cc + 8, o + 8);
          continue;
        }
        uint32_t w[8];
#pragma unroll
        for (int t = 0; t < 8; ++t) w[t] = pack_bf16(__uint_as_float(o[2 * t]), __uint_as_float(o[2 * t + 1]));
        if (staged) {
          *reinterpret_cast<uint4*>(srow + (((cc >> 3) ^ (r & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
          *reinterpret_cast<uint4*>(srow + ((((cc >> 3) + 1) ^ (r & 7)) << 4)) = make_uint4(w[4], w[5], w[6], w[7]);
        } else {
          store_row<16>(orow + cc, w, p.out_al32);
        }
      }
      __syncwarp();
      tc_fence_before();
      mbar_arrive(&bars->o_empty);
      if (valid && it.part >= 0 && h == 0) p.part_ml[it.part + r] = make_float2(m_ref, ltot);
      if (staged) fence_proxy_async_smem();  // the staged rows, for the TMA stores
      mbar_arrive(&bars->o_staged[qb]);
      if (it.grp >= 0) {
        // The split that completes its merge group combines the group's
        // partial rows: m = max m_p, l = sum l_p 2^(m_p - m), O = sum acc_p 2^(m_p - m) / l.
        // Release: the barrier orders every thread's partial writes before one
        // thread's fence and ticket; acquire: that thread's fence, then the barrier.
        int* flag_last = reinterpret_cast<int*>(tmem_slot + 1);
        named_barrier(5, 256);
        if (r == 0 && h == 0) {
          __threadfence();
          *flag_last = atomicAdd(p.tickets + it.grp, 1);
        }
        named_barrier(5, 256);
        const MergeGroup gr = p.groups[it.grp];
        if (*flag_last == gr.nsplit - 1) {
          if (r == 0 && h == 0) __threadfence();
          named_barrier(5, 256);
          // a warp takes four rows at a time, a lane four columns (a thread's own half row,
          // 16 columns at a time, was a longer chain of reads: 128 queries on 60000 keys
          // 199 us against 191)
          constexpr int kAt = 4;
#pragma unroll 1
          for (int r0 = kAt * (warp - 4); r0 < gr.nrows; r0 += kAt * 8) {
            const float2* ml = p.part_ml + gr.part_base + r0;
            const float* acc = p.part_acc + (int64_t)(gr.part_base + r0) * D + 4 * lane;
            const int live = min(kAt, gr.nrows - r0);
            float m[kAt], lsum[kAt];
            float4 o[kAt];
#pragma unroll
            for (int i = 0; i < kAt; ++i) {
              m[i] = -CUDART_INF_F;
              lsum[i] = 0.f;
              o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll 2
            for (int sp = 0; sp < gr.nsplit; ++sp) {
#pragma unroll
              for (int i = 0; i < kAt; ++i)
                if (i < live) m[i] = fmaxf(m[i], __ldcg(ml + sp * gr.nrows + i).x);
            }
#pragma unroll
            for (int i = 0; i < kAt; ++i)
              if (m[i] == -CUDART_INF_F) m[i] = 0.f;
#pragma unroll 2
            for (int sp = 0; sp < gr.nsplit; ++sp) {
#pragma unroll
              for (int i = 0; i < kAt; ++i) {
                if (i < live) {
                  const float2 a = __ldcg(ml + sp * gr.nrows + i);
                  const float4 x = __ldcg(reinterpret_cast<const float4*>(acc + (int64_t)(sp * gr.nrows + i) * D));
                  const float w = fast_exp2(a.x - m[i]);
                  lsum[i] = fmaf(w, a.y, lsum[i]);
                  o[i].x = fmaf(w, x.x, o[i].x);
                  o[i].y = fmaf(w, x.y, o[i].y);
                  o[i].z = fmaf(w, x.z, o[i].z);
                  o[i].w = fmaf(w, x.w, o[i].w);
                }
              }
            }
#pragma unroll
            for (int i = 0; i < kAt; ++i) {
              if (i < live) {
                const float minv = 1.f / lsum[i];
                const int grow = gr.row0 + r0 + i, gtok = grow / p.G, ggh = grow - gtok * p.G;
                __nv_bfloat16* mrow = static_cast<__nv_bfloat16*>(p.out) +
                                      ((int64_t)(qstart + gtok) * p.Hq + (int64_t)gr.kvh * p.G + ggh) * D;
                reinterpret_cast<uint2*>(mrow)[lane] =
                    make_uint2(pack_bf16(o[i].x * minv, o[i].y * minv), pack_bf16(o[i].z * minv, o[i].w * minv));
              }
            }
          }
        }
        named_barrier(5, 256);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

template <int kRun>
cudaError_t launch_t(const AttnParams& p, const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap,
                     const CUtensorMap& omap, int grid, cudaStream_t s) {
  static unsigned long long done_mask = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!(__atomic_load_n(&done_mask, __ATOMIC_ACQUIRE) & (1ull << dev))) {
    // the register split needs the block launched with kRegs registers per thread
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, mma_fp8block_kernel<kRun>);
    if (e != cudaSuccess) return e;
    if (fa.numRegs != kRegs) return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(mma_fp8block_kernel<kRun>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    __atomic_fetch_or(&done_mask, 1ull << dev, __ATOMIC_RELEASE);
  }
  if (p.no_wait) {  // beside the few-row kernel: a plain launch, as the bf16 kernel's
    mma_fp8block_kernel<kRun><<<dim3(grid), dim3(kThreads), kSmem, s>>>(p, qmap, kmap, vmap, omap);
    e = cudaGetLastError();
  } else {
    e = launch_pdl(mma_fp8block_kernel<kRun>, dim3(grid), dim3(kThreads), kSmem, s, p, qmap, kmap, vmap, omap);
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_mma_fp8block(const AttnParams& p, const CUtensorMap& qmap, const CUtensorMap& kmap,
                                const CUtensorMap& vmap, const CUtensorMap& omap, int grid, cudaStream_t s) {
  return p.bs >= 16 ? launch_t<16>(p, qmap, kmap, vmap, omap, grid, s)
                    : launch_t<8>(p, qmap, kmap, vmap, omap, grid, s);
}

}  // namespace pkv
