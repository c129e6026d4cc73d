// Attention weight paid to each cached token, for sequences of many rows
// (prefill chunks, observation windows, wide verify steps) of bf16 queries,
// over bf16 or FP8 pools: tcgen05.mma with TMEM accumulators.
// paged_attention_scores (scores.cu) plans the work; this kernel does both
// passes over the keys.
//
// With z[r][j] = scale * log2(e) * q_r . k_j for the rows r of one kv head:
//   stats items    rows on M:  S = Q K^T, (max, sum of exp2) of each row over
//                  a range of keys; a row tile's last item to be closed
//                  combines them to lse[r];
//   column items   keys on M:  S^T = K Q^T, so that a thread holds one key's
//                  logits of all rows: paid[j] = sum_r exp2(z[r][j] - lse[r])
//                  is a sum within the thread, and no weight leaves it.
// Swapping the operands costs nothing: Q and K are both K-major tiles.
//
// What bounds it: the epilogue groups, with many rows.  A 128 x 128 tile is
// 16384 exponentials in each pass and takes a group 1700 cycles, two groups at a
// time, next to 512 cycles of MMA (64 queries of 4 heads on 8 sequences of 6000
// to 16384 keys: 120 us; 128 queries: 216 us).  With few rows (a verify window
// of 40) K's 32 KB a tile from HBM instead, twice: 5 queries of 8 heads on 32 x
// 8192 keys 177 us, 6.1 TB/s.
// One thread that issued both groups' MMAs took 1500 cycles a tile and held
// them up (192 us and, 128 queries, 282 us; with its warp converged, so that
// descriptors and counters are uniform, 267 us).  Not faster: four groups of one
// accumulator each, with that one issuer (128 queries: 390 us); TMEM loads a chunk ahead of
// their use (278 us against 241 then).  A row tile's lse combined by the warp that
// closes it, instead of a head's by one, took 128 queries from 241 to 216 us.
// All stats items come before the column items.  Interleaved, a sequence's
// column items a short way behind its stats items so that they find K in L2,
// the waits for the lse cost more than the reads (verify batch 199 to 280 us
// over distances of one to two items an SM, against 194 us of the time).  The
// column items in reverse order, from the keys read last, wait for the last lse
// (verify batch 200 us against 192, prompt windows 135 against 117).
//
// An item is a range of keys of a head against one row tile (stats) or all row
// tiles that see any of it, one after the other (columns; each thread keeps its
// keys' sums in shared memory between row tiles).  The Q tile is resident, the
// range's K tiles are streamed.
//
// FP8 pools: a K tile's codes come to the slot that the converters make an fp16
// tile of, exactly, which the MMAs read; the resident Q tile becomes fp16 in place.
//
// Roles (448 threads, 704 with the converters; one CTA per SM, persistent):
//   warps 0, 3   producers, one per 64-column half of the tiles (one warp's
//                2 KB boxes go at about 100 cycles each): K by one
//                {64, 1, block_size, 1} box per physical block, Q by one
//                {64, G, 128 / G} box;
//   warps 1, 13  issue the MMAs, one for each epilogue group (warp 1 also
//                allocates TMEM);
//   warp 2       takes items from the queue, looks them up in the plan (in
//                shared memory up to kHeldSeqs sequences), reads the range's
//                block ids and publishes both in a ring (a producer
//                reading the ids of the next tile itself, a tile ahead, was
//                held to their latency: 1.7 us a tile).  A column item is
//                published once its head's lse are complete;
//   warps 4-11   two groups of 128 threads (thread = accumulator lane), which
//                take the item's tiles in turn;
//   warp 12      closes stats items: when both groups have written an item's
//                partials it counts the item, and the row tile's last one makes
//                it combine the rows' lse and announce them; the groups go on
//                without a fence or a wait for the count (all rows of a head,
//                by its last item, were rows * ranges partials for one warp to
//                read while the columns waited);
//   warps 14-21  (FP8) converters: 8 warps took 139 us where 4 took 148 (prompt
//                windows) and 227 us against 237 (verify batch); 130 and 204 us
//                with two issuers.
// Shared memory: 2 resident tiles and two streamed ones for either group (192 KB
// at head_dim 128).  TMEM: four 128-column accumulators.
//
// The wait for a head's lse ends: every stats item it depends on was taken
// from the queue before the column item, by a CTA that works its items off in
// order.  All waits are bounded (2 s, or the launch's limit, then the device
// error word says so and every role leaves); the 128 threads of a group settle failures at barriers
// that OR them, so none is left waiting.
#include <math_constants.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_tc.cuh"
#include "scores.cuh"

namespace pkv {
namespace {

constexpr int kFirstConverter = 14;  // warp
constexpr int kThreadsMma = kFirstConverter * 32, kConverters = 256;
constexpr int kTile = 128;      // rows or keys of a tile
constexpr int kCodeBytes = kTile * 128;  // an FP8 tile
// Each of the two epilogue groups has its own issuing warp, two streamed tiles
// and two accumulators: slots 2 w and 2 w + 1, in turn.  Every barrier's phases
// are so waited for in order.  Slots that both groups share would let a group
// that has few K tiles (row tiles that see one K tile of the range all belong to
// group 0) test a barrier whose previous phase is not complete, and take the
// phase before that one, of the same parity, for its own.
constexpr int kGroupSlots = 2;
constexpr int kSlots = 2 * kGroupSlots;
__device__ __forceinline__ int slot_of(int wg, int k) { return wg * kGroupSlots + k % kGroupSlots; }
__device__ __forceinline__ uint32_t phase_of(int k) { return k / kGroupSlots & 1; }
constexpr int kItems = 2;       // item ring
constexpr int kRangeTiles = kTcRange / kTile;
constexpr int kIds = kTcRange / 8;  // block ids of a range, at most
constexpr int kHeldSeqs = 256;  // sequences whose plan is kept in shared memory
constexpr float kRaise = 8.0f;  // log2 units a row maximum may exceed its reference by

enum { kDone = 0, kStats = 1, kCols = 2 };

struct alignas(16) Item {
  int64_t lse, part;
  int type, s, h, row;
  int L, n, rows, qstart;
  int tile0, tiles;   // row tiles: the first, and how many (stats: one)
  int key0, chunk, chunks, all_tiles;
};

struct Bars {
  uint64_t x_full[2][2], x_empty[2];                // resident tile [buffer][half]
  uint64_t y_full[kSlots][2], y_empty[kSlots];      // streamed tile [slot][half] (FP8: [slot][0], converted)
  uint64_t x_conv[2], c_full[kSlots];               // FP8: resident tile converted; a slot's codes
  uint64_t acc_full[kSlots], acc_empty[kSlots];
  uint64_t item_full[kItems], item_empty[kItems], item_closed[kItems];
};

template <int D, bool F8>
struct Lay {
  static constexpr int kThreads = kThreadsMma + (F8 ? kConverters : 0);
  // fp16 operands: the types' bits 7-12 are zero; N / 8 sits at bit 17
  static constexpr uint32_t kTypes = F8 ? ~0x1F80u : ~0u;
  static constexpr uint32_t kIdesc128 = idesc_bf16(128, 128, false, false) & kTypes;
  static constexpr uint32_t kIdesc16 = idesc_bf16(128, 16, false, false) & kTypes;
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kXOff = 0;
  static constexpr int kYOff = 2 * kTileBytes;
  static constexpr int kItemOff = kYOff + kSlots * kTileBytes;
  static constexpr int kIdOff = kItemOff + kItems * (int)sizeof(Item);
  static constexpr int kLseOff = kIdOff + kItems * kIds * 4;   // [group][2][128] negated lse
  static constexpr int kSumOff = kLseOff + 2 * 2 * kTile * 4;  // [tile of the range][128] column sums
  static constexpr int kBarOff = kSumOff + kRangeTiles * kTile * 4;
  static constexpr int kPlanOff = (kBarOff + (int)sizeof(Bars) + 16 + 15) & ~15;
  static constexpr int kSmem = kPlanOff + kHeldSeqs * (int)sizeof(SeqPlan) + 2 * (kHeldSeqs + 1) * 8 + 1024;
};
static_assert(sizeof(Item) % 16 == 0, "item slot");
static_assert(Lay<128, false>::kSmem <= 232448 && Lay<128, true>::kSmem <= 232448, "shared memory per CTA");

__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, const WaitCtl& w) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, w));
}

// K tiles of the item's range that row tile `tile` sees any key of.
__device__ __forceinline__ int tiles_seen(const ScoreParams& p, const Item& im, int tile) {
  const int last = min(im.n, (tile + 1) * p.tile_tok) - 1;  // the tile's last token
  const int ke = min(p.causal ? im.L - im.n + last + 1 : im.L, min(im.L, im.key0 + kTcRange));
  return ke > im.key0 ? (ke - im.key0 + kTile - 1) / kTile : 0;
}

// Column items: 32 logits of one key against rows' negated lse: the sum of
// their weights (in four running sums); kSome: of the rows in the mask alone,
// the others weigh nothing, whatever their logits and lse (NaN too).
template <bool kSome>
__device__ __forceinline__ void add_weights(const uint32_t (&z)[32], const float* nlse, f32x2 scale2, uint32_t mask,
                                            f32x2 (&sum)[2]) {
  auto weight = [&](float x, int e) {
    const float w = fast_exp2(x);
    return !kSome || (mask >> e & 1) ? w : 0.f;
  };
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    const float4 b = *reinterpret_cast<const float4*>(nlse + i);
    const float2 x0 = up2(fma2(pk2(__uint_as_float(z[i]), __uint_as_float(z[i + 1])), scale2, pk2(b.x, b.y)));
    const float2 x1 = up2(fma2(pk2(__uint_as_float(z[i + 2]), __uint_as_float(z[i + 3])), scale2, pk2(b.z, b.w)));
    sum[0] = add2(sum[0], pk2(weight(x0.x, i), weight(x0.y, i + 1)));
    sum[1] = add2(sum[1], pk2(weight(x1.x, i + 2), weight(x1.y, i + 3)));
  }
}

// kHook: the testing limit and fault are looked at (as arguments of every
// launch they cost the FP8 kernel two spilled registers and 1 % of a verify
// batch over FP8 pools).
template <int D, bool F8, bool kHook>
__global__ void __launch_bounds__(Lay<D, F8>::kThreads, 1) scores_mma_kernel(const ScoreParams p,
                                                                             const __grid_constant__ CUtensorMap qmap,
                                                                             const __grid_constant__ CUtensorMap kmap) {
  using Y = Lay<D, F8>;
  constexpr int kHalves = D / 64;
  constexpr int kYHalves = F8 ? 1 : kHalves;  // barriers that announce a streamed tile
  extern __shared__ __align__(16) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Bars* bars = reinterpret_cast<Bars*>(smem + Y::kBarOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Y::kBarOff + sizeof(Bars));
  Item* items = reinterpret_cast<Item*>(smem + Y::kItemOff);
  int* ids = reinterpret_cast<int*>(smem + Y::kIdOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WaitCtl wc{p.err, kHook ? wait_limit(p.wait_ns) : (uint32_t)kWaitTimeoutNs};

  if (threadIdx.x == 0) {
    for (int b = 0; b < 2; ++b) {
      for (int h = 0; h < 2; ++h) mbar_init(&bars->x_full[b][h], 1);
      mbar_init(&bars->x_empty[b], 2);  // the issuing warps
      mbar_init(&bars->x_conv[b], kConverters);
    }
    for (int i = 0; i < kSlots; ++i) {
      for (int h = 0; h < 2; ++h) mbar_init(&bars->y_full[i][h], F8 ? kConverters : 1);
      mbar_init(&bars->y_empty[i], 1);
      mbar_init(&bars->c_full[i], 1);
      mbar_init(&bars->acc_full[i], 1);
      mbar_init(&bars->acc_empty[i], 4);  // the four warps of the group that read it
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&bars->item_full[i], 1);
      // producers, the issuing warps, the groups' warps, the closer, the converters' warps
      mbar_init(&bars->item_empty[i], kHalves + 2 + 8 + 1 + (F8 ? kConverters / 32 : 0));
      mbar_init(&bars->item_closed[i], 256);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kSlots * 128);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  const uint32_t tmem = *tmem_slot;
  const uint32_t smem_base = smem_u32(smem);

  if (warp == 2) {
    // ================================================================ items
    const int64_t *o_stat = p.off[kTcStat], *o_col = p.off[kTcCol];
    const SeqPlan* plan = p.plan;
    if (p.B <= kHeldSeqs) {
      SeqPlan* plans = reinterpret_cast<SeqPlan*>(smem + Y::kPlanOff);
      int64_t* offs = reinterpret_cast<int64_t*>(plans + kHeldSeqs);
      for (int i = lane; i < p.B * (int)(sizeof(SeqPlan) / 8); i += 32)
        reinterpret_cast<int64_t*>(plans)[i] = reinterpret_cast<const int64_t*>(plan)[i];
      for (int i = lane; i <= p.B; i += 32) {
        offs[i] = o_stat[i];
        offs[kHeldSeqs + 1 + i] = o_col[i];
      }
      __syncwarp();
      plan = plans;
      o_stat = offs;
      o_col = offs + kHeldSeqs + 1;
    }
    const int64_t n_stat = o_stat[p.B], n_all = n_stat + o_col[p.B];
    // Items are taken no earlier than a slot is free: with three slots and one
    // item more in hand the SMs ended unevenly (prompt windows 145 us, 120 then).
    for (int it = 0;; ++it) {
      const int sl = it % kItems;
      if (!wait_all(&bars->item_empty[sl], ((it / kItems) & 1) ^ 1, wc)) break;
      int64_t u = 0;
      if (lane == 0) u = atomicAdd(p.counters, 1);
      u = __shfl_sync(0xffffffffu, u, 0);
      Item item{};
      if (u < n_all) {
        const bool cols = u >= n_stat;
        const int64_t* off = cols ? o_col : o_stat;
        const int64_t v = cols ? u - n_stat : u;
        const int s = find_seq(off, p.B, v, lane);
        const SeqPlan sp = plan[s];
        item.type = cols ? kCols : kStats;
        item.lse = sp.lse;
        item.part = sp.part;
        item.s = s;
        item.row = sp.row;
        item.L = sp.L;
        item.n = sp.n;
        item.rows = sp.rows;
        item.qstart = p.qsl[s];
        item.chunks = sp.chunks;
        item.all_tiles = sp.tiles;
        // row tiles innermost, then heads
        int w = (int)(v - off[s]);
        if (!cols) {
          item.tile0 = w % sp.tiles;
          item.tiles = 1;
          w /= sp.tiles;
        }
        item.chunk = w / p.Hkv;
        item.h = w - item.chunk * p.Hkv;
        item.key0 = item.chunk * kTcRange;
        if (cols) {  // from the first row tile that sees any of the range
          item.tile0 = p.causal ? max(0, item.key0 - (sp.L - sp.n)) / p.tile_tok : 0;
          item.tiles = sp.tiles - item.tile0;
        }
        // the range's blocks (outside the pool: read as zeros)
        const int nblk = (min(sp.L, item.key0 + kTcRange) - item.key0 + p.bs - 1) >> p.bs_log;
        const int32_t* bt = p.tables + (int64_t)s * p.max_blocks + (item.key0 >> p.bs_log);
        int id[kIds / 32];
#pragma unroll
        for (int k = 0; k < kIds / 32; ++k) {
          const int i = k * 32 + lane;
          id[k] = i < nblk ? __ldg(bt + i) : (int)p.num_blocks;
        }
#pragma unroll
        for (int k = 0; k < kIds / 32; ++k) {
          if (id[k] < 0 || id[k] > p.num_blocks || (id[k] == p.num_blocks && k * 32 + lane < nblk)) {
            raise_error(p.err, PKV_DEVERR_BLOCK_OUT_OF_RANGE);
            id[k] = (int)p.num_blocks;
          }
          ids[sl * kIds + k * 32 + lane] = id[k];
        }
        if (cols) {
          bool ok = true;
          if (lane == 0) {
            const uint64_t t0 = globaltimer();
            while (ld_acquire(p.ready + (int64_t)s * p.Hkv + item.h) != sp.tiles) {
              if (globaltimer() - t0 > wc.limit_ns) {
                raise_error(p.err, PKV_DEVERR_TIMEOUT);
                ok = false;
                break;
              }
            }
          }
          if (!__shfl_sync(0xffffffffu, (int)ok, 0)) break;
        }
      }
      __syncwarp();  // the ids are written
      if (lane == 0) {
        items[sl] = item;
        mbar_arrive(&bars->item_full[sl]);
      }
      __syncwarp();
      if (item.type == kDone) break;
    }
  } else if (warp == 0 || warp == 3) {
    // ================================================================ producers
    const int half = warp == 0 ? 0 : 1;
    if (half < kHalves) {
      if (lane == 0) {
        prefetch_tensormap(&qmap);
        prefetch_tensormap(&kmap);
      }
      const int nb_per_tile = kTile / p.bs;
      const int q_bytes = p.tile_tok * p.G * 128;  // one 64-column half of a row tile
      int ny0 = 0, ny1 = 0, nx = 0;  // streamed tiles of either group and resident tiles so far
      bool ok = true;
      // testing only: the first producer of one CTA leaves out its fault_tile-th
      // tile, of the resident tiles and the first streamed one to each, from 1, so
      // that the waits for it run out
      auto left_out = [&](int load) { return kHook && load == p.fault_tile && (half | blockIdx.x) == 0; };
      for (int it = 0; ok; ++it) {
        const int sl = it % kItems;
        if (!wait_all(&bars->item_full[sl], (it / kItems) & 1, wc)) break;
        const Item im = items[sl];
        int id[kRangeTiles];  // this lane's block of each K tile
#pragma unroll
        for (int i = 0; i < kRangeTiles; ++i) id[i] = ids[sl * kIds + min(kIds - 1, i * nb_per_tile + lane)];
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->item_empty[sl]);
        if (im.type == kDone) break;
        for (int tile = im.tile0; tile < im.tile0 + im.tiles && ok; ++tile) {
          const int ny = tiles_seen(p, im, tile);
          if (ny == 0) continue;
          const int xb = nx & 1;
          if (!wait_all(&bars->x_empty[xb], ((nx >> 1) & 1) ^ 1, wc)) {
            ok = false;
            break;
          }
          if (lane == 0 && !left_out(2 * nx + 1)) {
            mbar_arrive_expect_tx(&bars->x_full[xb][half], q_bytes);
            tma_load_3d(smem + Y::kXOff + xb * Y::kTileBytes + half * kHalf, &qmap, &bars->x_full[xb][half], half * 64,
                        im.h * p.G, im.qstart + tile * p.tile_tok);
          }
          ++nx;
#pragma unroll
          for (int i = 0; i < kRangeTiles; ++i) {
            // FP8: the first producer's alone, a key's codes are one 128-byte row
            if (i < ny && ok && (!F8 || half == 0)) {
              int& k = i & 1 ? ny1 : ny0;
              const int st = slot_of(i & 1, k);
              ok = wait_all(&bars->y_empty[st], phase_of(k) ^ 1, wc);
              if (ok) {
                uint64_t* full = F8 ? &bars->c_full[st] : &bars->y_full[st][half];
                const bool out = i == 0 && left_out(2 * nx);
                if (lane == 0 && !out) mbar_arrive_expect_tx(full, kTile * 128);
                __syncwarp();
                if (lane < nb_per_tile && !out)
                  tma_load_4d(smem + Y::kYOff + st * Y::kTileBytes + half * kHalf + lane * p.bs * 128, &kmap, full,
                              half * 64, im.h, 0, id[i]);
                ++k;
              }
            }
          }
        }
      }
      // none of this warp's copies may be in flight when the CTA ends (after
      // an ordinary end the issuing warps have waited for all of them)
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const int n = w ? ny1 : ny0;
        for (int k = max(0, n - kGroupSlots); k < n; ++k)
          wait_all(F8 ? &bars->c_full[slot_of(w, k)] : &bars->y_full[slot_of(w, k)][half], phase_of(k), wc);
      }
      for (int j = max(0, nx - 2); j < nx; ++j) wait_all(&bars->x_full[j & 1][half], (j >> 1) & 1, wc);
    }
  } else if (warp == 1 || warp == 13) {
    // ================================================================ MMA issuer
    // The warp stays together and only the issue itself is one lane's, so that
    // descriptors and counters are warp-uniform.
    const uint64_t dx0 = desc_k(smem_base + Y::kXOff), dy0 = desc_k(smem_base + Y::kYOff);
    const bool issues = lane == 0;
    const int wg = warp == 1 ? 0 : 1;
    int k = 0, nx = 0;  // this group's tiles and resident tiles so far
    bool ok = true;
    for (int it = 0; ok; ++it) {
      const int sl = it % kItems;
      if (!wait_all(&bars->item_full[sl], (it / kItems) & 1, wc)) break;
      const Item im = items[sl];
      __syncwarp();
      if (issues) mbar_arrive(&bars->item_empty[sl]);
      if (im.type == kDone) break;
      const int tile_rows = p.tile_tok * p.G;
      for (int tile = im.tile0; tile < im.tile0 + im.tiles && ok; ++tile) {
        const int ny = tiles_seen(p, im, tile);
        if (ny == 0) continue;
        const int xb = nx & 1;
        if (F8)
          ok = wait_all(&bars->x_conv[xb], (nx >> 1) & 1, wc);
        else
          for (int h = 0; h < kHalves && ok; ++h) ok = wait_all(&bars->x_full[xb][h], (nx >> 1) & 1, wc);
        if (!ok) break;
        ++nx;
        const uint64_t dx = desc_add(dx0, xb * Y::kTileBytes);
        // stats: rows on M; columns: rows on N, a multiple of 16 of them
        const int nr = (min(tile_rows, im.rows - tile * tile_rows) + 15) & ~15;
        const uint32_t idesc = im.type == kStats ? Y::kIdesc128 : Y::kIdesc16 + ((uint32_t)(nr - 16) >> 3 << 17);
        // the tile is waited for also where the group has no K tile of it, so that
        // the arrival counts for its own phase
        if (wg >= ny && issues) mbar_arrive(&bars->x_empty[xb]);
        for (int i = wg; i < ny; i += 2, ++k) {
          const int st = slot_of(wg, k);
          for (int h = 0; h < kYHalves && ok; ++h) ok = wait_all(&bars->y_full[st][h], phase_of(k), wc);
          ok = ok && wait_all(&bars->acc_empty[st], phase_of(k) ^ 1, wc);
          if (!ok) break;
          tc_fence_after();
          const uint64_t dy = desc_add(dy0, st * Y::kTileBytes);
          const uint64_t da = im.type == kStats ? dx : dy, db = im.type == kStats ? dy : dx;
          if (issues) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              umma_bf16(tmem + st * 128, desc_add(da, (kk >> 2) * kHalf + (kk & 3) * 32),
                        desc_add(db, (kk >> 2) * kHalf + (kk & 3) * 32), idesc, kk > 0 ? 1u : 0u);
            umma_commit(&bars->acc_full[st]);
            umma_commit(&bars->y_empty[st]);
            if (i + 2 >= ny) umma_commit(&bars->x_empty[xb]);
          }
          __syncwarp();
        }
      }
    }
    // leaving: the MMAs already issued finish before TMEM is freed
    for (int j = max(0, k - kGroupSlots); j < k; ++j) wait_all(&bars->acc_full[slot_of(wg, j)], phase_of(j), wc);
    __syncwarp();
  } else if (warp == 12) {
    // ================================================================ closer
    for (int it = 0;; ++it) {
      const int sl = it % kItems;
      const uint32_t ph = (it / kItems) & 1;
      if (!wait_all(&bars->item_full[sl], ph, wc)) break;
      const Item im = items[sl];
      if (im.type == kDone) break;
      // the slot is not given back before its closing phase has been seen: the
      // groups cannot be a phase further
      if (!wait_all(&bars->item_closed[sl], ph, wc)) break;
      if (lane == 0) mbar_arrive(&bars->item_empty[sl]);
      if (im.type != kStats) continue;
      // the groups' writes are ordered before this fence by their arrivals
      __threadfence();
      int done = 0;
      if (lane == 0) done = atomicAdd(tile_ticket(p, im.s, im.h, im.qstart, im.all_tiles, im.tile0), 1);
      if (__shfl_sync(0xffffffffu, done, 0) != im.chunks - 1) continue;
      // the row tile's last item: each row's lse from its partials, two a chunk
      __threadfence();
      const int parts = 2 * im.chunks, tile_rows = p.tile_tok * p.G;
      const int end = min(im.rows, (im.tile0 + 1) * tile_rows);
      for (int r = im.tile0 * tile_rows + lane; r < end; r += 32) {
        const float4* part = reinterpret_cast<const float4*>(p.part + im.part + ((int64_t)im.h * im.rows + r) * parts);
        float m = -CUDART_INF_F, l = 0.f;
#pragma unroll 8
        for (int c = 0; c < im.chunks; ++c) {
          const float4 v = __ldcg(part + c);
          const float mn = fmax3(m, v.x, v.z);
          const float mu = max_ref(mn);
          l = l * fast_exp2(m - mu) + (v.y * fast_exp2(v.x - mu) + v.w * fast_exp2(v.z - mu));
          m = mn;
        }
        p.lse[im.lse + (int64_t)im.h * im.rows + r] = m + log2f(l);
      }
      __threadfence();
      __syncwarp();
      if (lane == 0) add_release(p.ready + (int64_t)im.s * p.Hkv + im.h, 1);
    }
  } else if (F8 && warp >= kFirstConverter) {
    // ================================================================ converters
    const int c = threadIdx.x - kFirstConverter * 32;
    int ny0 = 0, ny1 = 0, nx = 0;  // streamed tiles of either group and resident tiles so far
    bool ok = true;
    // A wait that runs out in one warp may end well in another, so none leaves
    // but from a barrier: a K tile's or, at the end and where a wait for an item or
    // a resident tile ran out, one more.  Whichever of them the others are at, they
    // meet there, and leave together if any wait ran out.
    auto leave = [&](bool failed) { barrier_any(3, kConverters, failed); };
    for (int it = 0; ok; ++it) {
      const int sl = it % kItems;
      if (!wait_all(&bars->item_full[sl], (it / kItems) & 1, wc)) {
        leave(true);
        break;
      }
      const Item im = items[sl];
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->item_empty[sl]);
      if (im.type == kDone) {
        leave(false);
        break;
      }
      for (int tile = im.tile0; tile < im.tile0 + im.tiles && ok; ++tile) {
        const int ny = tiles_seen(p, im, tile);
        if (ny == 0) continue;
        // q, in place: whatever place the swizzle gave a value
        const int xb = nx & 1;
        for (int h = 0; h < kHalves && ok; ++h) ok = wait_all(&bars->x_full[xb][h], (nx >> 1) & 1, wc);
        if (!ok) {
          leave(true);
          break;
        }
        uint4* q = reinterpret_cast<uint4*>(smem + Y::kXOff + xb * Y::kTileBytes);
#pragma unroll 4
        for (int i = c; i < Y::kTileBytes / 16; i += kConverters) {
          const uint4 v = q[i];
          q[i] = make_uint4(bf16x2_to_f16x2(v.x), bf16x2_to_f16x2(v.y), bf16x2_to_f16x2(v.z), bf16x2_to_f16x2(v.w));
        }
        fence_proxy_async_smem();
        mbar_arrive(&bars->x_conv[xb]);
        ++nx;
        for (int i = 0; i < ny; ++i) {
          int& k = i & 1 ? ny1 : ny0;
          const int st = slot_of(i & 1, k);
          ok = wait_all(&bars->c_full[st], phase_of(k), wc);
          // 16 codes of a key at a time, all read before any of the fp16 tile, which
          // covers them, is written: to the swizzled halves the MMAs read
          constexpr int kEach = kCodeBytes / 16 / kConverters;
          uint8_t* dst = smem + Y::kYOff + st * Y::kTileBytes;
          const uint4* src = reinterpret_cast<const uint4*>(dst);
          uint4 v[kEach];
          if (ok) {
#pragma unroll
            for (int e = 0; e < kEach; ++e) v[e] = src[e * kConverters + c];
          }
          if (barrier_any(3, kConverters, !ok)) {
            ok = false;
            break;
          }
#pragma unroll
          for (int e = 0; e < kEach; ++e) {
            const int at = e * kConverters + c, key = at >> 3, ch = at & 7;
            const uint32_t in[4] = {v[e].x, v[e].y, v[e].z, v[e].w};
            uint32_t w[8];
#pragma unroll
            for (int o = 0; o < 8; ++o) w[o] = codes_to_f16(in[o >> 1] >> 16 * (o & 1) & 0xffffu);
            uint8_t* row = dst + (ch >> 2) * kHalf + key * 128;
            const int j0 = (ch & 3) * 2;
            *reinterpret_cast<uint4*>(row + ((j0 ^ (key & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4*>(row + (((j0 + 1) ^ (key & 7)) << 4)) = make_uint4(w[4], w[5], w[6], w[7]);
          }
          fence_proxy_async_smem();
          mbar_arrive(&bars->y_full[st][0]);
          ++k;
        }
      }
    }
  } else {
    // ================================================================ epilogue groups
    const int wg = (warp - 4) >> 2;
    const int q4 = warp & 3;
    const int t = q4 * 32 + lane;  // accumulator lane
    const uint32_t lane_base = tmem + ((uint32_t)(q4 * 32) << 16);
    float* nlse = reinterpret_cast<float*>(smem + Y::kLseOff) + wg * 2 * kTile;
    float* sums = reinterpret_cast<float*>(smem + Y::kSumOff) + t;
    const int tile_rows = p.tile_tok * p.G;
    const f32x2 scale2 = pk2(p.scale_log2, p.scale_log2);
    int k = 0, n_nl = 0;  // this group's tiles and lse buffers so far
    bool pending = false;
    for (int it = 0;; ++it) {
      const int sl = it % kItems;
      const bool fail = pending || !wait_all(&bars->item_full[sl], (it / kItems) & 1, wc);
      if (barrier_any(1 + wg, 128, fail)) break;
      const Item im = items[sl];
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->item_empty[sl]);
      if (im.type == kDone) break;
      if (im.type == kStats) {
        // ------------------------------------------------------- stats
        const int ny = tiles_seen(p, im, im.tile0);
        const int row = im.tile0 * tile_rows + t;
        const bool valid = t < tile_rows && row < im.rows;
        const int vis = p.causal ? min(im.L, im.L - im.n + row / p.G + 1) : im.L;
        float m = -CUDART_INF_F, l = 0.f;
        const bool live = __any_sync(0xffffffffu, valid);
        for (int i = wg; i < ny; i += 2) {
          if (pending) break;
          const int acc = slot_of(wg, k);
          pending = !wait_all(&bars->acc_full[acc], phase_of(k), wc);
          if (pending) break;
          ++k;
          tc_fence_after();
          if (live) {
            const int kb = im.key0 + i * kTile;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t z[32];
              tmem_ld32(lane_base + acc * 128 + c * 32, z);
              tmem_wait_ld();
              const int see = vis - (kb + c * 32);  // of these keys, how many the row sees
              if (!__all_sync(0xffffffffu, see >= 32)) {
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (e >= see) z[e] = 0xff800000u;  // -inf
              }
              float a[11];
#pragma unroll
              for (int e = 0; e < 10; ++e)
                a[e] = fmax3(__uint_as_float(z[3 * e]), __uint_as_float(z[3 * e + 1]), __uint_as_float(z[3 * e + 2]));
              a[10] = fmaxf(__uint_as_float(z[30]), __uint_as_float(z[31]));
              const float mx = fmaxf(fmax3(fmax3(a[0], a[1], a[2]), fmax3(a[3], a[4], a[5]), fmax3(a[6], a[7], a[8])),
                                     fmaxf(a[9], a[10])) * p.scale_log2;
              if (mx > m + kRaise) {  // false while both are -inf
                l *= fast_exp2(m - mx);
                m = mx;
              }
              const float neg = m == -CUDART_INF_F ? 0.f : -m;
              const f32x2 neg2 = pk2(neg, neg);
              f32x2 sum[2] = {pk2(0.f, 0.f), pk2(0.f, 0.f)};
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const float2 x0 = up2(fma2(pk2(__uint_as_float(z[e]), __uint_as_float(z[e + 1])), scale2, neg2));
                const float2 x1 = up2(fma2(pk2(__uint_as_float(z[e + 2]), __uint_as_float(z[e + 3])), scale2, neg2));
                sum[0] = add2(sum[0], pk2(fast_exp2(x0.x), fast_exp2(x0.y)));
                sum[1] = add2(sum[1], pk2(fast_exp2(x1.x), fast_exp2(x1.y)));
              }
              const float2 r = up2(add2(sum[0], sum[1]));
              l += r.x + r.y;
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->acc_empty[acc]);
        }
        if (pending) continue;  // leaves at the next agreement; the closer's wait runs out
        if (valid)
          p.part[im.part + ((int64_t)im.h * im.rows + row) * (2 * im.chunks) + im.chunk * 2 + wg] = make_float2(m, l);
        mbar_arrive(&bars->item_closed[sl]);
        continue;
      }
      // --------------------------------------------------------- columns
      const float* lse = p.lse + im.lse + (int64_t)im.h * im.rows;
      const int64_t at0 = ((int64_t)im.row * p.Hkv + im.h) * p.max_len;
      // rows of a row tile as negated lse; rows that are not there weigh nothing
      auto lse_of = [&](int tile) {
        const int row = tile * tile_rows + t;
        return t < tile_rows && row < im.rows ? -__ldcg(lse + row) : -CUDART_INF_F;
      };
      const int end = im.tile0 + im.tiles;  // the last row tile sees every key
      float next = lse_of(im.tile0);
      bool left = false;
      for (int tile = im.tile0; tile < end; ++tile) {
        const int ny = tiles_seen(p, im, tile);
        float* nl = nlse + (n_nl++ & 1) * kTile;
        nl[t] = next;
        // everyone's entry is written; the buffer's last readers passed the row tile before
        if (barrier_any(1 + wg, 128, pending)) {
          left = true;
          break;
        }
        if (tile + 1 < end) next = lse_of(tile + 1);
        const int first = tile * tile_rows, nr = min(tile_rows, im.rows - first);
        for (int i = wg; i < ny; i += 2) {
          if (pending) break;
          const int acc = slot_of(wg, k), j = im.key0 + i * kTile + t;
          const bool keeps = tile + 1 == end && j < im.L;  // this key's sum is complete: store it
          const bool adds = keeps && j < im.L - im.n && p.decay != 0.f;
          const float old = adds ? p.scores[at0 + j] : 0.f;
          pending = !wait_all(&bars->acc_full[acc], phase_of(k), wc);
          if (pending) break;
          ++k;
          tc_fence_after();
          // rows below `from` do not see key j
          const int from = p.causal ? max(0, j - (im.L - im.n)) * p.G - first : 0;
          f32x2 sum[2] = {pk2(0.f, 0.f), pk2(0.f, 0.f)};
#pragma unroll 1
          for (int c = 0; c < nr; c += 32) {
            uint32_t z[32];
            tmem_ld32(lane_base + acc * 128 + c, z);
            tmem_wait_ld();
            if (!__all_sync(0xffffffffu, from <= c) || c + 32 > nr) {
              // rows from .. nr - 1
              const uint32_t below = from - c >= 32 ? ~0u : (1u << max(0, from - c)) - 1u;
              add_weights<true>(z, nl + c, scale2, (nr - c >= 32 ? ~0u : (1u << (nr - c)) - 1u) & ~below, sum);
            } else {
              add_weights<false>(z, nl + c, scale2, ~0u, sum);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->acc_empty[acc]);
          const float2 r = up2(add2(sum[0], sum[1]));
          float paid = r.x + r.y;
          if (tile > im.tile0) paid += sums[i * kTile];  // this thread's own entry
          if (tile + 1 < end)
            sums[i * kTile] = paid;
          else if (keeps)
            p.out[at0 + j] = adds ? fmaf(p.decay, old, paid) : paid;
        }
        // K tiles that this row tile does not see start at the next one that does
        if (tile + 1 < end)
          for (int i = ny; i < kRangeTiles; ++i)
            if ((i & 1) == wg && tile == im.tile0) sums[i * kTile] = 0.f;
      }
      if (left) break;
      if (!pending) mbar_arrive(&bars->item_closed[sl]);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kSlots * 128);
}

template <int D, bool F8, bool kHook>
cudaError_t launch_t(const ScoreParams& p, const CUtensorMap& qmap, const CUtensorMap& kmap, int sms, cudaStream_t s) {
  static unsigned long long done_mask = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!(__atomic_load_n(&done_mask, __ATOMIC_ACQUIRE) & (1ull << dev))) {
    e = cudaFuncSetAttribute(scores_mma_kernel<D, F8, kHook>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<D, F8>::kSmem);
    if (e != cudaSuccess) return e;
    __atomic_fetch_or(&done_mask, 1ull << dev, __ATOMIC_RELEASE);
  }
  return launch_pdl(scores_mma_kernel<D, F8, kHook>, dim3(sms), dim3(Lay<D, F8>::kThreads), Lay<D, F8>::kSmem, s, p, qmap, kmap);
}

template <bool kHook>
cudaError_t launch_hook(const ScoreParams& p, int D, bool f8, const CUtensorMap& qmap, const CUtensorMap& kmap, int sms,
                        cudaStream_t s) {
  if (f8) return launch_t<128, true, kHook>(p, qmap, kmap, sms, s);
  return D == 64 ? launch_t<64, false, kHook>(p, qmap, kmap, sms, s) : launch_t<128, false, kHook>(p, qmap, kmap, sms, s);
}

}  // namespace

cudaError_t launch_scores_mma(const ScoreParams& p, int D, bool f8, const CUtensorMap& qmap, const CUtensorMap& kmap,
                              int sms, cudaStream_t s) {
  if (p.wait_ns || p.fault_tile) return launch_hook<true>(p, D, f8, qmap, kmap, sms, s);  // testing only
  return launch_hook<false>(p, D, f8, qmap, kmap, sms, s);
}

}  // namespace pkv
