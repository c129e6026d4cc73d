// Attention weight paid to each cached token, for sequences of many rows
// (prefill chunks, observation windows, wide verify steps) in bf16:
// tcgen05.mma with TMEM accumulators.  paged_attention_scores (scores.cu)
// plans the work; this kernel does both passes over the keys.
//
// With z[r][j] = scale * log2(e) * q_r . k_j for the rows r of one kv head:
//   stats items    rows on M:  S = Q K^T, (max, sum of exp2) of each row over
//                  a range of keys; the group that completes a head's last
//                  item combines them to lse[r];
//   column items   keys on M:  S^T = K Q^T, so that a thread holds one key's
//                  logits of all rows: paid[j] = sum_r exp2(z[r][j] - lse[r])
//                  is a sum within the thread, and no weight leaves it.
// Swapping the operands costs nothing: Q and K are both K-major tiles.
//
// What bounds it: the exponentials.  A 128 x 128 tile is 16384 of them, 1024
// cycles of the SM's 16 a cycle, in each pass, next to 512 cycles of MMA; with
// few rows (a verify window of 40) K's 32 KB a tile from HBM instead.  K is
// read from HBM once: a sequence's column items follow its stats items in the
// queue at a distance of two items an SM, so the second pass finds K in L2.
//
// An item pairs one resident tile with a list of streamed ones:
//   stats          Q tile resident, K tiles of the range streamed;
//   columns, one row tile in all:  the same (each K tile's keys are done
//                  after one pair);
//   columns, more row tiles:  a K tile resident, the row tiles that see it
//                  streamed, sums kept in registers.
//
// Roles (384 threads, one CTA per SM, persistent):
//   warps 0, 3   producers, one per 64-column half of the tiles (one warp's
//                2 KB boxes go at about 100 cycles each): K by one
//                {64, 1, block_size, 1} box per physical block, Q by one
//                {64, G, 128 / G} box;
//   warp 1       TMEM allocation, and the thread that issues the MMAs;
//   warp 2       takes items from the queue and publishes them in a ring;
//   warps 4-11   two groups of 128 threads (thread = accumulator lane), which
//                take the item's pairs in turn.
// Shared memory: 2 resident tiles and a 4-stage ring of streamed ones (192 KB
// at head_dim 128).  TMEM: four 128-column accumulators.
//
// A column item waits until its head's lse are complete: every stats item it
// depends on was taken from the queue before it, by a CTA that works its
// items off in order, so the wait ends.  All waits are bounded (2 s, then the
// device error word says so and every role leaves); the 128 threads of a
// group settle failures at barriers that OR them, so none is left waiting.
#include <math_constants.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_tc.cuh"
#include "scores.cuh"

namespace pkv {
namespace {

constexpr int kThreadsMma = 384;
constexpr int kTile = 128;     // rows or keys of a tile
constexpr int kStages = 4;     // streamed tiles
constexpr int kAccs = 4;       // accumulators
constexpr int kItems = 3;      // item ring
constexpr float kRaise = 8.0f;  // log2 units a row maximum may exceed its reference by

constexpr uint32_t kIdesc128 = idesc_bf16(128, 128, false, false);
constexpr uint32_t kIdesc16 = idesc_bf16(128, 16, false, false);  // N = 16; N / 8 sits at bit 17

enum { kDone = 0, kStats = 1, kColsK = 2, kColsQ = 3 };

struct alignas(16) Item {
  int64_t lse, part;
  int type, s, h, row;
  int L, n, rows, qstart;
  int x;       // resident tile: row tile (kStats, kColsK) or first key (kColsQ)
  int y0, ny;  // streamed tiles: first key / first row tile, and how many
  int chunk, chunks, tiles;
};

struct Bars {
  uint64_t x_full[2][2], x_empty[2];             // resident tile [buffer][half]
  uint64_t y_full[kStages][2], y_empty[kStages];  // streamed tile [stage][half]
  uint64_t acc_full[kAccs], acc_empty[kAccs];
  uint64_t item_full[kItems], item_empty[kItems];
  uint64_t xch_full, xch_empty;  // the second group's column sums
};

template <int D>
struct Lay {
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kXOff = 0;
  static constexpr int kYOff = 2 * kTileBytes;
  static constexpr int kItemOff = kYOff + kStages * kTileBytes;
  static constexpr int kLseOff = kItemOff + kItems * (int)sizeof(Item);
  static constexpr int kXchOff = kLseOff + 2 * 2 * kTile * 4;  // [group][2][128] negated lse
  static constexpr int kBarOff = (kXchOff + kTile * 4 + 15) & ~15;
  static constexpr int kSmem = kBarOff + (int)sizeof(Bars) + 32 + 1024;
};
static_assert(sizeof(Item) % 16 == 0, "item slot");
static_assert(Lay<128>::kSmem <= 232448, "shared memory per CTA");

__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, const WaitCtl& w) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, w));
}

// Column items: 32 logits of one key against rows' negated lse: the sum of
// their weights (in four running sums).
__device__ __forceinline__ void add_weights(const uint32_t (&z)[32], const float* nlse, f32x2 scale2, f32x2 (&sum)[2]) {
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    const float4 b = *reinterpret_cast<const float4*>(nlse + i);
    const float2 x0 = up2(fma2(pk2(__uint_as_float(z[i]), __uint_as_float(z[i + 1])), scale2, pk2(b.x, b.y)));
    const float2 x1 = up2(fma2(pk2(__uint_as_float(z[i + 2]), __uint_as_float(z[i + 3])), scale2, pk2(b.z, b.w)));
    sum[0] = add2(sum[0], pk2(fast_exp2(x0.x), fast_exp2(x0.y)));
    sum[1] = add2(sum[1], pk2(fast_exp2(x1.x), fast_exp2(x1.y)));
  }
}

template <int D>
__global__ void __launch_bounds__(kThreadsMma, 1) scores_mma_kernel(const ScoreParams p,
                                                                    const __grid_constant__ CUtensorMap qmap,
                                                                    const __grid_constant__ CUtensorMap kmap) {
  using Y = Lay<D>;
  constexpr int kHalves = D / 64;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Bars* bars = reinterpret_cast<Bars*>(smem + Y::kBarOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Y::kBarOff + sizeof(Bars));
  int* last_flag = reinterpret_cast<int*>(tmem_slot + 1);  // [2]
  Item* items = reinterpret_cast<Item*>(smem + Y::kItemOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WaitCtl wc{p.err, (uint32_t)kWaitTimeoutNs};

  if (threadIdx.x == 0) {
    for (int b = 0; b < 2; ++b) {
      for (int h = 0; h < 2; ++h) mbar_init(&bars->x_full[b][h], 1);
      mbar_init(&bars->x_empty[b], 1);
    }
    for (int i = 0; i < kStages; ++i) {
      for (int h = 0; h < 2; ++h) mbar_init(&bars->y_full[i][h], 1);
      mbar_init(&bars->y_empty[i], 1);
    }
    for (int i = 0; i < kAccs; ++i) {
      mbar_init(&bars->acc_full[i], 1);
      mbar_init(&bars->acc_empty[i], 4);  // the four warps of the group that read it
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&bars->item_full[i], 1);
      mbar_init(&bars->item_empty[i], kHalves + 1 + 8);  // producers, the MMA thread, eight epilogue warps
    }
    mbar_init(&bars->xch_full, 128);
    mbar_init(&bars->xch_empty, 128);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kAccs * 128);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  const uint32_t tmem = *tmem_slot;
  const uint32_t smem_base = smem_u32(smem);
  int* ready = p.tickets + (int64_t)p.B * p.Hkv;

  if (warp == 2) {
    // ================================================================ items
    const int64_t n_stat = __ldg(p.off[kTcStat] + p.B), n_all = n_stat + __ldg(p.off[kTcCol] + p.B);
    int* queue = ready + (int64_t)p.B * p.Hkv;
    for (int it = 0;; ++it) {
      const int sl = it % kItems;
      if (!wait_all(&bars->item_empty[sl], ((it / kItems) & 1) ^ 1, wc)) break;
      int64_t u = 0;
      if (lane == 0) u = atomicAdd(queue, 1);
      u = __shfl_sync(0xffffffffu, u, 0);
      Item item{};
      if (u < n_all) {
        // a place of the queue is a column item of the last sequence whose
        // column items start at or before it, or else a stats item
        int64_t v = u;
        bool cols = false;
        int s = 0;
        if (u >= __ldg(p.off[kTcAt])) {
          s = find_seq(p.off[kTcAt], p.B, u, lane);
          const int64_t at = __ldg(p.off[kTcAt] + s), before = __ldg(p.off[kTcCol] + s),
                        after = __ldg(p.off[kTcCol] + s + 1);
          cols = u < at + (after - before);
          v = cols ? u - at : u - after;
        }
        if (!cols) {
          s = find_seq(p.off[kTcStat], p.B, v, lane);
          v -= __ldg(p.off[kTcStat] + s);
        }
        const SeqPlan sp = p.plan[s];
        item.lse = sp.lse;
        item.part = sp.part;
        item.s = s;
        item.row = sp.row;
        item.L = sp.L;
        item.n = sp.n;
        item.rows = sp.rows;
        item.qstart = p.qsl[s];
        item.chunks = sp.chunks;
        item.tiles = sp.tiles;
        const int w = (int)v;
        if (cols && sp.tiles > 1) {
          // heads innermost; rows that see the tile's first key
          item.type = kColsQ;
          const int kt = w / p.Hkv;
          item.h = w - kt * p.Hkv;
          item.x = kt * kTile;
          item.y0 = p.causal ? max(0, item.x - (sp.L - sp.n)) / p.tile_tok : 0;
          item.ny = sp.tiles - item.y0;
        } else {
          item.type = cols ? kColsK : kStats;
          const int tile = w % sp.tiles, ch = w / sp.tiles;
          item.chunk = ch / p.Hkv;
          item.h = ch - item.chunk * p.Hkv;
          item.x = tile;
          item.y0 = item.chunk * kTcRange;
          // keys its last row sees (columns: all keys, each gets its score)
          const int last = min(sp.n, (tile + 1) * p.tile_tok) - 1;
          const int see = cols || !p.causal ? sp.L : sp.L - sp.n + last + 1;
          const int ke = min(see, min(sp.L, item.y0 + kTcRange));
          item.ny = ke > item.y0 ? (ke - item.y0 + kTile - 1) / kTile : 0;
        }
      }
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
      int g = 0, nx = 0;  // streamed and resident tiles so far
      bool ok = true;
      for (int it = 0; ok; ++it) {
        const int sl = it % kItems;
        if (!wait_all(&bars->item_full[sl], (it / kItems) & 1, wc)) break;
        const Item im = items[sl];
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->item_empty[sl]);
        if (im.type == kDone) break;
        if (im.ny == 0) continue;
        const int32_t* bt = p.tables + (int64_t)im.s * p.max_blocks;
        const int nblk = (im.L + p.bs - 1) / p.bs;
        auto block_of = [&](int key) {  // this lane's physical block of the tile (outside the pool: reads as zeros)
          const int lb = key / p.bs + lane;
          int b = (int)p.num_blocks;
          if (lane < nb_per_tile && lb < nblk) {
            const int x = __ldg(bt + lb);
            if (x >= 0 && x < p.num_blocks)
              b = x;
            else if (half == 0)
              raise_error(p.err, PKV_DEVERR_BLOCK_OUT_OF_RANGE);
          }
          return b;
        };
        auto load_k = [&](uint8_t* dst, uint64_t* bar, int phys) {
          if (lane == 0) mbar_arrive_expect_tx(bar, kTile * 128);
          __syncwarp();
          if (lane < nb_per_tile)
            tma_load_4d(dst + half * kHalf + lane * p.bs * 128, &kmap, bar, half * 64, im.h, 0, phys);
        };
        auto load_q = [&](uint8_t* dst, uint64_t* bar, int tile) {
          if (lane == 0) {
            mbar_arrive_expect_tx(bar, q_bytes);
            tma_load_3d(dst + half * kHalf, &qmap, bar, half * 64, im.h * p.G, im.qstart + tile * p.tile_tok);
          }
        };
        const int xb = nx & 1;
        if (!wait_all(&bars->x_empty[xb], ((nx >> 1) & 1) ^ 1, wc)) break;
        uint8_t* xd = smem + Y::kXOff + xb * Y::kTileBytes;
        if (im.type == kColsQ)
          load_k(xd, &bars->x_full[xb][half], block_of(im.x));
        else
          load_q(xd, &bars->x_full[xb][half], im.x);
        ++nx;
        int phys = im.type == kColsQ ? 0 : block_of(im.y0);
        for (int i = 0; i < im.ny; ++i, ++g) {
          const int st = g % kStages;
          const int next = im.type != kColsQ && i + 1 < im.ny ? block_of(im.y0 + (i + 1) * kTile) : 0;
          if (!wait_all(&bars->y_empty[st], ((g / kStages) & 1) ^ 1, wc)) {
            ok = false;
            break;
          }
          uint8_t* yd = smem + Y::kYOff + st * Y::kTileBytes;
          if (im.type == kColsQ)
            load_q(yd, &bars->y_full[st][half], im.y0 + i);
          else
            load_k(yd, &bars->y_full[st][half], phys);
          phys = next;
        }
      }
      // none of this warp's copies may be in flight when the CTA ends (after
      // an ordinary end the MMA thread has waited for all of them)
      for (int j = max(0, g - kStages); j < g; ++j) wait_all(&bars->y_full[j % kStages][half], (j / kStages) & 1, wc);
      for (int j = max(0, nx - 2); j < nx; ++j) wait_all(&bars->x_full[j & 1][half], (j >> 1) & 1, wc);
    }
  } else if (warp == 1) {
    // ================================================================ MMA issuer
    if (lane == 0) {
      const uint64_t dx0 = desc_k(smem_base + Y::kXOff), dy0 = desc_k(smem_base + Y::kYOff);
      int g = 0, nx = 0;
      bool ok = true;
      for (int it = 0; ok; ++it) {
        const int sl = it % kItems;
        if (!mbar_wait(&bars->item_full[sl], (it / kItems) & 1, wc)) break;
        const int type = items[sl].type, ny = items[sl].ny, rows = items[sl].rows, x = items[sl].x, y0 = items[sl].y0;
        mbar_arrive(&bars->item_empty[sl]);
        if (type == kDone) break;
        if (ny == 0) continue;
        const int xb = nx & 1;
        for (int h = 0; h < kHalves && ok; ++h) ok = mbar_wait(&bars->x_full[xb][h], (nx >> 1) & 1, wc);
        if (!ok) break;
        const int tile_rows = p.tile_tok * p.G;
        const uint64_t dx = desc_add(dx0, xb * Y::kTileBytes);
        for (int i = 0; i < ny; ++i, ++g) {
          const int st = g % kStages, acc = g % kAccs;
          for (int h = 0; h < kHalves && ok; ++h) ok = mbar_wait(&bars->y_full[st][h], (g / kStages) & 1, wc);
          if (!ok || !mbar_wait(&bars->acc_empty[acc], ((g / kAccs) & 1) ^ 1, wc)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t dy = desc_add(dy0, st * Y::kTileBytes);
          // rows on N in a column item: a multiple of 16
          const int tile = type == kColsQ ? y0 + i : x;
          const int nr = (min(tile_rows, rows - tile * tile_rows) + 15) & ~15;
          const uint32_t idesc = type == kStats ? kIdesc128 : kIdesc16 + ((uint32_t)(nr - 16) >> 3 << 17);
          const uint64_t da = type == kColsK ? dy : dx, db = type == kColsK ? dx : dy;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            umma_bf16(tmem + acc * 128, desc_add(da, (kk >> 2) * kHalf + (kk & 3) * 32),
                      desc_add(db, (kk >> 2) * kHalf + (kk & 3) * 32), idesc, kk > 0 ? 1u : 0u);
          umma_commit(&bars->acc_full[acc]);
          umma_commit(&bars->y_empty[st]);
          if (i == ny - 1) umma_commit(&bars->x_empty[xb]);
        }
        ++nx;
      }
      // leaving: the MMAs already issued finish before TMEM is freed
      for (int j = max(0, g - kAccs); j < g; ++j) mbar_wait(&bars->acc_full[j % kAccs], (j / kAccs) & 1, wc);
    }
    __syncwarp();
  } else {
    // ================================================================ epilogue groups
    const int wg = (warp - 4) >> 2;
    const int q4 = warp & 3;
    const int t = q4 * 32 + lane;  // accumulator lane
    const uint32_t lane_base = tmem + ((uint32_t)(q4 * 32) << 16);
    float* nlse = reinterpret_cast<float*>(smem + Y::kLseOff) + wg * 2 * kTile;
    float* xch = reinterpret_cast<float*>(smem + Y::kXchOff);
    const int tile_rows = p.tile_tok * p.G;
    const f32x2 scale2 = pk2(p.scale_log2, p.scale_log2);
    int g = 0, n_xch = 0;
    bool pending = false;
    for (int it = 0;; ++it) {
      const int sl = it % kItems;
      const bool fail = pending || !wait_all(&bars->item_full[sl], (it / kItems) & 1, wc);
      if (barrier_any(1 + wg, 128, fail)) break;
      const Item im = items[sl];
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->item_empty[sl]);
      if (im.type == kDone) break;
      const int64_t sh = (int64_t)im.s * p.Hkv + im.h;
      if (im.type == kStats) {
        // ------------------------------------------------------- stats
        const int row = im.x * tile_rows + t;
        const bool valid = t < tile_rows && row < im.rows;
        const int vis = p.causal ? min(im.L, im.L - im.n + row / p.G + 1) : im.L;
        float m = -CUDART_INF_F, l = 0.f;
        const bool live = __any_sync(0xffffffffu, valid);
        for (int i = 0; i < im.ny; ++i, ++g) {
          if ((i & 1) != wg || pending) continue;
          const int acc = g % kAccs;
          pending = !wait_all(&bars->acc_full[acc], (g / kAccs) & 1, wc);
          if (pending) continue;
          tc_fence_after();
          if (live) {
            const int kb = im.y0 + i * kTile;
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
        const int parts = 2 * im.chunks;
        if (valid && !pending)
          p.part[im.part + ((int64_t)im.h * im.rows + row) * parts + im.chunk * 2 + wg] = make_float2(m, l);
        __threadfence();
        if (barrier_any(1 + wg, 128, pending)) break;
        if (t == 0) last_flag[wg] = atomicAdd(p.tickets + sh, 1);
        named_barrier(1 + wg, 128);
        if (last_flag[wg] == parts * im.tiles - 1) {
          // the head's last item: each row's lse from its partials
          __threadfence();
          for (int r = t; r < im.rows; r += 128) {
            const float2* part = p.part + im.part + ((int64_t)im.h * im.rows + r) * parts;
            float mm = -CUDART_INF_F, ll = 0.f;
            for (int c = 0; c < parts; ++c) mm = fmaxf(mm, __ldcg(part + c).x);
            for (int c = 0; c < parts; ++c) {
              const float2 v = __ldcg(part + c);
              if (v.x != -CUDART_INF_F) ll += v.y * fast_exp2(v.x - mm);
            }
            p.lse[im.lse + (int64_t)im.h * im.rows + r] = mm + log2f(ll);
          }
          __threadfence();
          named_barrier(1 + wg, 128);
          if (t == 0) st_release(ready + sh, 1);
        }
        continue;
      }
      // --------------------------------------------------------- columns
      if (t == 0) {
        const uint64_t t0 = globaltimer();
        while (ld_acquire(ready + sh) == 0) {
          if (globaltimer() - t0 > kWaitTimeoutNs) {
            raise_error(p.err, PKV_DEVERR_TIMEOUT);
            pending = true;
            break;
          }
        }
      }
      if (barrier_any(1 + wg, 128, pending)) break;
      const float* lse = p.lse + im.lse + (int64_t)im.h * im.rows;
      const int64_t at0 = ((int64_t)im.row * p.Hkv + im.h) * p.max_len;
      // rows of a row tile as negated lse; rows that are not there weigh nothing
      auto lse_of = [&](int tile) {
        const int row = tile * tile_rows + t;
        return t < tile_rows && row < im.rows ? -__ldcg(lse + row) : -CUDART_INF_F;
      };
      // the weights of key j's accumulator lane against the rows of `tile`
      auto weigh = [&](int acc, int tile, int j, const float* nl, f32x2 (&sum)[2]) {
        const int first = tile * tile_rows, nr = min(tile_rows, im.rows - first);
        // rows below `from` do not see key j
        const int from = p.causal ? max(0, j - (im.L - im.n)) * p.G - first : 0;
#pragma unroll 1
        for (int c = 0; c < nr; c += 32) {
          uint32_t z[32];
          tmem_ld32(lane_base + acc * 128 + c, z);
          tmem_wait_ld();
          if (!__all_sync(0xffffffffu, from <= c) || c + 32 > nr) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (c + e < from || c + e >= nr) z[e] = 0xff800000u;  // -inf
          }
          add_weights(z, nl + c, scale2, sum);
        }
      };
      auto store = [&](int j, float paid, float old) {
        if (j < im.L) p.out[at0 + j] = j < im.L - im.n && p.decay != 0.f ? fmaf(p.decay, old, paid) : paid;
      };
      auto old_of = [&](int j) { return j < im.L - im.n && p.decay != 0.f ? p.scores[at0 + j] : 0.f; };
      if (im.type == kColsK) {
        nlse[t] = lse_of(im.x);
        if (barrier_any(1 + wg, 128, false)) break;
        for (int i = 0; i < im.ny; ++i, ++g) {
          if ((i & 1) != wg || pending) continue;
          const int acc = g % kAccs, j = im.y0 + i * kTile + t;
          const float old = old_of(j);
          pending = !wait_all(&bars->acc_full[acc], (g / kAccs) & 1, wc);
          if (pending) continue;
          tc_fence_after();
          f32x2 sum[2] = {pk2(0.f, 0.f), pk2(0.f, 0.f)};
          weigh(acc, im.x, j, nlse, sum);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->acc_empty[acc]);
          const float2 r = up2(add2(sum[0], sum[1]));
          store(j, r.x + r.y, old);
        }
        // nlse is rewritten only after the next item's agreement
      } else {
        const int j = im.x + t;
        const float old = wg == 0 ? old_of(j) : 0.f;
        f32x2 sum[2] = {pk2(0.f, 0.f), pk2(0.f, 0.f)};
        float next = wg < im.ny ? lse_of(im.y0 + wg) : 0.f;
        bool left = false;
        for (int i = 0; i < im.ny; ++i, ++g) {
          if ((i & 1) != wg) continue;
          const int acc = g % kAccs;
          float* nl = nlse + ((i >> 1) & 1) * kTile;
          nl[t] = next;
          // everyone's entry is written; the buffer's last readers passed the tile before
          if (barrier_any(1 + wg, 128, pending)) {
            left = true;
            break;
          }
          next = i + 2 < im.ny ? lse_of(im.y0 + i + 2) : 0.f;
          pending = !wait_all(&bars->acc_full[acc], (g / kAccs) & 1, wc);
          if (pending) continue;
          tc_fence_after();
          weigh(acc, im.y0 + i, j, nl, sum);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->acc_empty[acc]);
        }
        if (left) break;
        const float2 r = up2(add2(sum[0], sum[1]));
        // the second group hands its sums to the first
        if (wg == 1) {
          if (!pending) pending = !wait_all(&bars->xch_empty, (n_xch & 1) ^ 1, wc);
          if (!pending) {
            xch[t] = r.x + r.y;
            mbar_arrive(&bars->xch_full);
          }
        } else {
          if (!pending) pending = !wait_all(&bars->xch_full, n_xch & 1, wc);
          if (!pending) {
            const float other = xch[t];
            mbar_arrive(&bars->xch_empty);
            store(j, (r.x + r.y) + other, old);
          }
        }
        ++n_xch;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kAccs * 128);
}

template <int D>
cudaError_t launch_t(const ScoreParams& p, const CUtensorMap& qmap, const CUtensorMap& kmap, int sms, cudaStream_t s) {
  static unsigned long long done_mask = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!(__atomic_load_n(&done_mask, __ATOMIC_ACQUIRE) & (1ull << dev))) {
    e = cudaFuncSetAttribute(scores_mma_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<D>::kSmem);
    if (e != cudaSuccess) return e;
    __atomic_fetch_or(&done_mask, 1ull << dev, __ATOMIC_RELEASE);
  }
  return launch_pdl(scores_mma_kernel<D>, dim3(sms), dim3(kThreadsMma), Lay<D>::kSmem, s, p, qmap, kmap);
}

}  // namespace

cudaError_t launch_scores_mma(const ScoreParams& p, int D, const CUtensorMap& qmap, const CUtensorMap& kmap, int sms,
                              cudaStream_t s) {
  return D == 64 ? launch_t<64>(p, qmap, kmap, sms, s) : launch_t<128>(p, qmap, kmap, sms, s);
}

}  // namespace pkv
