// What the tensor-core kernels of few rows share: a thread holds one key's
// values of all rows; a reduction over a warp's keys; the merge groups.
#pragma once

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_tc.cuh"

namespace pkv {

// A merge group as the planner wrote it, read from L2 (see no_wait).
__device__ __forceinline__ MergeGroup load_group(const MergeGroup* g) {
  static_assert(sizeof(MergeGroup) == 48, "merge group");
  const int4* src = reinterpret_cast<const int4*>(g);
  const int4 a = __ldcg(src), b = __ldcg(src + 1), c = __ldcg(src + 2);
  MergeGroup m;
  m.seq = a.x; m.kvh = a.y; m.row0 = a.z; m.nrows = a.w;
  m.nsplit = b.x; m.part_base = b.y; m.pre_base = b.z; m.pre_n = b.w;
  m.pre_stride = c.x; m.pad0 = c.y; m.pad1 = c.z; m.pad2 = c.w;
  return m;
}

// A warp waits for a phase; true for every lane only if it completed for all.
__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, const WaitCtl& w) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, w));
}

// Reduce NR values per lane over the 32 lanes of a warp with `op`,
// transposing: the result returned by lane l is the reduction of value
// row_of(l) = l >> (5 - log2 NR), so NR values cost NR - 1 + 5 - log2 NR shuffles.
template <int NR, typename Op>
__device__ __forceinline__ float xreduce(float (&a)[NR], int lane, Op op) {
  constexpr int kLog = NR == 1 ? 0 : NR == 2 ? 1 : NR == 4 ? 2 : NR == 8 ? 3 : 4;
#pragma unroll
  for (int lvl = 0; lvl < kLog; ++lvl) {
    const int off = 16 >> lvl;
    const int half = NR >> (lvl + 1);
    const bool up = lane & off;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float send = up ? a[i] : a[i + half];
      const float keep = up ? a[i + half] : a[i];
      a[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, off));
    }
  }
  float x = a[0];
#pragma unroll
  for (int off = 16 >> kLog; off > 0; off >>= 1) x = op(x, __shfl_xor_sync(0xffffffffu, x, off));
  return x;
}

template <int NR>
__device__ __forceinline__ void tmem_ld_rows(uint32_t taddr, uint32_t (&v)[NR]) {
  if constexpr (NR == 4) tmem_ld4(taddr, v);
  else if constexpr (NR == 8) tmem_ld8(taddr, v);
  else tmem_ld16(taddr, v);
}
template <int NR>
__device__ __forceinline__ void tmem_st_rows(uint32_t taddr, const uint32_t (&v)[NR]) {
  if constexpr (NR == 4) tmem_st4(taddr, v);
  else if constexpr (NR == 8) tmem_st8(taddr, v);
  else tmem_st16(taddr, v);
}

struct MaxOp {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct AddOp {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};

}  // namespace pkv
