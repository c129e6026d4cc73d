// RMS norm of each q and k head, their rotary positions, and the slot-mapping
// scatter of the step's K/V rows, in one pass (paged_kv_write_norm_rope and its
// FP8 form).
//
// For a head x of a token at position p, with weight w (ones where none is
// given) and the angle a = p * inv_freq[i] of its pair i:
//   r = 1 / sqrt(mean(x^2) + eps),   z = r w x,
//   y1 = amp (z1 cos a - z2 sin a),  y2 = amp (z2 cos a + z1 sin a),
// as in rope_write.cu, whose angles these are.  V is not normed.  Squares are
// summed, and all of it computed, in fp32, and rounded once, to the output's
// type.
//
// HBM-bound: rows are read once and written once; the norm, a pass of its own
// over q and k elsewhere, costs no bytes here.  A warp takes a token, or some of
// its heads where tokens are few; a lane owns one place of a head (two 16-byte
// vectors: a pair's two sides), and its weights times cos and sin stay in
// registers while it goes through the heads.  The sum of squares is shuffled
// among the lanes of a head.
#include <math.h>

#include <algorithm>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "rope_rows.cuh"

namespace pkv {
namespace {

struct NormParams {
  const void* q;
  const void* k;
  const void* v;
  const void* qw;  // weights [D], or NULL: ones
  const void* kw;
  const int64_t* positions;
  const double* inv_freq;
  const int64_t* slots;  // NULL: no pools
  void* q_out;
  void* k_out;  // dense rows, or NULL
  void* kc;
  void* vc;
  int64_t T, num_slots, q_stride, k_stride, v_stride;  // strides in elements
  int Hq, Hkv, D, half;
  int interleaved, weights_f32, splits;
  float eps, amp;
  CodeScale k_scale, v_scale;  // of FP8 pools
  int* err;
};

constexpr int kWarps = 4;
constexpr int kBatch = 2;  // heads a lane loads at a time
constexpr int kBulkSmem = 112 * 1024;  // two CTAs an SM at least
// A lane's squares (at most 32 of them) are summed as they are, below 2^125 for |x| <
// 2^60; an eighth of its sum goes to the head's, which 1024 elements would take past
// fp32's range.  (A power of two: the same bits where both fit.)
constexpr float kSumShare = 0.125f;

// U: the rows' element (uint16_t: bf16 bits).  F8: the pools hold E4M3 codes.
// WIDE: a head has more places than a warp has lanes (long heads, or heads
// read by the element), so that its squares are summed in a pass of their own.
template <typename U, int VEC, bool F8, bool INTER, bool WIDE>
__global__ void __launch_bounds__(kWarps * 32) norm_rope_kernel(const NormParams p) {
  pdl_launch_dependents();  // what follows with programmatic launch reads nothing written here before it waits
  extern __shared__ float2 trig_all[];  // [warps][half]
  typedef Vec<U, VEC> V;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t w = (int64_t)blockIdx.x * kWarps + warp;
  const int64_t tok = w / p.splits;
  const int split = (int)(w - tok * p.splits);
  if (tok >= p.T) return;
  float2* trig = trig_all + warp * p.half;
  // this token's rows on their way to L2 while the angles are computed
  if (p.splits == 1) {
    auto fetch = [&](const void* rows, int64_t stride, int heads) {
      const char* at = static_cast<const char*>(rows) + tok * stride * (int64_t)sizeof(U);
      for (int i = lane * 128; i < heads * p.D * (int)sizeof(U); i += 32 * 128)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(at + i));
    };
    fetch(p.q, p.q_stride, p.Hq);
    fetch(p.k, p.k_stride, p.Hkv);
    if (p.slots) fetch(p.v, p.v_stride, p.Hkv);
  }
  const int64_t pos = p.positions[tok];
  int64_t slot = p.slots ? p.slots[tok] : -1;
  if (p.slots && slot >= p.num_slots) {
    if (lane == 0 && split == 0) raise_error(p.err, PKV_DEVERR_SLOT_OUT_OF_RANGE);
    slot = -1;
  }
  for (int j = lane; j < p.half; j += 32) trig[j] = turn_of(angle_of(pos, p.inv_freq[j]), p.amp);
  __syncwarp();

  const int places = (p.D / VEC + 1) / 2;  // of a head; the last may hold one vector
  const int rot_places = p.half / VEC;
  const int side = WIDE ? 1 : 32 / places;  // heads side by side
  const int y = WIDE ? 0 : lane / places;
  const bool idle = !WIDE && y >= side;  // lanes left over
  const float inv_d = 1.f / kSumShare / (float)p.D;

  auto weight = [&](const void* ws, int i) -> float {
    if (!ws) return 1.f;
    return p.weights_f32 ? static_cast<const float*>(ws)[i] : to_f(static_cast<const U*>(ws)[i]);
  };
  // a place's two columns
  auto columns = [&](int x, int& ca, int& cb, bool& rot, bool& two) {
    rot = x < rot_places;
    ca = rot ? (INTER ? 2 * x * VEC : x * VEC) : 2 * p.half + 2 * (x - rot_places) * VEC;
    cb = rot && !INTER ? p.half + x * VEC : ca + VEC;
    two = cb + VEC <= p.D;
  };
  // The factors of a place's values: y1 = r (f[0] x1 - f[1] x2), y2 = r (f[2] x2 + f[3] x1) of each pair.
  struct Factors {
    float f[4][VEC];
  };
  auto factors = [&](const void* ws, int x, Factors& t) {
    int ca, cb;
    bool rot, two;
    columns(x, ca, cb, rot, two);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      // the pair's two elements: (ca + e, cb + e), or, interleaved, (ca + 2e, ca + 2e + 1)
      const bool pairs = rot && INTER;
      const int i1 = pairs ? ca + 2 * e : ca + e, i2 = pairs ? ca + 2 * e + 1 : cb + e;
      const float w1 = weight(ws, i1), w2 = two ? weight(ws, i2) : 0.f;
      const float2 cs = rot ? trig[x * VEC + e] : make_float2(1.f, 0.f);
      t.f[0][e] = cs.x * w1;
      t.f[1][e] = cs.y * w2;
      t.f[2][e] = cs.x * w2;
      t.f[3][e] = cs.y * w1;
    }
  };
  auto turned = [&](const Factors& t, const V& a, const V& b, float r, bool rot, bool two, float (&ya)[VEC],
                    float (&yb)[VEC]) {
    if (!rot) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        ya[e] = t.f[0][e] * to_f(a.e[e]) * r;
        yb[e] = two ? t.f[2][e] * to_f(b.e[e]) * r : 0.f;
      }
    } else if (INTER) {
      float in[2 * VEC], out[2 * VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        in[e] = to_f(a.e[e]);
        in[VEC + e] = to_f(b.e[e]);
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        out[2 * e] = fmaf(in[2 * e], t.f[0][e], -in[2 * e + 1] * t.f[1][e]) * r;
        out[2 * e + 1] = fmaf(in[2 * e + 1], t.f[2][e], in[2 * e] * t.f[3][e]) * r;
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        ya[e] = out[e];
        yb[e] = out[VEC + e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float x1 = to_f(a.e[e]), x2 = to_f(b.e[e]);
        ya[e] = fmaf(x1, t.f[0][e], -x2 * t.f[1][e]) * r;
        yb[e] = fmaf(x2, t.f[2][e], x1 * t.f[3][e]) * r;
      }
    }
  };
  auto squares = [&](const V& a, const V& b, bool two) {
    float s[2] = {};  // the order of norm_rope_bulk_kernel: a row's bits do not depend on the step it comes in
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float x1 = to_f(a.e[e]), x2 = two ? to_f(b.e[e]) : 0.f;
      s[e & 1] = fmaf(x1, x1, s[e & 1]);
      s[e & 1] = fmaf(x2, x2, s[e & 1]);
    }
    return s[0] + s[1];
  };
  // sum over the lanes of a head (all the warp's lanes call it)
  auto head_sum = [&](float s) {
    if (WIDE || (places & (places - 1)) == 0) {
      for (int o = WIDE ? 16 : places >> 1; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      return s;
    }
    float t = 0.f;
    const int first = min(y, side - 1) * places;
    for (int i = 0; i < places; ++i) t += __shfl_sync(0xffffffffu, s, first + i);
    return t;
  };

  // A tensor's heads (src: the token's head 0), normed with ws and turned, or
  // as they are: put(head, column a, column b, both, values)
  auto go = [&](const U* src, int heads, const void* ws, bool norm, auto put) {
    int ca, cb;
    bool rot, two;
    if constexpr (WIDE) {
      for (int h = split; h < heads; h += p.splits) {
        const U* row = src + (int64_t)h * p.D;
        float r = 1.f;
        if (norm) {
          float s = 0.f;
          for (int x = lane; x < places; x += 32) {
            columns(x, ca, cb, rot, two);
            V b{};
            const V a = *reinterpret_cast<const V*>(row + ca);
            if (two) b = *reinterpret_cast<const V*>(row + cb);
            s += squares(a, b, two);
          }
          r = rsqrtf(fmaf(head_sum(s * kSumShare), inv_d, p.eps));
        }
        for (int x = lane; x < places; x += 32) {
          columns(x, ca, cb, rot, two);
          V b{};
          const V a = *reinterpret_cast<const V*>(row + ca);
          if (two) b = *reinterpret_cast<const V*>(row + cb);
          if (norm) {
            Factors t;
            factors(ws, x, t);
            float ya[VEC], yb[VEC];
            turned(t, a, b, r, rot, two, ya, yb);
            put(h, ca, cb, two, ya, yb, a, b);
          } else {
            float ya[VEC], yb[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
              ya[e] = to_f(a.e[e]);
              yb[e] = to_f(b.e[e]);
            }
            put(h, ca, cb, two, ya, yb, a, b);
          }
        }
      }
    } else {
      const int x = idle ? 0 : lane - y * places;
      columns(x, ca, cb, rot, two);
      Factors t;
      if (norm) factors(ws, x, t);
      const int hstep = side * p.splits;
      for (int base = split * side; base < heads; base += kBatch * hstep) {  // the same for every lane
        V a[kBatch], b[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int h = base + y + i * hstep;
          a[i] = b[i] = V{};
          if (!idle && h < heads) {
            a[i] = *reinterpret_cast<const V*>(src + (int64_t)h * p.D + ca);
            if (two) b[i] = *reinterpret_cast<const V*>(src + (int64_t)h * p.D + cb);
          }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int h = base + y + i * hstep;
          float ya[VEC], yb[VEC];
          if (norm) {
            const float r = rsqrtf(fmaf(head_sum(squares(a[i], b[i], two) * kSumShare), inv_d, p.eps));
            turned(t, a[i], b[i], r, rot, two, ya, yb);
          } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
              ya[e] = to_f(a[i].e[e]);
              yb[e] = to_f(b[i].e[e]);
            }
          }
          if (!idle && h < heads) put(h, ca, cb, two, ya, yb, a[i], b[i]);
        }
      }
    }
  };

  U* qo = static_cast<U*>(p.q_out) + tok * p.Hq * (int64_t)p.D;
  go(static_cast<const U*>(p.q) + tok * p.q_stride, p.Hq, p.qw, true,
     [&](int h, int ca, int cb, bool two, const float (&ya)[VEC], const float (&yb)[VEC], const V&, const V&) {
       U* dst = qo + (int64_t)h * p.D;
       store_rows<U, VEC>(dst + ca, ya);
       if (two) store_rows<U, VEC>(dst + cb, yb);
     });
  if (slot < 0 && !p.k_out) return;
  const int64_t at = slot * p.Hkv * (int64_t)p.D;
  U* ko = p.k_out ? static_cast<U*>(p.k_out) + tok * p.Hkv * (int64_t)p.D : nullptr;
  go(static_cast<const U*>(p.k) + tok * p.k_stride, p.Hkv, p.kw, true,
     [&](int h, int ca, int cb, bool two, const float (&ya)[VEC], const float (&yb)[VEC], const V&, const V&) {
       if (ko) {
         U* dst = ko + (int64_t)h * p.D;
         store_rows<U, VEC>(dst + ca, ya);
         if (two) store_rows<U, VEC>(dst + cb, yb);
       }
       if (slot < 0) return;
       const int64_t to = at + (int64_t)h * p.D;
       if constexpr (F8) {
         store_codes<VEC>(static_cast<uint8_t*>(p.kc) + to + ca, ya, p.k_scale);
         if (two) store_codes<VEC>(static_cast<uint8_t*>(p.kc) + to + cb, yb, p.k_scale);
       } else {
         store_rows<U, VEC>(static_cast<U*>(p.kc) + to + ca, ya);
         if (two) store_rows<U, VEC>(static_cast<U*>(p.kc) + to + cb, yb);
       }
     });
  if (slot < 0) return;
  go(static_cast<const U*>(p.v) + tok * p.v_stride, p.Hkv, nullptr, false,
     [&](int h, int ca, int cb, bool two, const float (&ya)[VEC], const float (&yb)[VEC], const V& a, const V& b) {
       const int64_t to = at + (int64_t)h * p.D;
       if constexpr (F8) {
         store_codes<VEC>(static_cast<uint8_t*>(p.vc) + to + ca, ya, p.v_scale);
         if (two) store_codes<VEC>(static_cast<uint8_t*>(p.vc) + to + cb, yb, p.v_scale);
       } else {
         *reinterpret_cast<V*>(static_cast<U*>(p.vc) + to + ca) = a;
         if (two) *reinterpret_cast<V*>(static_cast<U*>(p.vc) + to + cb) = b;
       }
     });
}

// The same for steps of many tokens: a warp goes from token to token, whose rows
// come to shared memory by bulk copies (a token's while the SM's other warps
// compute), so that registers do not hold what is on its way.  Vectors only and
// heads of at most 32 places; weights and angles wait in shared memory too.
// 16384 tokens of 32 and 8 heads of 128 into FP8 pools move 369 MB in 74.3 us,
// 0.73 of a copy's rate.  The instructions (sums across lanes, conversions; 0.58 of
// a scheduler's issue slots) are what it waits for.
template <typename U, bool F8, bool INTER>
__global__ void __launch_bounds__(kWarps * 32) norm_rope_bulk_kernel(const NormParams p, int token_bytes) {
  pdl_launch_dependents();  // what follows with programmatic launch reads nothing written here before it waits
  constexpr int VEC = 16 / sizeof(U);
  typedef Vec<U, VEC> V;
  // [2][D] weights, [warps][half] cos and sin, [warps] rows (128-byte aligned)
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t bars[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* weights = reinterpret_cast<float*>(smem);
  float2* trig = reinterpret_cast<float2*>(weights + 2 * p.D) + warp * p.half;
  uint8_t* rows = smem + ((2 * p.D * 4 + kWarps * p.half * 8 + 127) & ~127) + warp * token_bytes;
  uint64_t* bar = bars + warp;
  if (lane == 0) {
    mbar_init(bar, 1);
    fence_mbar_init();
  }
  for (int i = threadIdx.x; i < 2 * p.D; i += kWarps * 32) {
    const void* ws = i < p.D ? p.qw : p.kw;
    const int d = i < p.D ? i : i - p.D;
    weights[i] = !ws ? 1.f : p.weights_f32 ? static_cast<const float*>(ws)[d] : to_f(static_cast<const U*>(ws)[d]);
  }
  __syncthreads();
  const int q_bytes = p.Hq * p.D * (int)sizeof(U), kv_bytes = p.Hkv * p.D * (int)sizeof(U);
  auto fetch = [&](int64_t tok) {  // by lane 0
    mbar_arrive_expect_tx(bar, token_bytes);
    auto copy = [&](int at, const void* src, int64_t stride, int bytes) {
      asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                       smem_u32(rows + at)),
                   "l"(static_cast<const U*>(src) + tok * stride), "r"(bytes), "r"(smem_u32(bar))
                   : "memory");
    };
    copy(0, p.q, p.q_stride, q_bytes);
    copy(q_bytes, p.k, p.k_stride, kv_bytes);
    if (p.slots) copy(q_bytes + kv_bytes, p.v, p.v_stride, kv_bytes);
  };

  const int places = (p.D / VEC + 1) / 2, rot_places = p.half / VEC, side = 32 / places, y = lane / places;
  const bool idle = y >= side;  // lanes left over
  const int x = idle ? 0 : lane - y * places;
  const bool rot = x < rot_places;
  const int ca = rot ? (INTER ? 2 * x * VEC : x * VEC) : 2 * p.half + 2 * (x - rot_places) * VEC;
  const int cb = rot && !INTER ? p.half + x * VEC : ca + VEC;
  const bool two = cb + VEC <= p.D;
  const float inv_d = 1.f / kSumShare / (float)p.D;
  auto head_sum = [&](float s) {  // over the lanes of a head
    if ((places & (places - 1)) == 0) {
      for (int o = places >> 1; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      return s;
    }
    float t = 0.f;
    const int first = min(y, side - 1) * places;
    for (int i = 0; i < places; ++i) t += __shfl_sync(0xffffffffu, s, first + i);
    return t;
  };

  const int64_t step = (int64_t)gridDim.x * kWarps;
  int64_t tok = (int64_t)blockIdx.x * kWarps + warp;
  if (tok < p.T && lane == 0) fetch(tok);
  int64_t pos = tok < p.T ? p.positions[tok] : 0, slot = tok < p.T && p.slots ? p.slots[tok] : -1;
  for (uint32_t phase = 0; tok < p.T; phase ^= 1) {
    if (p.slots && slot >= p.num_slots) {
      if (lane == 0) raise_error(p.err, PKV_DEVERR_SLOT_OUT_OF_RANGE);
      slot = -1;
    }
    for (int j = lane; j < p.half; j += 32) trig[j] = turn_of(angle_of(pos, p.inv_freq[j]), p.amp);
    const int64_t next = tok + step, at = slot * p.Hkv * (int64_t)p.D;
    if (next < p.T) pos = p.positions[next];
    const int64_t next_slot = next < p.T && p.slots ? p.slots[next] : -1;
    __syncwarp();
    if (!__all_sync(0xffffffffu, mbar_wait(bar, phase, p.err))) {  // (a copy that takes 2 s: reported)
      mbar_wait(bar, phase, p.err);
      break;
    }
    // A tensor's heads (`from` of the token's bytes on): put(head, values of columns ca .., of cb ..)
    auto go = [&](int from, int heads, const float* ws, auto put) {
      const U* src = reinterpret_cast<const U*>(rows + from);
      // y1 = r (f0 x1 - f1 x2), y2 = r (f2 x2 + f3 x1) of each pair, two values an
      // instruction; past the rotary part f1 = f3 = 0.  Interleaved, c holds (f0, f2)
      // and d (-f1, f3) of each pair; else c, d are (f0 f0'), (-f1 -f1') of two
      // pairs and c2, d2 their (f2 f2'), (f3 f3').
      f32x2 c[VEC], d[VEC];  // (c2, d2: the second halves)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        // the pair's two elements: (ca + e, cb + e), or, interleaved, (ca + 2e, ca + 2e + 1)
        const float w1 = INTER ? (two || 2 * e < VEC ? ws[ca + 2 * e] : 0.f) : ws[ca + e];
        const float w2 = INTER ? (two || 2 * e < VEC ? ws[ca + 2 * e + 1] : 0.f) : two ? ws[cb + e] : 0.f;
        const float2 cs = rot ? trig[x * VEC + e] : make_float2(1.f, 0.f);
        if constexpr (INTER) {
          c[e] = pk2(cs.x * w1, cs.x * w2);
          d[e] = pk2(-cs.y * w2, cs.y * w1);
        } else {
          const int k = e >> 1;
          auto set = [&](f32x2& v, float f) {
            const float2 o = up2(v);
            v = e & 1 ? pk2(o.x, f) : pk2(f, 0.f);
          };
          set(c[k], cs.x * w1);
          set(d[k], -cs.y * w2);
          set(c[VEC / 2 + k], cs.x * w2);
          set(d[VEC / 2 + k], cs.y * w1);
        }
      }
      for (int base = 0; base < heads; base += side) {  // the same for every lane
        const int h = base + y;
        const bool live = !idle && h < heads;
        V a{}, b{};
        if (live) {
          a = *reinterpret_cast<const V*>(src + h * p.D + ca);
          if (two) b = *reinterpret_cast<const V*>(src + h * p.D + cb);
        }
        f32x2 xa[VEC / 2], xb[VEC / 2], s2 = pk2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < VEC / 2; ++k) {
          xa[k] = pk2(to_f(a.e[2 * k]), to_f(a.e[2 * k + 1]));
          xb[k] = pk2(to_f(b.e[2 * k]), to_f(b.e[2 * k + 1]));
          s2 = fma2(xa[k], xa[k], s2);
          s2 = fma2(xb[k], xb[k], s2);
        }
        const float2 s = up2(s2);
        const float r = rsqrtf(fmaf(head_sum((s.x + s.y) * kSumShare), inv_d, p.eps));
        const f32x2 r2 = pk2(r, r);
        float ya[VEC], yb[VEC];
#pragma unroll
        for (int k = 0; k < VEC / 2; ++k) {
          f32x2 u, v;
          if constexpr (INTER) {  // pairs are xa's, then xb's
            auto swapped = [](f32x2 z) {
              const float2 o = up2(z);
              return pk2(o.y, o.x);
            };
            u = fma2(xa[k], c[k], mul2(swapped(xa[k]), d[k]));
            v = fma2(xb[k], c[VEC / 2 + k], mul2(swapped(xb[k]), d[VEC / 2 + k]));
          } else {
            u = fma2(xa[k], c[k], mul2(xb[k], d[k]));
            v = fma2(xb[k], c[VEC / 2 + k], mul2(xa[k], d[VEC / 2 + k]));
          }
          const float2 ua = up2(mul2(u, r2)), vb = up2(mul2(v, r2));
          ya[2 * k] = ua.x;
          ya[2 * k + 1] = ua.y;
          yb[2 * k] = vb.x;
          yb[2 * k + 1] = vb.y;
        }
        if (live) put(h, ya, yb);
      }
    };
    U* qo = static_cast<U*>(p.q_out) + tok * p.Hq * (int64_t)p.D;
    go(0, p.Hq, weights, [&](int h, const float (&ya)[VEC], const float (&yb)[VEC]) {
      store_rows<U, VEC>(qo + h * p.D + ca, ya);
      if (two) store_rows<U, VEC>(qo + h * p.D + cb, yb);
    });
    if (slot >= 0 || p.k_out) {
      U* ko = p.k_out ? static_cast<U*>(p.k_out) + tok * p.Hkv * (int64_t)p.D : nullptr;
      go(q_bytes, p.Hkv, weights + p.D, [&](int h, const float (&ya)[VEC], const float (&yb)[VEC]) {
        if (ko) {
          store_rows<U, VEC>(ko + h * p.D + ca, ya);
          if (two) store_rows<U, VEC>(ko + h * p.D + cb, yb);
        }
        if (slot < 0) return;
        const int64_t to = at + h * p.D;
        if constexpr (F8) {
          store_codes<VEC>(static_cast<uint8_t*>(p.kc) + to + ca, ya, p.k_scale);
          if (two) store_codes<VEC>(static_cast<uint8_t*>(p.kc) + to + cb, yb, p.k_scale);
        } else {
          store_rows<U, VEC>(static_cast<U*>(p.kc) + to + ca, ya);
          if (two) store_rows<U, VEC>(static_cast<U*>(p.kc) + to + cb, yb);
        }
      });
    }
    if (slot >= 0) {
      const V* src = reinterpret_cast<const V*>(rows + q_bytes + kv_bytes);
      for (int i = lane; i < p.Hkv * p.D / VEC; i += 32) {
        const V a = src[i];
        if constexpr (F8) {
          float xa[VEC];
#pragma unroll
          for (int e = 0; e < VEC; ++e) xa[e] = to_f(a.e[e]);
          store_codes<VEC>(static_cast<uint8_t*>(p.vc) + at + i * VEC, xa, p.v_scale);
        } else {
          *reinterpret_cast<V*>(static_cast<U*>(p.vc) + at + i * VEC) = a;
        }
      }
    }
    __syncwarp();  // the rows and the angles are read
    tok = next;
    slot = next_slot;
    if (tok < p.T && lane == 0) fetch(tok);
  }
}

pkv_status fail(pkv_status st, const char* msg) {
  set_last_error(msg);
  return st;
}

template <typename U, int VEC, bool F8, bool WIDE>
cudaError_t launch_w(const NormParams& p, dim3 grid, size_t smem, cudaStream_t s) {
  if (p.interleaved)
    norm_rope_kernel<U, VEC, F8, true, WIDE><<<grid, kWarps * 32, smem, s>>>(p);
  else
    norm_rope_kernel<U, VEC, F8, false, WIDE><<<grid, kWarps * 32, smem, s>>>(p);
  return cudaGetLastError();
}

template <typename U, bool F8, bool INTER>
cudaError_t launch_bulk(const NormParams& p, int token_bytes, size_t smem, int sms, cudaStream_t s) {
  static unsigned long long done_mask = 0;
  int dev = 0, ctas = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  auto kernel = norm_rope_bulk_kernel<U, F8, INTER>;
  if (!(__atomic_load_n(&done_mask, __ATOMIC_ACQUIRE) & (1ull << dev))) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBulkSmem);
    if (e != cudaSuccess) return e;
    __atomic_fetch_or(&done_mask, 1ull << dev, __ATOMIC_RELEASE);
  }
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&ctas, kernel, kWarps * 32, smem);
  if (e != cudaSuccess) return e;
  const int64_t most = (p.T + kWarps - 1) / kWarps;
  const int grid = (int)std::min<int64_t>(most, (int64_t)sms * std::max(ctas, 1));
  kernel<<<grid, kWarps * 32, smem, s>>>(p, token_bytes);
  return cudaGetLastError();
}

template <typename U, bool F8>
cudaError_t launch(const NormParams& p0, bool vec, int sms, cudaStream_t s) {
  NormParams p = p0;
  constexpr int kV = 16 / sizeof(U);
  const int places = (p.D / (vec ? kV : 1) + 1) / 2, side = places <= 32 ? 32 / places : 1;
  // few tokens: a token's heads are spread over several warps, down to one
  // load of each lane
  const int most = (std::max(p.Hq, p.Hkv) + side - 1) / side;
  p.splits = 1;
  while (p.T * p.splits < (int64_t)sms * 8 && p.splits < most) p.splits *= 2;
  // tokens enough for every warp to take whole ones: their rows by bulk copies,
  // where four of them fit (32 and 8 heads of 128: 4216 tokens 36.5 us with a token's
  // loads by its lanes, 28.1 so; 16384 tokens into FP8 pools 122 and, with a division
  // to each code as then, 85.6)
  const int64_t token = ((int64_t)p.Hq + (p.slots ? 2 : 1) * p.Hkv) * p.D * (int64_t)sizeof(U);
  const int64_t bulk = (((int64_t)2 * p.D * 4 + kWarps * p.half * 8 + 127) & ~127) + kWarps * token;
  if (p.splits == 1 && vec && places <= 32 && bulk <= kBulkSmem)
    return p.interleaved ? launch_bulk<U, F8, true>(p, (int)token, (size_t)bulk, sms, s)
                         : launch_bulk<U, F8, false>(p, (int)token, (size_t)bulk, sms, s);
  const dim3 grid((unsigned)((p.T * p.splits + kWarps - 1) / kWarps));
  const size_t smem = (size_t)kWarps * p.half * sizeof(float2);
  if (places > 32) return vec ? launch_w<U, kV, F8, true>(p, grid, smem, s) : launch_w<U, 1, F8, true>(p, grid, smem, s);
  return vec ? launch_w<U, kV, F8, false>(p, grid, smem, s) : launch_w<U, 1, F8, false>(p, grid, smem, s);
}

pkv_status norm_rope(NormParams p, int64_t num_blocks, int block_size, int rotary, pkv_dtype dtype,
                     pkv_dtype weight_dtype, bool f8, void* stream) {
  set_last_error("");
  if (dtype != PKV_DTYPE_BF16 && dtype != PKV_DTYPE_F32) return fail(PKV_ERR_UNSUPPORTED, "dtype");
  if (weight_dtype != dtype && weight_dtype != PKV_DTYPE_F32)
    return fail(PKV_ERR_UNSUPPORTED, "weight_dtype must be the rows' or float32");
  const bool pools = p.kc || p.vc;
  if (p.T < 0 || p.Hq <= 0 || p.Hkv <= 0 || p.D <= 0 || num_blocks < 0 || block_size < 0 ||
      ((pools || f8) && (num_blocks == 0 || block_size == 0)))
    return fail(PKV_ERR_INVALID_ARG, "sizes must be positive (num_tokens >= 0)");
  if (rotary <= 0 || rotary % 2 != 0 || rotary > p.D)
    return fail(PKV_ERR_INVALID_ARG, "rotary_dim must be even, positive and at most head_dim");
  if (p.D > 1024) return fail(PKV_ERR_UNSUPPORTED, "head_dim above 1024");
  const int64_t row_q = (int64_t)p.Hq * p.D, row = (int64_t)p.Hkv * p.D;
  if (row > (1 << 24) || row_q > (1 << 24)) return fail(PKV_ERR_UNSUPPORTED, "heads * head_dim too large");
  if (!(p.eps > 0.f) || !isfinite(p.eps)) return fail(PKV_ERR_INVALID_ARG, "eps must be positive and finite");
  if (!(p.amp > 0.f) || !isfinite(p.amp)) return fail(PKV_ERR_INVALID_ARG, "amplitude must be positive and finite");
  if (f8 && (!(p.k_scale.value > 0.f) || !isfinite(p.k_scale.value) || !(p.v_scale.value > 0.f) || !isfinite(p.v_scale.value)))
    return fail(PKV_ERR_INVALID_ARG, "k_scale and v_scale must be positive and finite");
  if (p.q_stride == 0) p.q_stride = row_q;
  if (p.k_stride == 0) p.k_stride = row;
  if (p.v_stride == 0) p.v_stride = row;
  if (p.q_stride < row_q || p.k_stride < row || p.v_stride < row)
    return fail(PKV_ERR_INVALID_ARG, "token stride smaller than heads * head_dim");
  if (p.T > (int64_t)1 << 30) return fail(PKV_ERR_UNSUPPORTED, "num_tokens too large");
  if (p.T == 0) return PKV_OK;
  if (!p.q || !p.k || !p.positions || !p.inv_freq || !p.q_out) return fail(PKV_ERR_INVALID_ARG, "null pointer");
  if (!pools && !p.k_out) return fail(PKV_ERR_INVALID_ARG, "null pointer: neither pools nor k_out");
  if (pools && (!p.kc || !p.vc || !p.v || !p.slots))
    return fail(PKV_ERR_INVALID_ARG, "null pointer: pools want k_cache, v_cache, v and slot_mapping");
  if (!pools) p.slots = nullptr;
  const size_t es = dtype == PKV_DTYPE_BF16 ? 2 : 4, wes = weight_dtype == PKV_DTYPE_BF16 ? 2 : 4;
  auto bits = [](const void* x) { return reinterpret_cast<uintptr_t>(x); };
  if ((bits(p.kc) | bits(p.vc)) & 15u) return fail(PKV_ERR_INVALID_ARG, "caches must be 16-byte aligned");
  if ((bits(p.q) | bits(p.k) | bits(p.v) | bits(p.q_out) | bits(p.k_out)) & (es - 1) ||
      (bits(p.qw) | bits(p.kw)) & (wes - 1) || (bits(p.positions) | bits(p.slots) | bits(p.inv_freq)) & 7u)
    return fail(PKV_ERR_INVALID_ARG, "a tensor is not aligned to its elements");
  int sms = 0;
  pkv_status st = device_state(&sms, &p.err);
  if (st != PKV_OK) return st;
  p.half = rotary / 2;
  p.weights_f32 = weight_dtype == PKV_DTYPE_F32 ? 1 : 0;
  p.num_slots = num_blocks * block_size;
  p.k_scale = code_scale(p.k_scale.value);
  p.v_scale = code_scale(p.v_scale.value);
  // 16-byte vectors where every row, every head and the rotary halves allow them
  const int V = (int)(16 / es);
  const bool vec = p.D % V == 0 && p.half % V == 0 && p.q_stride % V == 0 && p.k_stride % V == 0 &&
                   (!pools || p.v_stride % V == 0) &&
                   ((bits(p.q) | bits(p.k) | bits(p.v) | bits(p.q_out) | bits(p.k_out)) & 15u) == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (es == 2)
    e = f8 ? launch<uint16_t, true>(p, vec, sms, s) : launch<uint16_t, false>(p, vec, sms, s);
  else
    e = f8 ? launch<float, true>(p, vec, sms, s) : launch<float, false>(p, vec, sms, s);
  if (e != cudaSuccess) return cuda_error(e, "paged_kv_write_norm_rope launch");
  return PKV_OK;
}

}  // namespace
}  // namespace pkv

extern "C" {

pkv_status paged_kv_write_norm_rope(const void* q, const void* k, const void* v, const void* q_weight,
                                    const void* k_weight, const int64_t* positions, const double* inv_freq,
                                    const int64_t* slot_mapping, void* q_out, void* k_out, void* k_cache,
                                    void* v_cache, int64_t num_tokens, int64_t num_blocks, int32_t block_size,
                                    int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t rotary_dim,
                                    int32_t interleaved, float eps, float amplitude, int64_t q_token_stride,
                                    int64_t k_token_stride, int64_t v_token_stride, pkv_dtype dtype,
                                    pkv_dtype weight_dtype, void* stream) {
  pkv::NormParams p{q, k, v, q_weight, k_weight, positions, inv_freq, slot_mapping, q_out, k_out, k_cache, v_cache,
                    num_tokens, 0, q_token_stride, k_token_stride, v_token_stride, num_q_heads, num_kv_heads,
                    head_dim, 0, interleaved ? 1 : 0, 0, 0, eps, amplitude, {1.f}, {1.f}, nullptr};
  return pkv::norm_rope(p, num_blocks, block_size, rotary_dim, dtype, weight_dtype, false, stream);
}

pkv_status paged_kv_write_norm_rope_fp8(const void* q, const void* k, const void* v, const void* q_weight,
                                        const void* k_weight, const int64_t* positions, const double* inv_freq,
                                        const int64_t* slot_mapping, void* q_out, void* k_out, void* k_cache,
                                        void* v_cache, int64_t num_tokens, int64_t num_blocks, int32_t block_size,
                                        int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                        int32_t rotary_dim, int32_t interleaved, float eps, float amplitude,
                                        int64_t q_token_stride, int64_t k_token_stride, int64_t v_token_stride,
                                        pkv_dtype dtype, pkv_dtype weight_dtype, float k_scale, float v_scale,
                                        void* stream) {
  pkv::NormParams p{q, k, v, q_weight, k_weight, positions, inv_freq, slot_mapping, q_out, k_out, k_cache, v_cache,
                    num_tokens, 0, q_token_stride, k_token_stride, v_token_stride, num_q_heads, num_kv_heads,
                    head_dim, 0, interleaved ? 1 : 0, 0, 0, eps, amplitude, {k_scale}, {v_scale}, nullptr};
  return pkv::norm_rope(p, num_blocks, block_size, rotary_dim, dtype, weight_dtype, true, stream);
}

}  // extern "C"
