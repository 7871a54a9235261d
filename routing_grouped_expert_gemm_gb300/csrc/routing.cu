// Routing to experts from given logits, and its gradient (moe_route,
// moe_route_bwd in include/moe.h).
//
// Row t of the logits x gives scores s_e = sigmoid(x_e), or softmax over the
// row; a logit of -inf has score 0 and is never selected.  The selection ranks
// key_e = s_e + b_e (without a bias: x itself, which both score functions
// keep in order), inside the topk_group groups whose sums of the group_top
// largest keys are largest; the weights come from s alone.
//
// The selection is that of fp64 keys (equal ones: the lower id).  Keys are
// computed in fp32 with a known error; where values on both sides of a border
// (of the kept groups, or of the k-th key) lie within that error of it, and are
// not exact ties (the same logit and bias), the warp decides that border again
// in fp64, computing the few keys that lie in the band (for groups those that
// may be among the largest of a group in the band).  With fp32 logits one row of
// some thousands is that close (16384 x 256 in 8 groups: 2 rows at the k-th key,
// 0.7 at the groups' border, which takes the warp 4 us and a call 2 to 3); fp32
// alone would pick another expert in some rows of a large batch.
//
// 16384 x 256 fp32 in 8 groups: 15.6 us, with the sums 19.8 us (17 MB at the
// copy rate would be 2.6 us; DRAM is at 9%, instruction issue at 57%), by softmax
// with the sums 31 us; 32768 x 384 bf16: 25.6 us; one row: 4.0 us a call in a chain.
//
// One warp per row, lane l holding the V consecutive experts l V .. l V + V - 1
// in registers: a row is read once, in 16-byte loads, and nothing but the
// results is written.  Consecutive experts per lane make "lowest id" the same
// as "lowest lane", and a group a set of neighbouring lanes.  The kernel is
// bound by instruction issue, not by memory, so what a row costs is counted in
// instructions (760 a row with groups, bias and sums).  The k-th largest
// of the lanes' maxima (k redux.sync maxima) is a lower bound for the k-th
// key; the keys above it, little more than k, move to one lane each, where a
// row's worth of ranking, ties, checks and weights is a few instructions for
// the whole warp.
#include <cfloat>
#include <cuda_fp16.h>

#include <new>
#include <type_traits>

#include "../../include/moe.h"
#include "common.cuh"

namespace moe {

constexpr int ROUTE_WARPS = 8;          // rows in flight per CTA
constexpr int route_ctas_per_sm(int V) { return V <= 12 ? 3 : 2; }  // what registers allow
constexpr float ROUTE_TINY = 1e-36f;    // keys below this have lost their relative precision (fp32 underflow)
constexpr float ROUTE_REL = 1.0f / 32768;  // relative error of keys, see key_tol
constexpr float ROUTE_U = 1.0f / 8388608;  // 2^-23: fp32's half ulp, two sides of a comparison

struct RouteParams {
  const void* logits;
  int64_t ld, T;  // row stride in elements
  int E, k, dtype, vec;
  const float* bias;
  int n_group, topk_group, group_top, gs, renorm;
  int split;           // route_sums_kernel follows
  int rows, more, ks;  // rows per warp, one more in the first `more` warps; log2 of the lanes of a row's slots (k rounded up)
  float scale;
  int* topk_idx;
  float* topk_w;
  int* counts;      // [E] (one CTA) or per-CTA partials [gridDim.x, E], or NULL
  float* prob_sum;  // the same
};

__device__ __forceinline__ float load_logit(const void* row, int dtype, int e) {
  if (dtype == MOE_DTYPE_FP32) return static_cast<const float*>(row)[e];
  if (dtype == MOE_DTYPE_BF16) return __bfloat162float(static_cast<const bf16*>(row)[e]);
  return __half2float(static_cast<const __half*>(row)[e]);
}

// This lane's V logits of a row (-inf past E).  vec: every row starts on a
// 16-byte boundary, so a lane whose V elements all exist takes them in
// vectors of the largest power of two that divides its bytes.  Not by __ldg: this
// launch may begin while the logits are still being written (launch_early), and
// the read-only path is for what no one writes during a kernel (it took 9.3 us in
// place of 9.7 for the gradient of 16384 x 256; elsewhere the same).
template <int V>
__device__ __forceinline__ void load_row(const void* row, int dtype, int vec, int lane, int E, float (&x)[V]) {
  const int e0 = lane * V;
  if (vec && e0 + V <= E) {
    if (dtype == MOE_DTYPE_FP32) {
      const float* s = static_cast<const float*>(row) + e0;
      if constexpr (V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
          const float4 w = reinterpret_cast<const float4*>(s)[i];
          x[4 * i] = w.x, x[4 * i + 1] = w.y, x[4 * i + 2] = w.z, x[4 * i + 3] = w.w;
        }
      } else if constexpr (V % 2 == 0) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
          const float2 w = reinterpret_cast<const float2*>(s)[i];
          x[2 * i] = w.x, x[2 * i + 1] = w.y;
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = s[i];
      }
      return;
    }
    uint32_t w[(V + 1) / 2];
    const uint16_t* s = static_cast<const uint16_t*>(row) + e0;
    if constexpr (V % 8 == 0) {
#pragma unroll
      for (int i = 0; i < V / 8; ++i) {
        const uint4 q = reinterpret_cast<const uint4*>(s)[i];
        w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
      }
    } else if constexpr (V % 4 == 0) {
#pragma unroll
      for (int i = 0; i < V / 4; ++i) {
        const uint2 q = reinterpret_cast<const uint2*>(s)[i];
        w[2 * i] = q.x, w[2 * i + 1] = q.y;
      }
    } else if constexpr (V % 2 == 0) {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) w[i] = reinterpret_cast<const uint32_t*>(s)[i];
    } else {
      w[0] = *s;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint16_t h = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
      x[i] = dtype == MOE_DTYPE_BF16 ? __uint_as_float((uint32_t)h << 16) : __half2float(__ushort_as_half(h));
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = e0 + i < E ? load_logit(row, dtype, e0 + i) : -INFINITY;
}

// Floats (no NaN) in the order of unsigned integers.
__device__ __forceinline__ uint32_t ord_bits(float f) {
  const uint32_t u = __float_as_uint(f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint32_t ord_of(float f) { return ord_bits(f + 0.0f); }  // -0 equals +0
constexpr uint32_t ORD_NONE = 0x007fffffu;  // -inf: keys up to this are not to be selected
constexpr uint32_t ORD_INF = 0xff800000u;   // +inf (a bias may be): exact, so without an error's band
__device__ __forceinline__ float ord_to(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
}

__device__ __forceinline__ float sum32(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float redux_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float redux_min(float v) {
  float r;
  asm volatile("redux.sync.min.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float max32(float v) { return redux_max(v == v ? v : -INFINITY); }  // NaN operands are passed over
__device__ __forceinline__ int add32(int v) { return __reduce_add_sync(0xffffffffu, v); }
// e^x = 2^(x log2 e): relative error (|x| + 3) 2^-24, flushed to 0 below 2^-126, infinite above 2^128
__device__ __forceinline__ float exp2_fast(float t) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(t));
  return y;
}
constexpr float LOG2E = 1.44269504f;
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 0 at -inf, 1 at +inf
__device__ __forceinline__ float sigmoid_fast(float x) { return rcp_fast(1.0f + exp2_fast(x * -LOG2E)); }
// How far apart two fp32 keys near f have to be for their order to be exact.  In
// units of 2^-24, one side:
// Sigmoid: e^-x is off by 1.22 |x| + 3 relative (the product, log2 e's rounding,
// ex2) and weighs 1 - s; the sum 1, the reciprocal 2: s ((1 - s) (1.22 |x| + 3) +
// 3), so at most 0.82 + 3 s, and relative to s at most 107 above ROUTE_TINY (x >
// -83).  Softmax, d = m - x: e^-d is off by 2.22 d + 3; the row's sum by the
// scores' mean of that (their mean d is at most ln 512) and its roundings, 38; the
// reciprocal 2: s (2.22 d + 43), so at most 0.82 + 43 s, relative at most 228.
// Then the rounding of s + b, |f|.
// Bounds of s: it is at most 1, and at most |f| + |b|.  Of keys up to 2 in size
// (with a neighbour this side of 3) the biases are at most 4: bmax is the largest
// |b| of those only, so that an expert held out or forced by a large bias does
// not make every row's border a close one (16384 x 256 with one expert at -1e4:
// 1.0 to 2.5 ms in place of 14 to 28 us).
constexpr float ROUTE_BIAS = 4.0f;
template <bool kSoft>
__device__ __forceinline__ float key_tol(float f, float bmax) {
  const float a = fminf(fabsf(f), FLT_MAX);  // (an infinite key is exact, and far from every finite one)
  const float s = a > 2.0f ? 1.0f : fminf(a + bmax, 1.0f);
  return fminf(ROUTE_REL * s + ROUTE_TINY, ROUTE_U * (1.0f + (kSoft ? 44.0f : 4.0f) * s)) + 1.25f * ROUTE_U * a;
}
// How far a group's score, the sum of its keys f1 and f2 (0 for none), may be off:
// each key's error as above, and the sum's rounding.
template <bool kSoft>
__device__ __forceinline__ float group_err(float score, float f1, float f2, float bmax) {
  const float a = fabsf(f1) + fabsf(f2), s = a > 2.0f ? 2.0f : fminf(a + 2.0f * bmax, 2.0f);
  const float of_scores = fminf(0.5f * ROUTE_REL * s + ROUTE_TINY, ROUTE_U * (1.0f + (kSoft ? 22.0f : 2.0f) * s));
  return of_scores + 0.625f * ROUTE_U * fminf(a + fabsf(score), FLT_MAX);
}
// e^(x - m), m the row's maximum; an infinite one is its own limit, those logits share the row
__device__ __forceinline__ float soft_score(float x, float m) {
  return m == INFINITY ? (x == m ? 1.0f : x != x ? x : 0.0f) : exp2_fast((x - m) * LOG2E);
}
// x - m where an infinite maximum is its own limit (0), not NaN
__device__ __forceinline__ float below(float x, float m) { return x == m ? 0.0f : x - m; }

// ------------------------------------------------------------------ decisions in fp64
__device__ __forceinline__ unsigned long long ord_of64(double f) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(f + 0.0);
  return u ^ ((unsigned long long)((long long)u >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double ord_to64(unsigned long long u) {
  return __longlong_as_double((long long)(u & 0x8000000000000000ull ? u ^ 0x8000000000000000ull : ~u));
}
__device__ __forceinline__ unsigned long long max32_64(unsigned long long v) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32));
  const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
  return ((unsigned long long)hi << 32) | lo;
}
__device__ __forceinline__ double sum32d(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Softmax's maximum and sum over a row, in fp64.  Whole warp.
template <int V>
__device__ __forceinline__ void softmax_stats64(const RouteParams& p, const void* row, int lane, double* m, double* z) {
  double x[V], lm = -INFINITY, lz = 0.0;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const float f = lane * V + j < p.E ? load_logit(row, p.dtype, lane * V + j) : -INFINITY;
    x[j] = f == f ? (double)f : -INFINITY;
    lm = fmax(lm, x[j]);
  }
  *m = ord_to64(max32_64(ord_of64(lm)));
#pragma unroll
  for (int j = 0; j < V; ++j) lz += x[j] > -INFINITY ? exp(x[j] == *m ? 0.0 : x[j] - *m) : 0.0;
  *z = sum32d(lz);
}
// one expert's key (value, for groups without a bias); -inf if it is not to be selected
template <bool kSoft>
__device__ __forceinline__ double key64(const RouteParams& p, const void* row, int e, double m, double z) {
  const double x = (double)load_logit(row, p.dtype, e);
  if (!(x > -INFINITY)) return -INFINITY;
  double s = kSoft ? exp(x == m ? 0.0 : x - m) / z : 1.0 / (1.0 + exp(-x));
  if (p.bias) s += (double)p.bias[e];
  return s > -INFINITY ? s : -INFINITY;
}

// The kept groups, as bits.  state, for lane g's group: 2 kept, 0 not kept, 1
// to be decided by the candidates' keys (bits of this lane's experts, which
// hold the largest of every such group).  Whole warp.
template <int V, bool kSoft>
__device__ __noinline__ unsigned groups_fp64(const RouteParams& p, const void* row, uint32_t cand, int state, float m32,
                                             int* buf) {
  const int lane = threadIdx.x & 31, e0 = lane * V;
  double m = m32, z = 1.0;
  if (kSoft && p.bias) softmax_stats64<V>(p, row, lane, &m, &z);  // (without a bias the row's sum cancels)
  unsigned long long score = state == 2 ? ~0ull : 0ull, best1 = 0, best2 = 0;  // lane g: of group g so far
  // the candidates, one per lane, 32 at a time
  int before = __popc(cand);
  const int mine = before;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += v;
  }
  const int total = __shfl_sync(0xffffffffu, before, 31);
  before -= mine;
  for (int c0 = 0; c0 < total; c0 += 32) {
    for (uint32_t c = cand, at = (uint32_t)before; c; c &= c - 1, ++at)
      if ((int)at >= c0 && (int)at < c0 + 32) buf[at - c0] = e0 + __ffs(c) - 1;
    __syncwarp();
    const int n = min(32, total - c0);
    unsigned long long key = 0ull;
    int g = -1;
    if (lane < n) {
      const int e = buf[lane];
      const double v = key64<kSoft>(p, row, e, m, z);
      key = v > -INFINITY ? ord_of64(v) : 0ull;
      g = e / p.gs;
    }
    __syncwarp();
    for (int i = 0; i < n; ++i) {
      const unsigned long long v = __shfl_sync(0xffffffffu, key, i);
      const int vg = __shfl_sync(0xffffffffu, g, i);
      if (vg == lane) {
        best2 = max(best2, min(best1, v));
        best1 = max(best1, v);
      }
    }
  }
  if (state == 1) score = p.group_top > 1 && best2 ? ord_of64(ord_to64(best1) + ord_to64(best2)) : best1;
  int rank = 0;
  for (int g = 0; g < p.n_group; ++g) {
    const unsigned long long v = __shfl_sync(0xffffffffu, score, g);
    rank += (v > score || (v == score && g < lane)) ? 1 : 0;
  }
  return __ballot_sync(0xffffffffu, lane < p.n_group && rank < p.topk_group);
}

// Whether this lane's candidate (expert e, -1 for none; ids ascend with the
// lanes) is one of the `need` with the largest keys.  Softmax: z32, the row's
// sum in fp32 (off by less than 2.4e-6), scales all of the candidates' scores
// alike, so it decides unless the border is within that of how far they lie
// apart (and the keys' own roundings); the sum in fp64 costs more than all the
// rest.  Whole warp.
template <int V, bool kSoft>
__device__ __noinline__ bool band_fp64(const RouteParams& p, const void* row, int e, int need, float m32, float z32) {
  const int lane = threadIdx.x & 31;
  double m = m32, z = z32;
  bool in = false;
  for (int pass = 0; pass < (kSoft ? 2 : 1); ++pass) {
    if (pass == 1) softmax_stats64<V>(p, row, lane, &m, &z);
    const double k = e >= 0 ? key64<kSoft>(p, row, e, m, z) : -INFINITY;
    const unsigned long long key = e >= 0 ? ord_of64(k) : 0ull;
    int rank = 0;
    for (unsigned left = __ballot_sync(0xffffffffu, e >= 0); left; left &= left - 1) {
      const int i = __ffs(left) - 1;
      const unsigned long long v = __shfl_sync(0xffffffffu, key, i);
      rank += (v > key || (v == key && i < lane)) ? 1 : 0;
    }
    in = e >= 0 && rank < need;
    if (kSoft && pass == 0) {
      const float s32 = e >= 0 ? (float)(k - (p.bias ? (double)p.bias[e] : 0.0)) : 0.0f;
      const float far = max32(e >= 0 ? s32 : -INFINITY) + max32(e >= 0 ? -s32 : -INFINITY);  // largest less smallest
      const double lo = ord_to64(~max32_64(in ? ~key : 0ull));
      const unsigned long long out = max32_64(e >= 0 && !in ? key : 0ull);
      if (!out || lo - ord_to64(out) > 2.4e-6 * (double)far + 1e-15 + 4.5e-16 * fabs(lo)) break;
    }
  }
  return in;
}
// The same for candidates as bits of each lane's experts.
template <int V, bool kSoft>
__device__ __noinline__ uint32_t wide_band_fp64(const RouteParams& p, const void* row, uint32_t cand, int need) {
  const int lane = threadIdx.x & 31, e0 = lane * V;
  double m = 0.0, z = 1.0;
  if (kSoft) softmax_stats64<V>(p, row, lane, &m, &z);
  uint32_t sel = 0;
  unsigned long long best = 0;
  int bj = 0;
  auto scan = [&]() {
    best = 0;
    for (uint32_t c = cand; c; c &= c - 1) {
      const int j = __ffs(c) - 1;
      const unsigned long long v = ord_of64(key64<kSoft>(p, row, e0 + j, m, z));
      if (v > best) best = v, bj = j;
    }
  };
  scan();
  __syncwarp();
  for (int i = 0; i < need; ++i) {
    const unsigned long long t = max32_64(best);
    if (!t) break;
    if (lane == __ffs(__ballot_sync(0xffffffffu, best == t)) - 1) {
      sel |= 1u << bj;
      cand &= ~(1u << bj);
      scan();
    }
    __syncwarp();
  }
  return sel;
}

// This lane's V keys of a row again, from the same bits as in route_kernel
// (-inf: not to be selected); by_score: the scores in place of x.
template <int V, bool kSoft>
__device__ __forceinline__ void keys_again(const RouteParams& p, const void* row, float m, float inv_z, bool by_score,
                                           uint32_t (&key)[V]) {
  const int e0 = (threadIdx.x & 31) * V;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const float x = e0 + j < p.E ? load_logit(row, p.dtype, e0 + j) : -INFINITY;
    float f = x + 0.0f;
    if (p.bias || by_score) {
      const float b = p.bias && e0 + j < p.E ? p.bias[e0 + j] : 0.0f;
      const float s = kSoft ? soft_score(x, m) : sigmoid_fast(x);
      f = by_score ? s : kSoft ? fmaf(s, inv_z, b) : s + b;
    }
    key[j] = ord_bits(x > -INFINITY && f > -INFINITY ? f : -INFINITY);
  }
}

// Groups whose scores are too close to the border: lane g has group g's smaller
// key that counts, whether it ranks as kept and whether it may lie on either
// side.  The kept groups, as bits.  Whole warp.
template <int V, bool kSoft>
__device__ __noinline__ unsigned decide_groups(const RouteParams& p, const void* row, uint32_t least, bool in, bool band,
                                               float m, float inv_z, float bmax, int* buf) {
  const int lane = threadIdx.x & 31, e0 = lane * V;
  uint32_t key[V], cand = 0;
  keys_again<V, kSoft>(p, row, m, inv_z, !p.bias && p.group_top > 1, key);
  // in those groups, the keys that may be among their largest
  uint32_t from = 0xffffffffu;
  if (band) {
    const float f = ord_to(least);
    from = least < ORD_INF ? ord_of(f - key_tol<kSoft>(f, bmax)) : ORD_INF;
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const uint32_t v = __shfl_sync(0xffffffffu, from, min((e0 + j) / p.gs, 31));
    cand |= key[j] > ORD_NONE && key[j] >= v ? 1u << j : 0u;
  }
  return groups_fp64<V, kSoft>(p, row, cand, band ? 1 : in ? 2 : 0, m, buf);
}

// The k largest of a row with more than 32 candidates -- many equal keys, or
// few lanes that hold many: one maximum after the other.  Whole warp.
template <int V, bool kSoft>
__device__ __noinline__ void select_wide(const RouteParams& p, const void* row, float m, float inv_z, unsigned kept, float bmax,
                                         int* sel_out) {
  const int lane = threadIdx.x & 31, e0 = lane * V;
  const bool with_keys = p.bias != nullptr;
  uint32_t key[V], a1 = 0;
  keys_again<V, kSoft>(p, row, m, inv_z, false, key);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if (key[j] <= ORD_NONE || (p.n_group > 1 && !((kept >> min((e0 + j) / p.gs, 31)) & 1u))) key[j] = 0;
    a1 = max(a1, key[j]);
  }
  uint32_t kth = 0;
  int n = 0, taken = 0;
  for (; n < p.k; ++n) {
    const uint32_t best = __reduce_max_sync(0xffffffffu, a1);
    kth = best;  // (not 0: there are more than 32 candidates)
    if (lane == __ffs(__ballot_sync(0xffffffffu, a1 == best)) - 1) {
      ++taken;
      int ge = 0;  // the next one of this lane, counting equal keys
      a1 = 0;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        ge += key[j] >= best ? 1 : 0;
        a1 = max(a1, key[j] < best ? key[j] : 0u);
      }
      if (ge > taken) a1 = best;
    }
    __syncwarp();
  }
  // the selected: keys above the k-th, and as many equal ones, lowest ids first, as there is room for
  uint32_t gt = 0, eq = 0;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    gt |= key[j] > kth ? 1u << j : 0u;
    eq |= key[j] == kth ? 1u << j : 0u;
  }
  uint32_t band = 0;
  bool decide = false;
  if (with_keys) {
    const float fk = ord_to(kth), tol = key_tol<kSoft>(fk, bmax);
    const uint32_t lo = ord_of(fk - tol), hi = ord_of(fk + tol);
    uint32_t over = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      over |= key[j] > hi ? 1u << j : 0u;
      band |= key[j] >= lo && key[j] <= hi ? 1u << j : 0u;
    }
    float lx = 0.0f, lb = 0.0f;
    bool some = false, mixed = false;
    for (uint32_t c = band; c; c &= c - 1) {
      const int ee = e0 + __ffs(c) - 1;
      const float xe = load_logit(row, p.dtype, ee), be = p.bias[ee];
      mixed |= some && (xe != lx || be != lb);
      lx = xe, lb = be, some = true;
    }
    __syncwarp();
    const int first = __ffs(__ballot_sync(0xffffffffu, some)) - 1;
    const float rx = __shfl_sync(0xffffffffu, lx, first), rb = __shfl_sync(0xffffffffu, lb, first);
    decide = __any_sync(0xffffffffu, mixed || (some && (lx != rx || lb != rb)));
    if (decide) gt = over, eq = band;
  }
  const int room = p.k - add32(__popc(gt));
  uint32_t sel = gt;
  if (decide) {
    sel |= wide_band_fp64<V, kSoft>(p, row, eq, room);
  } else {
    int b4 = __popc(eq);
    const int own = b4;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, b4, o);
      if (lane >= o) b4 += v;
    }
    for (int left = room - (b4 - own); eq && left > 0; eq &= eq - 1, --left) sel |= eq & -eq;
  }
  __syncwarp();
  int at = __popc(sel);
  const int own = at;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, at, o);
    if (lane >= o) at += v;
  }
  at -= own;
  for (; sel; sel &= sel - 1) sel_out[at++] = e0 + __ffs(sel) - 1;
}

// ------------------------------------------------------------------ forward
template <int V, bool kSoft>
__global__ void __launch_bounds__(ROUTE_WARPS * 32, route_ctas_per_sm(V)) route_kernel(const __grid_constant__ RouteParams p) {
  __shared__ int s_hist[E_MAX];
  __shared__ __align__(16) float s_key[ROUTE_WARPS][32];  // candidates: key and expert
  __shared__ int s_id[ROUTE_WARPS][32];
  __shared__ int s_sel[ROUTE_WARPS][32];        // selected experts of up to 32 >> ks rows
  __shared__ float s_row[ROUTE_WARPS][32][2];   // softmax: the row's maximum and 1 / sum (NaN: the row has one)
  __shared__ float s_p[ROUTE_WARPS][32 * V];
  __shared__ __align__(16) float s_bias[32 * V];                   // NaN as -inf: never selected
  __shared__ __align__(16) float s_keys[ROUTE_WARPS][32 * V];  // the row's keys
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e0 = lane * V;
  const bool sums = p.prob_sum != nullptr, grouped = p.n_group > 1;
  const bool with_keys = p.bias != nullptr;                             // the order is s + b's, not x's
  const bool group_scores = grouped && (with_keys || p.group_top > 1);  // groups are ranked by computed values
  const bool scored = with_keys || sums || group_scores || (kSoft && !p.renorm);
  // groups made of whole, aligned sets of lanes are ranked by butterflies
  const int glanes = p.gs / V;
  const bool aligned_groups = grouped && p.gs % V == 0 && (glanes & (glanes - 1)) == 0 && glanes <= 32;
  // The sums' kernel may take its place and wait.  (Not whatever else follows on the stream: its CTAs would sit where
  // this launch's run, 17.0 against 18.5 us.)
  if (p.split) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");  // for what is before this launch, see launch_early
  if (p.counts) {
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) s_hist[e] = 0;
    __syncthreads();
  }
  float bmax = 0.0f, acc[V];
  uint32_t gid[(V + 3) / 4];  // the experts' groups, a byte each (aligned groups: the lane's, once)
#pragma unroll
  for (int j = 0; j < V; ++j) acc[j] = 0.0f;
#pragma unroll
  for (int j = 0; j < (V + 3) / 4; ++j) gid[j] = 0;
  if (aligned_groups) {
    gid[0] = (uint32_t)min(lane / glanes, 31);
  } else if (grouped) {
#pragma unroll
    for (int j = 0; j < V; ++j) gid[j / 4] |= (uint32_t)min((e0 + j) / p.gs, 31) << (8 * (j % 4));
  }
  float* bias = s_bias + e0;
  if (with_keys) {  // every warp writes the same
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float v = e0 + j < p.E ? p.bias[e0 + j] : 0.0f;
      bmax = fmaxf(bmax, fabsf(v) <= ROUTE_BIAS ? fabsf(v) : 0.0f);
      bias[j] = v == v ? v : -INFINITY;
    }
    __syncwarp();
  }
  bmax = max32(bmax);
  const size_t row_bytes = (size_t)p.ld * (p.dtype == MOE_DTYPE_FP32 ? 4 : 2);

  const uint32_t lt = (1u << lane) - 1u;
  const int wid = blockIdx.x * ROUTE_WARPS + warp;
  const int64_t t_from = (int64_t)wid * p.rows + min(wid, p.more), t_to = t_from + p.rows + (wid < p.more ? 1 : 0);
  for (int64_t tb = t_from; tb < t_to; tb += 32 >> p.ks) {
  // select for as many rows as have their slots in one warp, then weigh them together
  const int n_rows = (int)min((int64_t)(32 >> p.ks), t_to - tb);
  s_sel[warp][lane] = -1;
  __syncwarp();
  for (int r = 0; r < n_rows; ++r) {
    const void* row = static_cast<const uint8_t*>(p.logits) + (size_t)(tb + r) * row_bytes;
    float x[V];
    load_row<V>(row, p.dtype, p.vec, lane, p.E, x);

    // scores, where anything needs them: s (sigmoid) or e^(x - m) (softmax), z the row's sum
    float s[V];
    float m = 0.0f, z = 1.0f;
    bool nan_row = false;
    auto row_max = [&]() {
      float lm = -INFINITY;
#pragma unroll
      for (int j = 0; j < V; ++j) lm = fmaxf(lm, x[j]);
      return max32(lm);
    };
    if (kSoft && (scored || !p.renorm)) m = row_max();
    if (scored) {
      if (kSoft) {
#pragma unroll
        for (int j = 0; j < V; ++j) s[j] = soft_score(x[j], m);
        if (m == -INFINITY) {
#pragma unroll
          for (int j = 0; j < V; ++j) s[j] = x[j] != x[j] ? x[j] : 0.0f;
        }
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) s[j] = sigmoid_fast(x[j]);
      }
      if (kSoft || sums) {
        float lz = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) lz += s[j];
        z = sum32(lz);
        nan_row = z != z;
        if (kSoft && nan_row) {  // the NaNs are not selected; the others keep their order
          lz = 0.0f;
#pragma unroll
          for (int j = 0; j < V; ++j) lz += x[j] > -INFINITY ? s[j] : 0.0f;
          z = sum32(lz);
        }
      }
    }
    if (kSoft && !scored) {
      bool nan = false;
#pragma unroll
      for (int j = 0; j < V; ++j) nan |= x[j] != x[j];
      nan_row = __any_sync(0xffffffffu, nan);
    }
    const float inv_z = z > 0.0f ? rcp_fast(z) : 0.0f;
    if (sums) {  // normalised scores, s over the row's sum
      if (!kSoft && z < 1e-6f) m = row_max();  // (larger sums have no score that underflows and counts)
      if (!kSoft && z < 1e-6f && m < -20.0f && m > -INFINITY) {  // e^x to fp32 precision: shifted against underflow
        float u[V], lz = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          u[j] = exp2_fast((x[j] - m) * LOG2E);
          lz += u[j];
        }
        const float inv = rcp_fast(sum32(lz));
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] += u[j] * inv;
      } else {
        const float inv = nan_row ? NAN : inv_z;
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] += s[j] * inv;
      }
    }

    // the order of the experts: -inf is not to be selected
    float key[V];
    if (with_keys) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float f = kSoft ? fmaf(s[j], inv_z, bias[j]) : s[j] + bias[j];
        key[j] = x[j] > -INFINITY ? f : -INFINITY;
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) key[j] = fmaxf(x[j], -INFINITY);  // (NaN too)
    }

    unsigned kept_groups = ~0u;
    if (grouped) {
      // each group's two largest; without a bias of the (order-keeping) scores, or, for the maximum alone, of x
      const bool by_score = group_scores && !with_keys;
      float g1 = -INFINITY, g2 = -INFINITY;  // lane g: those of group g
      if (aligned_groups) {
        float t1 = -INFINITY, t2 = -INFINITY;
        auto take = [&](float v) {
          t2 = fmaxf(t2, fminf(t1, v));
          t1 = fmaxf(t1, v);
        };
        if (by_score) {
#pragma unroll
          for (int j = 0; j < V; ++j) take(key[j] > -INFINITY ? s[j] : -INFINITY);
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j) take(key[j]);
        }
#pragma unroll 2
        for (int o = 1; o < glanes; o <<= 1) {
          const float u1 = __shfl_xor_sync(0xffffffffu, t1, o), u2 = __shfl_xor_sync(0xffffffffu, t2, o);
          t2 = fmaxf(fmaxf(t2, u2), fminf(t1, u1));
          t1 = fmaxf(t1, u1);
        }
        const int from = (lane * glanes) & 31;
        g1 = __shfl_sync(0xffffffffu, t1, from);
        g2 = __shfl_sync(0xffffffffu, t2, from);
        if (lane >= p.n_group) g1 = g2 = -INFINITY;
      } else {
        for (int g = 0; g < p.n_group; ++g) {
          const int lo = g * p.gs - e0, hi = lo + p.gs;
          float t1 = -INFINITY, t2 = -INFINITY;
#pragma unroll
          for (int j = 0; j < V; ++j) {
            float v = by_score ? (key[j] > -INFINITY ? s[j] : -INFINITY) : key[j];
            v = j >= lo && j < hi ? v : -INFINITY;
            t2 = fmaxf(t2, fminf(t1, v));
            t1 = fmaxf(t1, v);
          }
          const float w1 = redux_max(t1);
          const unsigned own = __ballot_sync(0xffffffffu, t1 == w1);
          const float w2 = redux_max(lane == __ffs(own) - 1 ? t2 : t1);
          if (lane == g) g1 = w1, g2 = w2;
        }
      }
      // the topk_group largest scores, the lowest group first among equals; a group without an expert has -inf
      float score = g1;
      if (group_scores && p.group_top > 1 && g2 > -INFINITY) score = fmaxf(g1 + g2, -FLT_MAX);
      float thr = -INFINITY;
      {
        float a = score;
#pragma unroll 4
        for (int i = 0; i < p.topk_group; ++i) {
          thr = redux_max(a);
          a = a == thr ? -INFINITY : a;
        }
      }
      bool in = score > -INFINITY && score >= thr;
      unsigned kept = __ballot_sync(0xffffffffu, in);
      if (__popc(kept) > p.topk_group) {  // (equal scores count once above)
        s_key[warp][lane] = score;
        __syncwarp();
        int rank = 0;  // the number of larger scores
        for (int g = 0; g < p.n_group; ++g) rank += s_key[warp][g] > score ? 1 : 0;
        __syncwarp();
        in = in && rank < p.topk_group;
        kept = __ballot_sync(0xffffffffu, in);
        thr = redux_min(in ? score : INFINITY);
        if (__popc(kept) > p.topk_group) {  // equal scores across the border: the lowest groups
          const unsigned over = __ballot_sync(0xffffffffu, in && score > thr), same = kept & ~over;
          in = in && (score > thr || __popc(same & lt) < p.topk_group - __popc(over));
          kept = __ballot_sync(0xffffffffu, in);
        }
      }
      if (group_scores) {
        // each group's own error: one of large biases may be far off without its being near the border
        const bool two = p.group_top > 1 && g2 > -INFINITY;
        const float err = group_err<kSoft>(score, g1, two ? g2 : 0.0f, bmax);
        const float hi = redux_max(in ? -INFINITY : score + err), lo = redux_min(in ? score - err : INFINITY);
        if (hi > -INFINITY && !(lo > hi)) {
          const bool band = score > -INFINITY && (in ? score - err <= hi : score + err >= lo);
          kept = decide_groups<V, kSoft>(p, row, ord_of(two ? g2 : g1), in, band, m, inv_z, bmax, s_id[warp]);
        }
      }
      kept_groups = kept;
      if (aligned_groups) {
        const bool keep = (kept >> gid[0]) & 1u;  // all of a lane's experts are in one group
#pragma unroll
        for (int j = 0; j < V; ++j) key[j] = keep ? key[j] : -INFINITY;
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (!((kept >> ((gid[j / 4] >> (8 * (j % 4))) & 31u)) & 1u)) key[j] = -INFINITY;
      }
    }
    float a1 = -INFINITY;  // this lane's largest key
#pragma unroll
    for (int j = 0; j < V; ++j) a1 = fmaxf(a1, key[j]);

    // k lanes' maxima at least reach `floor`, so the k-th key does too (-inf: fewer lanes have keys)
    float floor = -INFINITY;
    {
      float a = a1;
#pragma unroll 4
      for (int i = 0; i < p.k; ++i) {
        floor = redux_max(a);
        a = a == floor ? -INFINITY : a;
      }
    }
    // candidates: the keys from there up, and those that their error might lift there (an infinite bias is exact)
    if (with_keys && fabsf(floor) < INFINITY) floor -= key_tol<kSoft>(floor, bmax);
    floor = fmaxf(floor, -FLT_MAX);
    uint32_t cand = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) cand |= key[j] >= floor ? 1u << j : 0u;
    int before = __popc(cand);
    const int mine = before;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += v;
    }
    const int n_cand = __shfl_sync(0xffffffffu, before, 31);
    before -= mine;
    if (n_cand <= 32) {  // one lane each, ids ascending with the lanes
      float* keys = s_keys[warp] + e0;
#pragma unroll
      for (int j = 0; j < V; ++j) keys[j] = key[j];
      for (uint32_t c = cand; c; c &= c - 1) s_id[warp][before++] = e0 + __ffs(c) - 1;
      __syncwarp();
      const int e = s_id[warp][lane];
      const float c = lane < n_cand ? s_keys[warp][e] : -INFINITY;
      s_key[warp][lane] = c;
      __syncwarp();
      int rank = 0;  // of a key, the number of larger ones
      for (int i = 0; i < n_cand; i += 4) {
        const float4 v = *reinterpret_cast<const float4*>(&s_key[warp][i]);
        rank += v.x > c ? 1 : 0;
        rank += v.y > c ? 1 : 0;
        rank += v.z > c ? 1 : 0;
        rank += v.w > c ? 1 : 0;
      }
      bool in = c > -INFINITY && rank < p.k;
      unsigned who = __ballot_sync(0xffffffffu, in);
      const float kth = redux_min(in ? c : INFINITY);
      if (__popc(who) > p.k) {  // equal keys across the border: the lowest ids
        const unsigned over = __ballot_sync(0xffffffffu, in && c > kth), same = who & ~over;
        in = in && (c > kth || __popc(same & lt) < p.k - __popc(over));
        who = __ballot_sync(0xffffffffu, in);
      }
      if (with_keys && n_cand > p.k) {
        // candidates within the error of the k-th: unless all of them are one logit with one bias, fp64 decides
        const float tol = key_tol<kSoft>(kth, bmax);
        const bool close = c > -INFINITY && !(fabsf(c - kth) > tol);
        const unsigned band = __ballot_sync(0xffffffffu, close);
        if (band & ~who) {
          const float xe = close ? load_logit(row, p.dtype, e) : 0.0f, be = close ? p.bias[e] : 0.0f;
          const int first = __ffs(band) - 1;
          const float rx = __shfl_sync(0xffffffffu, xe, first), rb = __shfl_sync(0xffffffffu, be, first);
          if (__any_sync(0xffffffffu, close && (xe != rx || be != rb))) {
            in = in && !close;
            in |= band_fp64<V, kSoft>(p, row, close ? e : -1, p.k - __popc(__ballot_sync(0xffffffffu, in)), m, z);
            who = __ballot_sync(0xffffffffu, in);
          }
        }
      }
      if (in) s_sel[warp][(r << p.ks) + __popc(who & lt)] = e;
    } else {
      select_wide<V, kSoft>(p, row, m, inv_z, kept_groups, bmax, &s_sel[warp][r << p.ks]);
    }
    if (kSoft && lane == 0) {
      s_row[warp][r][0] = m;
      s_row[warp][r][1] = nan_row ? NAN : inv_z;
    }
    __syncwarp();
  }

  // weights, one lane per slot of the rows
  const int r = lane >> p.ks, slot = lane & ((1 << p.ks) - 1);
  const int64_t t = tb + r;
  const int e = r < n_rows ? s_sel[warp][lane] : -1;
  const bool on = e >= 0;
  const float xs = on ? load_logit(static_cast<const uint8_t*>(p.logits) + (size_t)t * row_bytes, p.dtype, e) : -INFINITY;
  const float nan = kSoft && on ? s_row[warp][r][1] : 0.0f;
  float w = 0.0f;
  if (p.renorm) {  // over the selected: a common factor cancels, so scores that underflow are shifted
    float ms = xs;
    for (int o = 1 << p.ks >> 1; o > 0; o >>= 1) ms = fmaxf(ms, __shfl_xor_sync(0xffffffffu, ms, o));
    if (on) w = kSoft || ms < -20.0f ? expf(below(xs, ms)) : 1.0f / (1.0f + expf(-xs));
    float tot = w;
    for (int o = 1 << p.ks >> 1; o > 0; o >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, o);
    if (on) w = w / tot * p.scale;  // (one expert: exactly scale)
  } else if (on) {
    w = (kSoft ? expf(below(xs, s_row[warp][r][0])) * nan : 1.0f / (1.0f + expf(-xs))) * p.scale;
  }
  if (nan != nan) w = nan;
  if (r < n_rows && slot < p.k) {
    p.topk_idx[t * p.k + slot] = e;
    p.topk_w[t * p.k + slot] = w;
    if (p.counts && on) atomicAdd(&s_hist[e], 1);  // (integers: any order gives the same)
  }
  __syncwarp();
  }

  if (p.counts || sums) {
    if (sums) {
#pragma unroll
      for (int j = 0; j < V; ++j) s_p[warp][e0 + j] = acc[j];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
      const size_t o = (size_t)blockIdx.x * p.E + e;
      if (p.counts) p.counts[o] = s_hist[e];
      if (sums) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < ROUTE_WARPS; ++w) v += s_p[w][e];
        p.prob_sum[o] = v;
      }
    }
  }
}

// Sums over the CTAs' partials in a fixed order: a CTA per 32 experts, its 32
// warps taking every 32nd partial, then the warps in turn.  Launched while
// route_kernel still runs (programmatic dependency), it waits for it here.
__global__ void __launch_bounds__(1024) route_sums_kernel(const int* pc, const float* pp, int n, int E, int* counts,
                                                          float* prob_sum) {
  __shared__ int s_c[32][32];
  __shared__ float s_f[32][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = blockIdx.x * 32 + lane;
  int c = 0;
  float f = 0.0f;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // partials in flight; 16 need the registers of a whole SM, so that the launch cannot take its place early (1 us more),
  // and a loop without bounds checks has its last few one after the other (1.1 us more)
  constexpr int B = 8;
  if (e < E) {
    for (int i0 = warp; i0 < n; i0 += 32 * B) {
      int vc[B];
      float vf[B];
#pragma unroll
      for (int q = 0; q < B; ++q) {
        const int i = i0 + 32 * q;
        vc[q] = pc && i < n ? pc[(size_t)i * E + e] : 0;
        vf[q] = pp && i < n ? pp[(size_t)i * E + e] : 0.0f;
      }
#pragma unroll
      for (int q = 0; q < B; ++q) c += vc[q], f += vf[q];
    }
  }
  s_c[warp][lane] = c;
  s_f[warp][lane] = f;
  __syncthreads();
  if (warp == 0 && e < E) {
    c = 0;
    f = 0.0f;
#pragma unroll
    for (int w = 0; w < 32; ++w) {
      c += s_c[w][lane];
      f += s_f[w][lane];
    }
    if (counts) counts[e] = c;
    if (prob_sum) prob_sum[e] = f;
  }
}

// ------------------------------------------------------------------ gradient
struct RouteBwdParams {
  const void* logits;
  void* dlogits;
  int64_t ld, dld, T;
  int E, k, dtype, vec, dvec, renorm;
  int rows, more, ks;  // as in RouteParams
  float scale;
  const int* topk_idx;
  const float* dtopk_w;
  const float* dprob_sum;
};

// With q_i = s_i / sum_sel s over the selected, P_e = s_e / sum s over the row:
//   renormalised:  a_i = scale q_i (dw_i - sum_j q_j dw_j);  else a_i = scale s_i dw_i
//   c_e = P_e (d_e - sum_f P_f d_f), d the gradient of prob_sum
//   sigmoid: dx_e = (a_e + c_e) (1 - s_e)
//   softmax: dx_e = a_e + c_e, less s_e sum_i a_i where not renormalised
// (a and c are ds_e times s_e, so nothing is divided by a small score.)
// A row is read once and written once.  The selected experts' terms are made
// for several rows at once, one lane per slot (32 >> ks rows), and meet the
// row's through shared memory.  Renormalised weights, and sigmoid ones, without
// prob_sum need the selected logits only, so the row itself is not read.
// 16384 x 256 fp32 with prob_sum: 9.6 us (33.5 MB at the copy rate would be
// 5.1 us; what is left is the latency of a row's load and reductions, four to
// five rows a warp), without 6.4 us; 32768 x 384 bf16: 19.0 us (7.8).
template <int V, bool kSoft>
__global__ void __launch_bounds__(ROUTE_WARPS * 32, route_ctas_per_sm(V)) route_bwd_kernel(const __grid_constant__ RouteBwdParams p) {
  __shared__ __align__(16) float s_a[ROUTE_WARPS][32 * V];
  __shared__ float s_ai[ROUTE_WARPS][32];
  __shared__ int s_e[ROUTE_WARPS][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e0 = lane * V;
  const bool sums = p.dprob_sum != nullptr, dense = sums || (kSoft && !p.renorm);
  const int size = p.dtype == MOE_DTYPE_FP32 ? 4 : 2, slots = 1 << p.ks;
  float* a = s_a[warp];
  float d[V];
  asm volatile("griddepcontrol.wait;" ::: "memory");  // for what is before this launch, see launch_early
#pragma unroll
  for (int j = 0; j < V; ++j) {
    a[j * 32 + lane] = 0.0f;
    d[j] = sums && e0 + j < p.E ? p.dprob_sum[e0 + j] : 0.0f;
  }
  __syncwarp();
  const int wid = blockIdx.x * ROUTE_WARPS + warp;
  const int64_t t_from = (int64_t)wid * p.rows + min(wid, p.more), t_to = t_from + p.rows + (wid < p.more ? 1 : 0);
  for (int64_t tb = t_from; tb < t_to; tb += 32 >> p.ks) {
    const int n_rows = (int)min((int64_t)(32 >> p.ks), t_to - tb);
    {  // the selected experts' a (softmax not renormalised: dw, the row's scores follow below)
      const int r = lane >> p.ks, slot = lane & (slots - 1);
      int e = -1;
      float dw = 0.0f, xs = -INFINITY;
      if (r < n_rows && slot < p.k) {
        e = p.topk_idx[(tb + r) * p.k + slot];
        if (e < 0 || e >= p.E) e = -1;
      }
      if (e >= 0) {
        dw = p.dtopk_w[(tb + r) * p.k + slot] * p.scale;
        xs = load_logit(static_cast<const uint8_t*>(p.logits) + (size_t)(tb + r) * p.ld * size, p.dtype, e);
      }
      const bool on = e >= 0 && !(xs == -INFINITY);
      float ai = 0.0f;
      if (p.renorm) {
        float ms = xs;
        for (int o = slots >> 1; o > 0; o >>= 1) ms = fmaxf(ms, __shfl_xor_sync(0xffffffffu, ms, o));
        float q = 0.0f;
        if (on) q = kSoft || ms < -20.0f ? expf(below(xs, ms)) : 1.0f / (1.0f + expf(-xs));
        float tot = q;
        for (int o = slots >> 1; o > 0; o >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, o);
        q = tot == 0.0f ? 0.0f : q / tot;  // (one expert: exactly 1, so that its gradient is 0)
        float qd = q * dw;
        for (int o = slots >> 1; o > 0; o >>= 1) qd += __shfl_xor_sync(0xffffffffu, qd, o);
        ai = q * (dw - qd);
      } else if (on) {
        ai = kSoft ? dw : dw / (1.0f + expf(-xs));
      }
      if (!kSoft && !dense && on) ai /= 1.0f + expf(xs);  // times 1 - s
      s_ai[warp][lane] = ai;
      s_e[warp][lane] = e;
      __syncwarp();
    }
    for (int r = 0; r < n_rows; ++r) {
      const int64_t t = tb + r;
      const int e = lane < p.k ? s_e[warp][(r << p.ks) + lane] : -1;
      if (e >= 0) a[e] = s_ai[warp][(r << p.ks) + lane];
      __syncwarp();
      float o[V];
#pragma unroll
      for (int j = 0; j < V; ++j) o[j] = a[e0 + j];
      if (dense) {
        float x[V], s[V], c1[V];  // c1: 1 - s
        load_row<V>(static_cast<const uint8_t*>(p.logits) + (size_t)t * p.ld * size, p.dtype, p.vec, lane, p.E, x);
        auto row_max = [&]() {
          float lm = -INFINITY;
#pragma unroll
          for (int j = 0; j < V; ++j) lm = fmaxf(lm, x[j]);
          return max32(lm);
        };
        float z = 0.0f;
        if (kSoft) {
          const float m = row_max();
#pragma unroll
          for (int j = 0; j < V; ++j) {
            s[j] = x[j] == m ? 1.0f : exp2_fast((x[j] - m) * LOG2E);
            if (x[j] == -INFINITY) s[j] = 0.0f;
            z += s[j];
          }
          z = sum32(z);
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const float y = exp2_fast(-fabsf(x[j]) * LOG2E), h = rcp_fast(1.0f + y);  // e^-|x|: s and 1 - s keep their bits
            s[j] = x[j] >= 0.0f ? h : y * h;
            c1[j] = x[j] >= 0.0f ? y * h : h;
            z += s[j];
          }
          z = sum32(z);
          if (z < 1e-6f) {  // scores that may underflow: e^x there, so the share is softmax's
            const float m = row_max();
            if (m < -20.0f && m > -INFINITY) {
              z = 0.0f;
#pragma unroll
              for (int j = 0; j < V; ++j) {
                s[j] = exp2_fast((x[j] - m) * LOG2E);
                z += s[j];
              }
              z = sum32(z);
            }
          }
        }
        const float inv_z = z == 0.0f ? 0.0f : rcp_fast(z);
#pragma unroll
        for (int j = 0; j < V; ++j) s[j] *= inv_z;  // normalised
        if (kSoft && !p.renorm) {
          float asum = 0.0f;
#pragma unroll
          for (int j = 0; j < V; ++j) asum += o[j] * s[j];
          asum = sum32(asum);
#pragma unroll
          for (int j = 0; j < V; ++j) o[j] = s[j] * (o[j] - asum);
        }
        if (sums) {
          float ld = 0.0f;
#pragma unroll
          for (int j = 0; j < V; ++j) ld += s[j] * d[j];
          ld = sum32(ld);
#pragma unroll
          for (int j = 0; j < V; ++j) o[j] += s[j] * (d[j] - ld);
        }
        if (!kSoft) {
#pragma unroll
          for (int j = 0; j < V; ++j) o[j] *= c1[j];
        }
      }
      // one rounding to the logits' type
      uint8_t* out = static_cast<uint8_t*>(p.dlogits) + (size_t)t * p.dld * size;
      if (p.dtype == MOE_DTYPE_FP32) {
        float* dst = reinterpret_cast<float*>(out) + e0;
        if (V % 4 == 0 && p.dvec && e0 + V <= p.E) {
#pragma unroll
          for (int i = 0; i < V / 4; ++i)
            reinterpret_cast<float4*>(dst)[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j)
            if (e0 + j < p.E) dst[j] = o[j];
        }
      } else {
        uint16_t h[V + 1];
#pragma unroll
        for (int j = 0; j < V; ++j)
          h[j] = p.dtype == MOE_DTYPE_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(o[j]))
                                           : __half_as_ushort(__float2half_rn(o[j]));
        uint16_t* dst = reinterpret_cast<uint16_t*>(out) + e0;
        if (V % 4 == 0 && p.dvec && e0 + V <= p.E) {
#pragma unroll
          for (int i = 0; i < V / 4; ++i)
            reinterpret_cast<uint2*>(dst)[i] = make_uint2((uint32_t)h[4 * i] | ((uint32_t)h[4 * i + 1] << 16),
                                                          (uint32_t)h[4 * i + 2] | ((uint32_t)h[4 * i + 3] << 16));
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j)
            if (e0 + j < p.E) dst[j] = h[j];
        }
      }
      __syncwarp();
      if (e >= 0) a[e] = 0.0f;
      __syncwarp();
    }
  }
}

// ------------------------------------------------------------------ routing given to the layer
// What the built-in router leaves for the schedule, from a given routing: the
// experts and weights of every slot, the route histogram of every 128-token
// chunk, and the persistent kernel's counters and stamps as they start.  One
// thread per token.  Every slot gets an expert of its own, since the layer
// takes k distinct routes per token: an empty slot (or one whose index is out
// of range or a repetition) the lowest expert that the token does not use,
// with weight 0 and a mark in topk_logit.
__global__ void __launch_bounds__(BM) given_routes_kernel(const __grid_constant__ FwdParams p, const int* idx, const float* wt) {
  __shared__ int s_hist[E_MAX];
  const int t = blockIdx.x * BM + threadIdx.x;
  for (int i = blockIdx.x * BM + threadIdx.x; i < p.n_counters; i += gridDim.x * BM) p.counters[i] = 0;
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.stamps) {
    p.stamps[STAMP_START] = p.stamps[STAMP_COMBINE_START] = ~0ull;
    p.stamps[STAMP_LAST_FILL] = p.stamps[STAMP_COMBINE_END] = 0ull;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.status + 1, FLAG_ROUTES_GIVEN);
  for (int e = threadIdx.x; e < p.E; e += BM) s_hist[e] = 0;
  __syncthreads();
  if (t < p.T) {
    int ex[TOPK_MAX];
    bool bad = false;
#pragma unroll
    for (int s = 0; s < TOPK_MAX; ++s) {
      ex[s] = -1;
      if (s < p.k) {
        const int e = idx[(size_t)t * p.k + s];
        bool ok = e >= 0 && e < p.E;
        bad |= !ok && e != -1;
#pragma unroll
        for (int q = 0; q < s; ++q)
          if (ok && ex[q] == e) ok = false, bad = true;
        ex[s] = ok ? e : -1;
      }
    }
    int next = 0;  // the lowest expert not looked at yet (k <= E: one is always left)
#pragma unroll
    for (int s = 0; s < TOPK_MAX; ++s) {
      if (s >= p.k) break;
      const bool fill = ex[s] < 0;
      if (fill) {
        for (bool used = true; used; ++next) {
          used = false;
#pragma unroll
          for (int q = 0; q < TOPK_MAX; ++q) used |= ex[q] == next;
        }
        ex[s] = next - 1;
      }
      const size_t o = (size_t)t * p.k + s;
      p.topk_idx[o] = ex[s];
      p.topk_w[o] = fill ? 0.0f : wt[o];
      p.topk_logit[o] = fill ? 1.0f : 0.0f;
      atomicAdd(&s_hist[ex[s]], 1);
    }
    if (bad) atomicOr(p.status + 1, FLAG_ROUTES_INVALID);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += BM) p.chunk_counts[(size_t)blockIdx.x * p.E + e] = s_hist[e];
}

// MXFP8 plans: x in 32-element blocks (OCP MX E4M3 codes, E8M0 scales), as the
// router pass leaves it; a thread per block.
__global__ void __launch_bounds__(256) quantize_rows_kernel(const bf16* x, int64_t blocks, uint8_t* xq, uint8_t* xs) {
  for (int64_t b = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; b < blocks; b += (int64_t)gridDim.x * blockDim.x) {
    float v[32];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(x + b * 32) + i);
      const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&w);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = __bfloat1622float2(h[j]);
        v[8 * i + 2 * j] = f.x;
        v[8 * i + 2 * j + 1] = f.y;
      }
    }
    uint32_t c[8];
    xs[b] = (uint8_t)mx_quantize32(v, c);
    uint4* d = reinterpret_cast<uint4*>(xq + b * 32);
    d[0] = make_uint4(c[0], c[1], c[2], c[3]);
    d[1] = make_uint4(c[4], c[5], c[6], c[7]);
  }
}

cudaError_t launch_given_routes(const FwdParams& p, const int* topk_idx, const float* topk_w, cudaStream_t stream) {
  cudaError_t err = cudaMemsetAsync(p.status, 0, 2 * sizeof(int), stream);  // status and warning bits
  if (err != cudaSuccess) return err;
  given_routes_kernel<<<p.n_chunks, BM, 0, stream>>>(p, topk_idx, topk_w);
  err = cudaGetLastError();
  if (err != cudaSuccess || !p.xq) return err;
  const int64_t blocks = (int64_t)p.T * p.D / 32, grid = (blocks + 255) / 256;
  quantize_rows_kernel<<<(unsigned)(grid < 152 * 16 ? grid : 152 * 16), 256, 0, stream>>>(p.x, blocks, p.xq, p.xs);
  return cudaGetLastError();
}

}  // namespace moe

// ------------------------------------------------------------------ C ABI
using namespace moe;

struct moe_route_plan {
  moe_route_config cfg;
  int device, num_sms;
};

namespace {

size_t dtype_size(int d) { return d == MOE_DTYPE_FP32 ? 4 : 2; }
bool route_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// CTAs of a forward over T rows: enough for every row, at most what the GPU
// keeps resident (each CTA's sums over its rows are one partial result)
int64_t route_grid(const moe_route_plan* pl, int64_t T) {
  const int64_t need = (T + ROUTE_WARPS - 1) / ROUTE_WARPS, most = (int64_t)pl->num_sms * route_ctas_per_sm((int)(pl->cfg.E + 31) / 32);
  return need < most ? need : most;
}

template <typename F>
cudaError_t by_width(int E, F&& f) {
  const int v = (E + 31) / 32;  // experts per lane
  if (v <= 1) return f(std::integral_constant<int, 1>{});
  if (v <= 2) return f(std::integral_constant<int, 2>{});
  if (v <= 4) return f(std::integral_constant<int, 4>{});
  if (v <= 8) return f(std::integral_constant<int, 8>{});
  if (v <= 12) return f(std::integral_constant<int, 12>{});
  return f(std::integral_constant<int, 16>{});
}

// Launch; the grid is set up while what is before it on the stream still runs,
// and waits for that itself (a chain of single-token calls: 6.15 us a call
// without, 4.5 us with; 4.0 us in a graph, where the host's 3.8 us do not count).
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), unsigned grid, unsigned threads, cudaStream_t st, const A&... a) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(grid);
  lc.blockDim = dim3(threads);
  lc.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = at;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, kernel, (P)a...);
}

bool on_device(const moe_route_plan* pl) {
  int cur = -1;
  return cudaGetDevice(&cur) == cudaSuccess && cur == pl->device;
}

}  // namespace

extern "C" {

int moe_route_plan_create(const moe_route_config* cfg, moe_route_plan** out) {
  if (!cfg || !out) return MOE_ERR_INVALID_ARG;
  *out = nullptr;
  moe_route_config c = *cfg;
  if (c.score_fn != MOE_SCORE_SIGMOID && c.score_fn != MOE_SCORE_SOFTMAX) return MOE_ERR_INVALID_ARG;
  if (c.logits_dtype < MOE_DTYPE_FP32 || c.logits_dtype > MOE_DTYPE_FP16) return MOE_ERR_INVALID_ARG;
  if (c.renormalize != 0 && c.renormalize != 1) return MOE_ERR_INVALID_ARG;
  if (c.group_top != 1 && c.group_top != 2) return MOE_ERR_INVALID_ARG;
  if (!(c.scale - c.scale == 0.0f)) return MOE_ERR_INVALID_ARG;  // finite
  if (c.E < 1 || c.E > E_MAX || c.k < 1 || c.k > TOPK_MAX) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (c.n_group < 1 || c.n_group > 32 || c.E % c.n_group || c.topk_group < 1 || c.topk_group > c.n_group ||
      c.k > c.topk_group * (c.E / c.n_group))
    return MOE_ERR_UNSUPPORTED_SHAPE;
  int dev = 0, sms = 0, major = 0, minor = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
    return MOE_ERR_CUDA;
  if (major != 10 || minor != 3) return MOE_ERR_UNSUPPORTED_DEVICE;
  moe_route_plan* pl = new (std::nothrow) moe_route_plan;
  if (!pl) return MOE_ERR_INVALID_ARG;
  pl->cfg = c;
  pl->device = dev;
  pl->num_sms = sms;
  *out = pl;
  return MOE_OK;
}

int moe_route_plan_destroy(moe_route_plan* plan) {
  delete plan;
  return MOE_OK;
}

size_t moe_route_workspace_bytes(const moe_route_plan* plan, int64_t T) {
  if (!plan || T < 0) return 0;
  const int64_t grid = route_grid(plan, T);
  return grid > 1 ? (size_t)grid * plan->cfg.E * 8 : 256;  // per CTA: counts (int32) and score sums (fp32)
}

int moe_route(const moe_route_plan* pl, int64_t T, const void* logits, int64_t logits_stride, const float* bias,
              int32_t* topk_idx, float* topk_w, int32_t* expert_counts, float* prob_sum, void* workspace,
              size_t workspace_bytes, moe_stream_t stream_) {
  if (!pl || T < 0) return MOE_ERR_INVALID_ARG;
  const moe_route_config& c = pl->cfg;
  cudaStream_t stream = (cudaStream_t)stream_;
  if (logits_stride == 0) logits_stride = c.E;
  if (logits_stride < c.E || T > (int64_t)1 << 40 || logits_stride > (int64_t)1 << 20) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!logits || !topk_idx || !topk_w || !route_aligned(logits, dtype_size(c.logits_dtype)) ||
                !route_aligned(topk_idx, 4) || !route_aligned(topk_w, 4)))
    return MOE_ERR_INVALID_ARG;
  if (!route_aligned(bias, 4) || !route_aligned(expert_counts, 4) || !route_aligned(prob_sum, 4)) return MOE_ERR_INVALID_ARG;
  const int64_t grid = route_grid(pl, T);
  const bool sums = expert_counts || prob_sum, split = sums && grid > 1;
  if (split) {
    if (!workspace || !route_aligned(workspace, 16)) return MOE_ERR_INVALID_ARG;
    if (workspace_bytes < moe_route_workspace_bytes(pl, T)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  }
  if (!on_device(pl)) return MOE_ERR_INVALID_ARG;
  if (T == 0) {  // nothing to route; the sums of no tokens are zero
    if (expert_counts && cudaMemsetAsync(expert_counts, 0, 4 * c.E, stream) != cudaSuccess) return MOE_ERR_CUDA;
    if (prob_sum && cudaMemsetAsync(prob_sum, 0, 4 * c.E, stream) != cudaSuccess) return MOE_ERR_CUDA;
    return MOE_OK;
  }
  RouteParams p{};
  p.logits = logits;
  p.ld = logits_stride;
  p.T = T;
  p.E = (int)c.E;
  p.k = (int)c.k;
  p.dtype = c.logits_dtype;
  p.vec = route_aligned(logits, 16) && logits_stride * (int64_t)dtype_size(c.logits_dtype) % 16 == 0;
  p.bias = bias;
  p.n_group = (int)c.n_group;
  p.topk_group = (int)c.topk_group;
  p.group_top = c.group_top;
  p.gs = (int)(c.E / c.n_group);
  p.renorm = c.renormalize;
  p.rows = (int)(T / (grid * ROUTE_WARPS));
  p.more = (int)(T % (grid * ROUTE_WARPS));
  while ((1 << p.ks) < p.k) ++p.ks;
  p.scale = c.scale;
  p.topk_idx = topk_idx;
  p.topk_w = topk_w;
  int* pc = split ? static_cast<int*>(workspace) : nullptr;
  float* pp = split ? static_cast<float*>(workspace) + grid * c.E : nullptr;
  p.split = split;
  p.counts = expert_counts ? (split ? pc : expert_counts) : nullptr;
  p.prob_sum = prob_sum ? (split ? pp : prob_sum) : nullptr;
  auto launch = [&](auto soft) {
    return by_width(p.E, [&](auto v) {
      return launch_early(route_kernel<decltype(v)::value, decltype(soft)::value>, (unsigned)grid, ROUTE_WARPS * 32, stream, p);
    });
  };
  const cudaError_t err = c.score_fn == MOE_SCORE_SOFTMAX ? launch(std::true_type{}) : launch(std::false_type{});
  if (err != cudaSuccess) return MOE_ERR_CUDA;
  if (split) {
    if (launch_early(route_sums_kernel, (unsigned)((c.E + 31) / 32), 1024, stream, expert_counts ? (const int*)pc : nullptr,
                     prob_sum ? (const float*)pp : nullptr, (int)grid, p.E, (int*)expert_counts, prob_sum) != cudaSuccess)
      return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

int moe_route_bwd(const moe_route_plan* pl, int64_t T, const void* logits, int64_t logits_stride,
                  const int32_t* topk_idx, const float* dtopk_w, const float* dprob_sum, void* dlogits,
                  int64_t dlogits_stride, moe_stream_t stream_) {
  if (!pl || T < 0) return MOE_ERR_INVALID_ARG;
  const moe_route_config& c = pl->cfg;
  cudaStream_t stream = (cudaStream_t)stream_;
  const size_t size = dtype_size(c.logits_dtype);
  if (logits_stride == 0) logits_stride = c.E;
  if (dlogits_stride == 0) dlogits_stride = c.E;
  if (logits_stride < c.E || dlogits_stride < c.E || T > (int64_t)1 << 40 || logits_stride > (int64_t)1 << 20 ||
      dlogits_stride > (int64_t)1 << 20)
    return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!logits || !topk_idx || !dtopk_w || !dlogits || !route_aligned(logits, size) ||
                !route_aligned(dlogits, size) || !route_aligned(topk_idx, 4) || !route_aligned(dtopk_w, 4)))
    return MOE_ERR_INVALID_ARG;
  if (!route_aligned(dprob_sum, 4)) return MOE_ERR_INVALID_ARG;
  if (!on_device(pl)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  RouteBwdParams p{};
  p.logits = logits;
  p.dlogits = dlogits;
  p.ld = logits_stride;
  p.dld = dlogits_stride;
  p.T = T;
  p.E = (int)c.E;
  p.k = (int)c.k;
  p.dtype = c.logits_dtype;
  p.vec = route_aligned(logits, 16) && logits_stride * (int64_t)size % 16 == 0;
  p.dvec = route_aligned(dlogits, 16) && dlogits_stride * (int64_t)size % 16 == 0;
  p.renorm = c.renormalize;
  p.scale = c.scale;
  p.topk_idx = topk_idx;
  p.dtopk_w = dtopk_w;
  p.dprob_sum = dprob_sum;
  int64_t grid = (T + ROUTE_WARPS - 1) / ROUTE_WARPS;
  const int64_t most = (int64_t)pl->num_sms * (p.E <= 128 ? 5 : route_ctas_per_sm((p.E + 31) / 32));  // what stays resident
  if (grid > most) grid = most;
  p.rows = (int)(T / (grid * ROUTE_WARPS));
  p.more = (int)(T % (grid * ROUTE_WARPS));
  while ((1 << p.ks) < p.k) ++p.ks;
  auto launch = [&](auto soft) {
    return by_width(p.E, [&](auto v) {
      return launch_early(route_bwd_kernel<decltype(v)::value, decltype(soft)::value>, (unsigned)grid, ROUTE_WARPS * 32, stream, p);
    });
  };
  const cudaError_t err = c.score_fn == MOE_SCORE_SOFTMAX ? launch(std::true_type{}) : launch(std::false_type{});
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
