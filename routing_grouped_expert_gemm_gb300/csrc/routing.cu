// Routing to experts from given logits, and its gradient (moe_route,
// moe_route_bwd in include/moe.h).
//
// Row t of the logits x gives scores s_e = sigmoid(x_e), or softmax over the
// row; a logit of -inf has score 0 and is never selected.  The selection ranks
// key_e = s_e + b_e (without a bias: x itself, which both score functions
// keep in order), inside the topk_group groups whose sums of the group_top
// largest keys are largest; the weights come from s alone.
//
// The selection is that of exact arithmetic.  Keys are computed in fp32 with a
// known error; where a value on the losing side of the border (of the kept
// groups, or of the k-th key) lies within that error of the border, and is not
// an exact tie (the same logit and bias, decided by the lower id), the warp
// decides the row again in fp64.  About one row in 1000 is that close with
// fp32 logits, so the fp64 units do not show in the time; fp32 alone would
// pick another expert in some rows of a large batch.
//
// One warp per row, 8 rows in flight per CTA, lane l holding the V consecutive
// experts l V .. l V + V - 1 in registers: a row is read once, in 16-byte
// loads, and nothing but the results is written.  Consecutive experts per lane
// make "lowest id" the same as "lowest lane", so a tie costs nothing, and make
// a group a set of neighbouring lanes.
#include <cuda_fp16.h>

#include <new>
#include <type_traits>

#include "../../include/moe.h"
#include "common.cuh"

namespace moe {

constexpr int ROUTE_WARPS = 8;          // rows in flight per CTA
constexpr int ROUTE_CTAS_PER_SM = 4;    // of the persistent grid that sums over tokens
constexpr float ROUTE_TINY = 1e-36f;    // keys below this have lost their relative precision (fp32 underflow)

struct RouteParams {
  const void* logits;
  int64_t ld, T;  // row stride in elements
  int E, k, dtype, vec;
  const float* bias;
  int n_group, topk_group, group_top, gs, renorm;
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
// vectors of the largest power of two that divides its bytes.
template <int V>
__device__ __forceinline__ void load_row(const void* row, int dtype, int vec, int lane, int E, float (&x)[V]) {
  const int e0 = lane * V;
  if (vec && e0 + V <= E) {
    if (dtype == MOE_DTYPE_FP32) {
      const float* s = static_cast<const float*>(row) + e0;
      if constexpr (V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
          const float4 w = __ldg(reinterpret_cast<const float4*>(s) + i);
          x[4 * i] = w.x, x[4 * i + 1] = w.y, x[4 * i + 2] = w.z, x[4 * i + 3] = w.w;
        }
      } else if constexpr (V % 2 == 0) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
          const float2 w = __ldg(reinterpret_cast<const float2*>(s) + i);
          x[2 * i] = w.x, x[2 * i + 1] = w.y;
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = __ldg(s + i);
      }
      return;
    }
    uint32_t w[(V + 1) / 2];
    const uint16_t* s = static_cast<const uint16_t*>(row) + e0;
    if constexpr (V % 8 == 0) {
#pragma unroll
      for (int i = 0; i < V / 8; ++i) {
        const uint4 q = __ldg(reinterpret_cast<const uint4*>(s) + i);
        w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
      }
    } else if constexpr (V % 4 == 0) {
#pragma unroll
      for (int i = 0; i < V / 4; ++i) {
        const uint2 q = __ldg(reinterpret_cast<const uint2*>(s) + i);
        w[2 * i] = q.x, w[2 * i + 1] = q.y;
      }
    } else if constexpr (V % 2 == 0) {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) w[i] = __ldg(reinterpret_cast<const uint32_t*>(s) + i);
    } else {
      w[0] = __ldg(s);
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

// Floats in the order of unsigned integers; nothing finite or infinite maps to 0.
__device__ __forceinline__ uint32_t ord_of(float f) {
  const uint32_t u = __float_as_uint(f + 0.0f);  // -0 equals +0
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float ord_to(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
}

__device__ __forceinline__ float sum32(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float sum16(float v) {  // both halves of the warp alike
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float max32(float v) {  // NaN operands are passed over
  return ord_to(__reduce_max_sync(0xffffffffu, ord_of(v == v ? v : -INFINITY)));
}
// x - m where an infinite maximum is its own limit (0), not NaN
__device__ __forceinline__ float below(float x, float m) { return x == m ? 0.0f : x - m; }

// ------------------------------------------------------------------ the decision in fp64
__device__ __forceinline__ double shfl_xor_d(double v, int o) { return __shfl_xor_sync(0xffffffffu, v, o); }
__device__ __forceinline__ double max32d(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmax(v, shfl_xor_d(v, o));
  return v;
}

// Which of this lane's V experts are selected, as bits, computed in fp64 from
// the row in memory.  Whole warp.
template <int V, bool kSoft>
__device__ __noinline__ uint32_t select_fp64(const RouteParams& p, const void* row) {
  const int lane = threadIdx.x & 31, e0 = lane * V;
  double key[V];
  uint32_t live = 0;
  double m = -INFINITY;
  for (int j = 0; j < V; ++j) {
    const double x = e0 + j < p.E ? (double)load_logit(row, p.dtype, e0 + j) : -INFINITY;
    key[j] = x;
    if (x > -INFINITY) {
      live |= 1u << j;
      m = fmax(m, x);
    }
  }
  m = max32d(m);
  double z = 0.0;
  for (int j = 0; j < V; ++j) {
    if (!((live >> j) & 1)) continue;
    if (kSoft) {
      key[j] = exp(key[j] == m ? 0.0 : key[j] - m);
      z += key[j];
    } else {
      key[j] = 1.0 / (1.0 + exp(-key[j]));
    }
  }
  if (kSoft)
    for (int o = 16; o > 0; o >>= 1) z += shfl_xor_d(z, o);
  for (int j = 0; j < V; ++j) {
    if (!((live >> j) & 1)) continue;
    if (kSoft) key[j] /= z;
    if (p.bias) key[j] += (double)p.bias[e0 + j];
    if (!(key[j] > -INFINITY)) live &= ~(1u << j);
  }
  if (p.n_group > 1) {
    double mine = -INFINITY;  // lane g: the score of group g
    for (int g = 0; g < p.n_group; ++g) {
      double b1 = -INFINITY, b2 = -INFINITY;
      for (int j = 0; j < V; ++j) {
        if (!((live >> j) & 1) || (e0 + j) / p.gs != g) continue;
        if (key[j] > b1) b2 = b1, b1 = key[j];
        else if (key[j] > b2) b2 = key[j];
      }
      const double t1 = max32d(b1);
      const unsigned own = __ballot_sync(0xffffffffu, b1 == t1);
      const double t2 = max32d(lane == __ffs(own) - 1 ? b2 : b1);
      const double s = p.group_top > 1 && t2 > -INFINITY ? t1 + t2 : t1;
      if (lane == g) mine = s;
    }
    int rank = 0;
    for (int g = 0; g < p.n_group; ++g) {
      const double s = __shfl_sync(0xffffffffu, mine, g);
      rank += (s > mine || (s == mine && g < lane)) ? 1 : 0;
    }
    const unsigned kept = __ballot_sync(0xffffffffu, lane < p.n_group && rank < p.topk_group);
    for (int j = 0; j < V; ++j)
      if (e0 + j < p.E && !((kept >> ((e0 + j) / p.gs)) & 1u)) live &= ~(1u << j);
    if (!p.bias)  // without a bias the order is the logits'
      for (int j = 0; j < V; ++j)
        if ((live >> j) & 1) key[j] = (double)load_logit(row, p.dtype, e0 + j);
  }
  uint32_t sel = 0;
  for (int i = 0; i < p.k; ++i) {
    double b = -INFINITY;
    int bj = -1;
    for (int j = 0; j < V; ++j)
      if (((live >> j) & 1) && (bj < 0 || key[j] > b)) b = key[j], bj = j;
    const double t = max32d(b);
    const unsigned own = __ballot_sync(0xffffffffu, bj >= 0 && b == t);
    if (!own) break;
    if (lane == __ffs(own) - 1) {
      sel |= 1u << bj;
      live &= ~(1u << bj);
    }
  }
  return sel;
}

// ------------------------------------------------------------------ forward
// A row without a border close enough to matter is decided in fp32.  Error of
// a key: sigmoid, 4 ulp of s (expf 2, sum and quotient 1 each) plus the
// rounding of s + b: below 2^-20 (|key| + max |b|) for both sides of a
// comparison.  Softmax adds the rounding of x - m, (m - x) 2^-24 relative and
// at most 104 before exp underflows: below 2^-16.
template <int V, bool kSoft>
__global__ void __launch_bounds__(ROUTE_WARPS * 32) route_kernel(const RouteParams p) {
  constexpr float REL = kSoft ? 1.0f / 65536 : 1.0f / 1048576;
  __shared__ int s_hist[E_MAX];
  __shared__ int s_e[ROUTE_WARPS][TOPK_MAX];
  __shared__ float s_x[ROUTE_WARPS][TOPK_MAX];
  __shared__ float s_p[ROUTE_WARPS][E_MAX];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e0 = lane * V;
  const bool sums = p.prob_sum != nullptr, grouped = p.n_group > 1;
  const bool with_keys = p.bias != nullptr;                                // the order is s + b's, not x's
  const bool group_scores = grouped && (with_keys || p.group_top > 1);     // groups are ranked by computed values
  // groups made of whole, aligned sets of lanes are ranked by butterflies
  const int glanes = p.gs / V;
  const bool aligned_groups = grouped && p.gs % V == 0 && (glanes & (glanes - 1)) == 0 && glanes <= 32;
  if (p.counts) {
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) s_hist[e] = 0;
    __syncthreads();
  }
  float b[V], bmax = 0.0f, acc[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    b[j] = with_keys && e0 + j < p.E ? p.bias[e0 + j] : 0.0f;
    bmax = fmaxf(bmax, fabsf(b[j]));
    acc[j] = 0.0f;
  }
  bmax = max32(bmax);
  const size_t row_bytes = (size_t)p.ld * (p.dtype == MOE_DTYPE_FP32 ? 4 : 2);

  for (int64_t t = (int64_t)blockIdx.x * ROUTE_WARPS + warp; t < p.T; t += (int64_t)gridDim.x * ROUTE_WARPS) {
    const void* row = static_cast<const uint8_t*>(p.logits) + (size_t)t * row_bytes;
    float x[V];
    load_row<V>(row, p.dtype, p.vec, lane, p.E, x);

    // scores: s (sigmoid) or e^(x - m) (softmax; z is the row's sum), where anything needs them
    float s[V];
    float m = 0.0f, z = 1.0f;
    bool nan_row = false;
    if (kSoft || sums) {
      float lm = -INFINITY;
      bool nan = false;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        lm = fmaxf(lm, x[j]);
        nan |= x[j] != x[j];
      }
      m = max32(lm);
      nan_row = __any_sync(0xffffffffu, nan);
    }
    if (kSoft ? (with_keys || sums || group_scores || !p.renorm) : (with_keys || sums || group_scores)) {
      float lz = 0.0f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        s[j] = 0.0f;
        if (x[j] > -INFINITY) s[j] = kSoft ? expf(below(x[j], m)) : 1.0f / (1.0f + expf(-x[j]));
        lz += s[j];
      }
      if (kSoft || sums) z = sum32(lz);
    }
    if (sums) {  // normalised scores, s over the row's sum
      if (!kSoft && m < -20.0f && m > -INFINITY) {  // e^x to fp32 precision: shifted, so that it does not underflow
        float u[V], lz = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          u[j] = x[j] > -INFINITY ? expf(x[j] - m) : 0.0f;
          lz += u[j];
        }
        const float inv = 1.0f / sum32(lz);
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] += u[j] * inv;
      } else {
        const float inv = nan_row ? NAN : (z > 0.0f ? 1.0f / z : 0.0f);
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] += s[j] * inv;
      }
    }

    // order of the experts as integers, 0 = not to be selected
    uint32_t key[V];
    const float inv_z = kSoft ? (z > 0.0f ? 1.0f / z : 0.0f) : 1.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float f = x[j];
      if (with_keys) f = (kSoft ? s[j] * inv_z : s[j]) + b[j];
      key[j] = x[j] > -INFINITY && f > -INFINITY ? ord_of(f) : 0u;
    }

    bool close = false;  // some border is within the keys' error
    if (grouped) {
      // the two largest of each group; without a bias the (order-keeping) scores, or for the maximum alone x itself
      uint32_t gk[V];
#pragma unroll
      for (int j = 0; j < V; ++j) gk[j] = group_scores && !with_keys ? (key[j] ? ord_of(s[j]) : 0u) : key[j];
      uint32_t g1 = 0, g2 = 0;  // lane g: the largest two of group g
      if (aligned_groups) {
        uint32_t t1 = 0, t2 = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          t2 = max(t2, min(t1, gk[j]));
          t1 = max(t1, gk[j]);
        }
        for (int o = 1; o < glanes; o <<= 1) {
          const uint32_t u1 = __shfl_xor_sync(0xffffffffu, t1, o), u2 = __shfl_xor_sync(0xffffffffu, t2, o);
          t2 = max(max(t2, u2), min(t1, u1));
          t1 = max(t1, u1);
        }
        const int from = (lane * glanes) & 31;
        g1 = __shfl_sync(0xffffffffu, t1, from);
        g2 = __shfl_sync(0xffffffffu, t2, from);
        if (lane >= p.n_group) g1 = g2 = 0;
      } else {
        for (int g = 0; g < p.n_group; ++g) {
          const int lo = g * p.gs - e0, hi = lo + p.gs;
          uint32_t t1 = 0, t2 = 0;
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const uint32_t v = j >= lo && j < hi ? gk[j] : 0u;
            t2 = max(t2, min(t1, v));
            t1 = max(t1, v);
          }
          const uint32_t w1 = __reduce_max_sync(0xffffffffu, t1);
          const unsigned own = __ballot_sync(0xffffffffu, t1 == w1);
          const uint32_t w2 = __reduce_max_sync(0xffffffffu, lane == __ffs(own) - 1 ? t2 : t1);
          if (lane == g) g1 = w1, g2 = w2;
        }
      }
      // rank of lane g's group; a group without an expert ranks last
      uint32_t score = g1;
      if (group_scores && p.group_top > 1 && g2) score = ord_of(ord_to(g1) + ord_to(g2));
      int rank = 0;
      for (int g = 0; g < p.n_group; ++g) {
        const uint32_t v = __shfl_sync(0xffffffffu, score, g);
        rank += (v > score || (v == score && g < lane)) ? 1 : 0;
      }
      const bool in = lane < p.n_group && rank < p.topk_group;
      const unsigned kept = __ballot_sync(0xffffffffu, in);
      if (group_scores && p.topk_group < p.n_group) {
        const uint32_t lo = __reduce_min_sync(0xffffffffu, in ? score : 0xffffffffu);
        const uint32_t hi = __reduce_max_sync(0xffffffffu, in || lane >= p.n_group ? 0u : score);
        if (hi) {
          const float fl = ord_to(lo), fh = ord_to(hi);
          close = !(fl - fh > REL * (fabsf(fl) + 4.0f * bmax) + ROUTE_TINY);
        }
      }
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (e0 + j < p.E && !((kept >> ((e0 + j) / p.gs)) & 1u)) key[j] = 0;
    }

    // the k largest, the lowest id first among equals
    uint32_t sel = 0, lbest = 0, last = 0;
    int lj = 0, owner = 0;
    int n_sel = 0;
    auto scan = [&]() {
      lbest = 0;
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (key[j] > lbest && !((sel >> j) & 1u)) lbest = key[j], lj = j;
    };
    scan();
    for (; n_sel < p.k; ++n_sel) {
      const uint32_t best = __reduce_max_sync(0xffffffffu, lbest);
      if (!best) break;
      last = best;
      owner = __ffs(__ballot_sync(0xffffffffu, lbest == best)) - 1;
      if (lane == owner) {
        sel |= 1u << lj;
        scan();
      }
    }
    if (with_keys && n_sel == p.k) {
      // keys within the error of the k-th: unless all of them are the same logit and bias, it is too close
      const float fk = ord_to(last), tol = REL * (fabsf(fk) + bmax) + ROUTE_TINY;
      float lx = 0.0f, lb = 0.0f;
      bool some = false, mixed = false;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (key[j] && !(fabsf(ord_to(key[j]) - fk) > tol)) {
          mixed |= some && (x[j] != lx || b[j] != lb);
          lx = x[j], lb = b[j], some = true;
        }
      }
      const unsigned who = __ballot_sync(0xffffffffu, some);
      const int first = __ffs(who) - 1;  // (the k-th itself is among them)
      const float rx = __shfl_sync(0xffffffffu, lx, first), rb = __shfl_sync(0xffffffffu, lb, first);
      close |= __any_sync(0xffffffffu, mixed || (some && (lx != rx || lb != rb)));
    }
    if (close) sel = select_fp64<V, kSoft>(p, row);

    // slots in ascending id: one lane per slot
    const int mine = __popc(sel);
    int before = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += n;
    }
    n_sel = __shfl_sync(0xffffffffu, before, 31);
    before -= mine;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if ((sel >> j) & 1u) {
        s_e[warp][before] = e0 + j;
        s_x[warp][before] = x[j];
        ++before;
      }
    }
    __syncwarp();
    const bool on = lane < n_sel;
    const int e = on ? s_e[warp][lane] : -1;
    const float xs = on ? s_x[warp][lane] : -INFINITY;
    __syncwarp();
    float w = 0.0f;
    if (p.renorm) {  // over the selected: a common factor cancels, so scores that underflow are shifted
      const float ms = max32(xs);
      if (on) w = kSoft || ms < -20.0f ? expf(below(xs, ms)) : 1.0f / (1.0f + expf(-xs));
      const float tot = sum16(w);
      if (on) w = w / tot * p.scale;
    } else if (on) {
      w = (kSoft ? expf(below(xs, m)) * inv_z : 1.0f / (1.0f + expf(-xs))) * p.scale;
    }
    if (kSoft && nan_row && on) w = NAN;
    if (lane < p.k) {
      p.topk_idx[t * p.k + lane] = e;
      p.topk_w[t * p.k + lane] = w;
      if (p.counts && on) atomicAdd(&s_hist[e], 1);  // (integers: any order gives the same)
    }
  }

  if (p.counts || sums) {
    if (sums) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (e0 + j < p.E) s_p[warp][e0 + j] = acc[j];
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

// Sums over the CTAs' partials in a fixed order: a CTA per 32 experts, its
// warps taking every 8th partial, then the warps in turn.
__global__ void __launch_bounds__(256) route_sums_kernel(const int* pc, const float* pp, int n, int E, int* counts,
                                                         float* prob_sum) {
  __shared__ int s_c[8][32];
  __shared__ float s_f[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = blockIdx.x * 32 + lane;
  int c = 0;
  float f = 0.0f;
  if (e < E) {
#pragma unroll 4
    for (int i = warp; i < n; i += 8) {
      if (pc) c += pc[(size_t)i * E + e];
      if (pp) f += pp[(size_t)i * E + e];
    }
  }
  s_c[warp][lane] = c;
  s_f[warp][lane] = f;
  __syncthreads();
  if (warp == 0 && e < E) {
    c = 0;
    f = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
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
// A row is read once and written once; the selected experts' terms, one per
// lane, meet the row's through shared memory.  Renormalised weights without
// prob_sum need the selected logits only, so the row itself is not read.
template <int V, bool kSoft>
__global__ void __launch_bounds__(ROUTE_WARPS * 32) route_bwd_kernel(const RouteBwdParams p) {
  __shared__ __align__(16) float s_a[ROUTE_WARPS][32 * V];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e0 = lane * V;
  const bool sums = p.dprob_sum != nullptr, dense = sums || (kSoft && !p.renorm);
  const int size = p.dtype == MOE_DTYPE_FP32 ? 4 : 2;
  float* a = s_a[warp];
  float d[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    a[j * 32 + lane] = 0.0f;
    d[j] = sums && e0 + j < p.E ? p.dprob_sum[e0 + j] : 0.0f;
  }
  __syncwarp();
  for (int64_t t = (int64_t)blockIdx.x * ROUTE_WARPS + warp; t < p.T; t += (int64_t)gridDim.x * ROUTE_WARPS) {
    const void* row = static_cast<const uint8_t*>(p.logits) + (size_t)t * p.ld * size;
    float x[V], s[V];
    int e = -1;
    float dw = 0.0f, xs = -INFINITY;
    if (lane < p.k) {
      e = p.topk_idx[t * p.k + lane];
      if (e < 0 || e >= p.E) e = -1;
    }
    if (e >= 0) {
      dw = p.dtopk_w[t * p.k + lane] * p.scale;
      xs = load_logit(row, p.dtype, e);
    }
    float m = 0.0f, z = 1.0f;
    bool shifted = false;
    if (dense) {
      load_row<V>(row, p.dtype, p.vec, lane, p.E, x);
      float lm = -INFINITY, lz = 0.0f;
#pragma unroll
      for (int j = 0; j < V; ++j) lm = fmaxf(lm, x[j]);
      m = max32(lm);
      shifted = kSoft || (m < -20.0f && m > -INFINITY);  // sigmoid = e^x there: its share without underflow
#pragma unroll
      for (int j = 0; j < V; ++j) {
        s[j] = 0.0f;
        if (!(x[j] == -INFINITY)) s[j] = shifted ? expf(below(x[j], m)) : 1.0f / (1.0f + expf(-x[j]));
        lz += s[j];
      }
      z = sum32(lz);
    }
    const float inv_z = z == 0.0f ? 0.0f : 1.0f / z;

    // the selected experts' terms
    float ai = 0.0f;
    if (p.renorm) {
      const float ms = max32(xs);
      float q = 0.0f;
      if (e >= 0 && !(xs == -INFINITY)) q = kSoft || ms < -20.0f ? expf(below(xs, ms)) : 1.0f / (1.0f + expf(-xs));
      const float tot = sum16(q);
      q = tot == 0.0f ? 0.0f : q / tot;
      ai = q * (dw - sum16(q * dw));
    } else if (e >= 0 && !(xs == -INFINITY)) {
      ai = dw * (kSoft ? expf(below(xs, m)) * inv_z : 1.0f / (1.0f + expf(-xs)));
    }
    const float asum = kSoft && !p.renorm ? sum32(ai) : 0.0f;
    if (!kSoft && e >= 0 && !dense) ai *= 1.0f / (1.0f + expf(xs));  // 1 - s
    if (e >= 0) a[e] = ai;
    __syncwarp();

    float o[V];
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] = a[e0 + j];
    if (dense) {
      float ld = 0.0f;
      if (sums) {
#pragma unroll
        for (int j = 0; j < V; ++j) ld += s[j] * d[j];
        ld = sum32(ld) * inv_z;
      }
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float pe = s[j] * inv_z;
        o[j] -= kSoft ? pe * asum : 0.0f;
        if (sums) o[j] += pe * (d[j] - ld);
        if (!kSoft) o[j] *= 1.0f / (1.0f + expf(x[j]));  // 1 - s
        if (x[j] == -INFINITY) o[j] = 0.0f;
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
  const int64_t need = (T + ROUTE_WARPS - 1) / ROUTE_WARPS, most = (int64_t)pl->num_sms * ROUTE_CTAS_PER_SM;
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
  p.scale = c.scale;
  p.topk_idx = topk_idx;
  p.topk_w = topk_w;
  int* pc = split ? static_cast<int*>(workspace) : nullptr;
  float* pp = split ? static_cast<float*>(workspace) + grid * c.E : nullptr;
  p.counts = expert_counts ? (split ? pc : expert_counts) : nullptr;
  p.prob_sum = prob_sum ? (split ? pp : prob_sum) : nullptr;
  auto launch = [&](auto soft) {
    return by_width(p.E, [&](auto v) {
      route_kernel<decltype(v)::value, decltype(soft)::value><<<(unsigned)grid, ROUTE_WARPS * 32, 0, stream>>>(p);
      return cudaGetLastError();
    });
  };
  const cudaError_t err = c.score_fn == MOE_SCORE_SOFTMAX ? launch(std::true_type{}) : launch(std::false_type{});
  if (err != cudaSuccess) return MOE_ERR_CUDA;
  if (split) {
    route_sums_kernel<<<(unsigned)((c.E + 31) / 32), 256, 0, stream>>>(expert_counts ? pc : nullptr, prob_sum ? pp : nullptr,
                                                                     (int)grid, p.E, expert_counts, prob_sum);
    if (cudaGetLastError() != cudaSuccess) return MOE_ERR_CUDA;
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
  const int64_t most = (int64_t)pl->num_sms * 8;
  if (grid > most) grid = most;
  auto launch = [&](auto soft) {
    return by_width(p.E, [&](auto v) {
      route_bwd_kernel<decltype(v)::value, decltype(soft)::value><<<(unsigned)grid, ROUTE_WARPS * 32, 0, stream>>>(p);
      return cudaGetLastError();
    });
  };
  const cudaError_t err = c.score_fn == MOE_SCORE_SOFTMAX ? launch(std::true_type{}) : launch(std::false_type{});
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
