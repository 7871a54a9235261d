// The layer for a few tokens (moe_decode, moe_decode_routed in include/moe.h).
//
//   out_t = f_s(x_t) + sum over the slots of g f_e(x_t),   f(x) = W_down (SiLU(W_gate x) * W_up x)
//
// With T <= 64 tokens the layer is bound by the weights of the experts that have
// a token: each is read once, 6 D I bytes an expert in bf16, and there are only 2 n
// operations per weight for its n tokens.  So the kernel is a stream of weights
// that keeps every SM's TMA loads in flight from its first microsecond to its
// last, with whatever else has to be done placed beside it:
//
//   - One cooperative launch, one CTA per SM.  The tensor core multiplies tiles
//     of 128 weight rows (the M side) by the tokens of that expert (the N side, 16
//     to 64 columns): a step is 128 rows x 128 bytes (16 KB of weights) and its
//     tokens' 128 bytes each, eight to eleven steps in flight on an SM.
//   - The steps of a phase lie in one line (expert, tile, K) and every CTA takes an
//     equal stretch of it, so that SMs finish together whatever the number of
//     experts; a tile cut by a border leaves fp32 partial sums (a few KB beside
//     hundreds of KB of weights) that its CTAs add in CTA order, so results do not
//     depend on timing.
//   - Three phases: the shared expert's up/gate projections, which need no
//     routing and stream while the router works; the routed experts' up/gate
//     projections; all down projections, one output tile at a time over all its
//     experts, so that a token's weighted sum ends in one place.  Weights do not
//     depend on anything, so the loads of the next phase start while its inputs are
//     still being made.
//   - The router's products (T E D) run on the CUDA cores of all SMs first, with a bound
//     of its error beside every logit; where the k-th and the next logit are
//     closer than fp32 sums can tell apart, the undecided experts are decided in
//     fp64.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cstring>

#include "../../include/moe.h"
#include "common.cuh"
#include "plan.cuh"

namespace moe {

constexpr int DEC_MAX_T = 64;                       // tokens: bits of a 64-bit mask, columns of an accumulator
constexpr int DEC_MAX_R = DEC_MAX_T * TOPK_MAX;     // routes
constexpr int DEC_MAX_STAGES = 12;
constexpr int DEC_THREADS = 256;
constexpr int DEC_A_BYTES = 128 * 128;              // weights of a step
constexpr int DEC_MIN_STEPS = 4;                    // of a CTA's stretch: fewer and partial sums outweigh the steps
constexpr int DEC_SLOTS = 3;                        // partial sums of a CTA: its first, its last and a whole tile

struct DecodeParams {
  int T, D, I, E, k, I_s;
  int score_fn, given, mx;
  int ncap;       // columns of a step's tokens (T rounded up to 16)
  int n_stages, stage_bytes;
  long long timeout_ns;
  const bf16* x;
  const bf16* w_router;
  const float* b_router;
  const int* in_idx;    // given routing
  const float* in_w;
  bf16* out;
  int* out_idx;         // exports, or null
  float* out_w;
  int* status;
  int* counters;        // [3 gridDim + 2]
  float2* logits;       // [T, E] logit, what it may be off by
  int* topk_idx;        // [T, k]
  float* topk_w;
  uint8_t* xq;          // MXFP8: x as codes [T, D] and scales [T, D / 32]
  uint8_t* xs;
  void* h;              // [R, I] bf16, or codes
  uint8_t* hs;          // [R, I / 32]
  bf16* h_s;            // [64, I_s]
  float* slots;         // [gridDim][DEC_SLOTS][ncap][256]
  float* slots_s;       // the same for the shared expert's up/gate phase
  const uint8_t* sf_up;
  const uint8_t* sf_gate;
  const uint8_t* sf_down;
};

struct DecodeMaps {
  CUtensorMap x;       // [T, D] box {64, ncap}
  CUtensorMap x_rows;  // [T, D] bf16 box {64, 1}, or codes box {128, 1}
  CUtensorMap w_up, w_gate, w_down;     // box {64, 128} (codes {128, 128})
  CUtensorMap ws_up, ws_gate, ws_down;  // box {64, 128}
  CUtensorMap h;       // [R, I] box {64, 16} (codes {128, 16})
  CUtensorMap h_s;     // [64, I_s] box {64, 16}
};

// What every CTA knows of the routing, in shared memory
struct DecodeSched {
  unsigned long long mask[E_MAX];  // tokens of every expert
  float w[DEC_MAX_R];              // weight of every route
  uint16_t idx[DEC_MAX_R];         // expert of every route, 0xffff: none
  uint16_t row[DEC_MAX_R];         // route of every row (rows: by expert, then token)
  uint16_t off[E_MAX];             // first row of every expert
  uint16_t act_e[E_MAX];           // experts with a token
  int scan[4];
  int n_act;
};

constexpr int dec_smem_fixed() { return (int)sizeof(DecodeSched) + 1024 /* alignment */ + 512 /* barriers */; }

// One phase of the step line
struct Phase {
  int L;      // steps of a tile
  int total;  // steps of the phase
  int q;      // of a CTA's stretch
  __device__ __forceinline__ int owner(int step) const { return step / q; }
};
__device__ __forceinline__ Phase make_phase(int tiles, int L) {
  Phase f;
  f.L = L;
  f.total = tiles * L;
  f.q = max((f.total + (int)gridDim.x - 1) / (int)gridDim.x, DEC_MIN_STEPS);
  return f;
}

enum : int { PH_SHARED = 0, PH_UP = 1, PH_DOWN = 2 };

// A run of steps with one weight matrix and one set of tokens: one accumulator
struct Seg {
  int phase, tile;
  int part;    // PH_SHARED, PH_UP: 0 up rows, 1 gate rows; PH_DOWN: -1 the shared expert, else index of the active expert
  int act;     // index of the active expert (PH_UP, routed part of PH_DOWN)
  int k0, k1;  // steps of the part
  bool first, last;  // of the tile in this CTA
};

// The segments of this CTA in order.  Every role of the CTA walks them by itself.
struct Walk {
  int phase = -1, pos = 0, hi = 0, lo = 0;
  Phase f{1, 0, 1};
  __device__ __forceinline__ Phase phase_of(const DecodeParams& p, int ph, int n_act) const {
    const int kd = p.D / (p.mx ? BK_MX : BK);
    if (ph == PH_SHARED) return make_phase(p.I_s / 128, 2 * (p.D / BK));
    if (ph == PH_UP) return make_phase(n_act * (p.I / 128), 2 * kd);
    return make_phase(p.D / 128, p.I_s / BK + n_act * (p.I / (p.mx ? BK_MX : BK)));
  }
  __device__ __forceinline__ void enter(const DecodeParams& p, int ph, int n_act) {
    phase = ph;
    f = phase_of(p, ph, n_act);
    lo = min(f.total, (int)blockIdx.x * f.q);
    hi = min(f.total, lo + f.q);
    pos = lo;
  }
  __device__ __forceinline__ bool next(const DecodeParams& p, Seg& s) {
    if (pos >= hi) return false;
    s.phase = phase;
    s.tile = pos / f.L;
    int r = pos - s.tile * f.L, len;
    s.first = pos == lo || r == 0;
    if (phase != PH_DOWN) {
      const int half = f.L / 2;
      s.part = r >= half;
      s.act = phase == PH_UP ? s.tile / (p.I / 128) : -1;
      s.k0 = r - s.part * half;
      len = half - s.k0;
    } else {
      const int ks = p.I_s / BK, ki = p.I / (p.mx ? BK_MX : BK);
      if (r < ks) {
        s.part = s.act = -1;
        s.k0 = r;
        len = ks - r;
      } else {
        s.part = s.act = (r - ks) / ki;
        s.k0 = r - ks - s.act * ki;
        len = ki - s.k0;
      }
    }
    len = min(len, hi - pos);
    s.k1 = s.k0 + len;
    pos += len;
    s.last = pos == hi || pos == (s.tile + 1) * f.L;
    return true;
  }
};

__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// ------------------------------------------------------------------ router
// Logits of all tokens, four warps per expert and group of 8 tokens, each a
// quarter of D in chunks of 256 (8 elements a lane).  Beside a logit what fp32 may be off by:
// a product passes through at most `depth` additions, each of half an ulp (2^-24) of
// a sum that is at most the sum of magnitudes, and the bias through one.
__device__ __forceinline__ float dec_depth(int D) { return (float)((D / 256 + 3) / 4 * 8 + 8 + 4); }

__device__ __forceinline__ void unpack8(const uint4& q, float (&f)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(w[i] << 16), f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
}

__device__ void router_logits(const DecodeParams& p, float2* red /* [2][4][8] */) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, team = warp >> 2, quarter = warp & 3;
  const int groups = (p.T + 7) / 8, items = p.E * groups, chunks = p.D / 256;
  for (int first = blockIdx.x * 2; first < items; first += gridDim.x * 2) {
    const int item = first + team;
    const bool on = item < items;
    const int e = on ? item / groups : 0, t0 = on ? (item % groups) * 8 : 0;
    float acc[8], mag[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = mag[i] = 0.0f;
    if (on) {
      const uint4* w = reinterpret_cast<const uint4*>(p.w_router + (size_t)e * p.D) + lane;
      const uint4* x = reinterpret_cast<const uint4*>(p.x + (size_t)t0 * p.D) + lane;
      for (int c0 = quarter; c0 < chunks; c0 += 32) {
        uint4 wq[8];
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (c0 + 4 * c < chunks) wq[c] = __ldg(w + (c0 + 4 * c) * 32);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          if (c0 + 4 * c >= chunks) break;
          float wf[8];
          unpack8(wq[c], wf);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (t0 + i >= p.T) break;
            float xf[8];
            unpack8(__ldg(x + (size_t)i * (p.D / 8) + (c0 + 4 * c) * 32), xf);
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[i] = fmaf(xf[j], wf[j], acc[i]), mag[i] = fmaf(fabsf(xf[j]), fabsf(wf[j]), mag[i]);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (t0 + i >= p.T) break;
#pragma unroll
      for (int m = 16; m >= 1; m >>= 1) {
        acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], m);
        mag[i] += __shfl_xor_sync(0xffffffffu, mag[i], m);
      }
      if (lane == 0) red[(team * 4 + quarter) * 8 + i] = make_float2(acc[i], mag[i]);
    }
    named_bar_sync(1 + team, 128);
    if (quarter == 0 && lane < 8 && on && t0 + lane < p.T) {
      float2 s = red[team * 32 + lane];
#pragma unroll
      for (int q = 1; q < 4; ++q) s.x += red[(team * 4 + q) * 8 + lane].x, s.y += red[(team * 4 + q) * 8 + lane].y;
      s.y *= dec_depth(p.D) * (1.0f / 16777216.0f);
      if (p.b_router) {
        s.x += p.b_router[e];
        s.y += fabsf(s.x) * (1.0f / 16777216.0f);
      }
      if (!(s.x - s.x == 0.0f)) s.y = 0.0f;  // infinite or NaN: nothing to decide
      p.logits[(size_t)(t0 + lane) * p.E + e] = s;
    }
    named_bar_sync(1 + team, 128);
  }
}

__device__ __forceinline__ uint32_t dec_key(float f) {  // order of floats as unsigned integers, NaN lowest
  if (f != f) return 0u;
  f += 0.0f;  // -0 equals +0
  const uint32_t u = __float_as_uint(f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

// The undecided experts of a token (bit i of `und` in lane l: expert l + 32 i)
// ranked in fp64; the `want` first are added to `sel`.
__device__ __noinline__ uint32_t decide_fp64(const DecodeParams& p, int t, uint32_t und, uint32_t sel, int want) {
  const int lane = threadIdx.x & 31;
  double v[E_MAX / 32];
  for (int i = 0; i * 32 < p.E; ++i) {
    uint32_t who = __ballot_sync(0xffffffffu, und >> i & 1);
    while (who) {
      const int l = __ffs(who) - 1, e = l + 32 * i;
      who &= who - 1;
      double s = 0.0;
      const bf16 *x = p.x + (size_t)t * p.D, *w = p.w_router + (size_t)e * p.D;
      for (int d = lane; d < p.D; d += 32) s = fma((double)__bfloat162float(x[d]), (double)__bfloat162float(w[d]), s);
      for (int m = 16; m >= 1; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
      if (p.b_router) s += (double)p.b_router[e];
      if (lane == l) v[i] = s;
    }
  }
  for (int n = 0; n < want; ++n) {
    double best = 0.0;
    int id = 1 << 20;
    for (int i = 0; i * 32 < p.E; ++i)
      if ((und >> i & 1) && (id == 1 << 20 || v[i] > best)) best = v[i], id = lane + 32 * i;
    for (int m = 16; m >= 1; m >>= 1) {
      const double b = __shfl_xor_sync(0xffffffffu, best, m);
      const int j = __shfl_xor_sync(0xffffffffu, id, m);
      if (j != 1 << 20 && (id == 1 << 20 || b > best || (b == best && j < id))) best = b, id = j;
    }
    if (id != 1 << 20 && (id & 31) == lane) und &= ~(1u << (id >> 5)), sel |= 1u << (id >> 5);
  }
  return sel;
}

// Experts and weights of token t, one warp
__device__ void token_topk(const DecodeParams& p, int t) {
  const int lane = threadIdx.x & 31, k = p.k;
  float v[E_MAX / 32], err[E_MAX / 32];
  uint32_t left = 0u, key[E_MAX / 32];
  float most = 0.0f;
#pragma unroll
  for (int i = 0; i < E_MAX / 32; ++i) {
    const int e = lane + 32 * i;
    v[i] = err[i] = 0.0f, key[i] = 0u;
    if (e < p.E) {
      const float2 q = __ldcg(p.logits + (size_t)t * p.E + e);
      v[i] = q.x, err[i] = q.y, key[i] = dec_key(q.x);
      most = fmaxf(most, q.y);
      left |= 1u << i;
    }
  }
  uint32_t sel = 0u;
  for (int n = 0; n < k; ++n) {
    uint32_t b = 0u;
    int id = 1 << 20;
#pragma unroll
    for (int i = 0; i < E_MAX / 32; ++i)
      if ((left >> i & 1) && (id == 1 << 20 || key[i] > b)) b = key[i], id = lane + 32 * i;
    const uint32_t m = __reduce_max_sync(0xffffffffu, b);
    id = (int)__reduce_min_sync(0xffffffffu, b == m ? (unsigned)id : 1u << 20);
    if ((id & 31) == lane) left &= ~(1u << (id >> 5)), sel |= 1u << (id >> 5);
  }
  // lowest that a selected logit may be, highest that another may be
  float lo = INFINITY, hi = -INFINITY;
#pragma unroll
  for (int i = 0; i < E_MAX / 32; ++i) {
    if (sel >> i & 1) lo = fminf(lo, v[i] - err[i]);
    else if (left >> i & 1) hi = fmaxf(hi, v[i] + err[i]);
  }
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, d));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, d));
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
  }
  if (most > 0.0f && lo <= hi) {  // (exact logits that are equal are ties, decided above)
    uint32_t und = 0u;
    int want = 0;
#pragma unroll
    for (int i = 0; i < E_MAX / 32; ++i) {
      const bool in = sel >> i & 1;
      if (in ? v[i] - err[i] <= hi : (left >> i & 1) && v[i] + err[i] >= lo) und |= 1u << i, want += in;
    }
    want = (int)__reduce_add_sync(0xffffffffu, (unsigned)want);
    sel = decide_fp64(p, t, und, sel & ~und, want);
  }
  // the selected in ascending order: slot = number of selected experts below
  int slot = 0;
#pragma unroll
  for (int i = 0; i < E_MAX / 32; ++i) {
    if (32 * i >= p.E) break;
    const uint32_t row = __ballot_sync(0xffffffffu, sel >> i & 1);
    if (sel >> i & 1) {
      const int s = slot + __popc(row & ((1u << lane) - 1u));
      p.topk_idx[(size_t)t * k + s] = lane + 32 * i;
      p.topk_w[(size_t)t * k + s] = v[i];  // the logit, for now
      if (p.out_idx) p.out_idx[(size_t)t * k + s] = lane + 32 * i;
    }
    slot += __popc(row);
  }
  __syncwarp();
  // weights over their sum.  Softmax: exp(l - m); sigmoid: exp(min(l, 0)) / (1 + exp(-|l|)), both factors scaled so
  // that the largest is near 1 (logits far below 0 leave fp32's range otherwise)
  const float l = lane < k ? *(volatile float*)(p.topk_w + (size_t)t * k + lane) : -INFINITY;
  const bool soft = p.score_fn == MOE_SCORE_SOFTMAX;
  const float a = soft ? l : fminf(l, 0.0f);
  float m = a;
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  float s = lane < k ? expf(a - m) : 0.0f;
  if (!soft && lane < k) s /= 1.0f + expf(-fabsf(l));
  float sum = s;
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if (lane < k) {
    p.topk_w[(size_t)t * k + lane] = s / sum;
    if (p.out_w) p.out_w[(size_t)t * k + lane] = s / sum;
  }
}

// The routing into shared memory, by the 128 threads of the epilogue warps
__device__ void build_schedule(const DecodeParams& p, DecodeSched& s, int tid) {
  const int R = p.T * p.k;
  const int* idx = p.given ? p.in_idx : p.topk_idx;
  const float* wt = p.given ? p.in_w : p.topk_w;
  for (int e = tid; e < p.E; e += 128) s.mask[e] = 0ull;
  for (int r = tid; r < R; r += 128) {
    const int e = __ldcg(idx + r);
    const bool ok = e >= 0 && e < p.E;
    if (!ok && e != -1 && blockIdx.x == 0) atomicOr(p.status + 1, FLAG_ROUTES_INVALID);
    s.idx[r] = ok ? (uint16_t)e : (uint16_t)0xffffu;
    s.w[r] = __ldcg(wt + r);
  }
  named_bar_sync(3, 128);
  if (p.given) {  // a second slot of a token with the same expert is an empty one
    for (int r = tid; r < R; r += 128) {
      const int t = r / p.k;
      const uint16_t e = s.idx[r];
      bool twice = false;
      for (int q = t * p.k; q < r; ++q) twice |= e != 0xffffu && s.idx[q] == e;
      if (twice && blockIdx.x == 0) atomicOr(p.status + 1, FLAG_ROUTES_INVALID);
      if (!twice && e != 0xffffu) atomicOr(&s.mask[e], 1ull << t);
      s.row[r] = twice;  // (marked; the slots before it still have to be seen)
    }
    named_bar_sync(3, 128);
    for (int r = tid; r < R; r += 128)
      if (s.row[r]) s.idx[r] = 0xffffu;
  } else {
    for (int r = tid; r < R; r += 128) atomicOr(&s.mask[s.idx[r]], 1ull << (r / p.k));
  }
  named_bar_sync(3, 128);
  // rows and active experts before every expert: thread i takes experts 4 i .. 4 i + 3
  int rows = 0, act = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int e = 4 * tid + j;
    const int n = e < p.E ? __popcll(s.mask[e]) : 0;
    rows += n, act += n > 0;
  }
  const int lane = tid & 31, w = tid >> 5;
  int sum = rows | act << 16;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, sum, d);
    if (lane >= d) sum += o;
  }
  if (lane == 31) s.scan[w] = sum;
  named_bar_sync(3, 128);
  int before = sum - (rows | act << 16);
  for (int i = 0; i < w; ++i) before += s.scan[i];
  rows = before & 0xffff, act = before >> 16;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int e = 4 * tid + j;
    if (e < p.E) {
      const int n = __popcll(s.mask[e]);
      s.off[e] = (uint16_t)rows;
      if (n) s.act_e[act++] = (uint16_t)e;
      rows += n;
    }
  }
  if (tid == 127) s.n_act = act;
  named_bar_sync(3, 128);
  for (int r = tid; r < R; r += 128) {
    const uint16_t e = s.idx[r];
    if (e != 0xffffu) s.row[s.off[e] + __popcll(s.mask[e] & ((1ull << (r / p.k)) - 1ull))] = (uint16_t)r;
  }
}

// ------------------------------------------------------------------ sums of cut tiles
// A CTA's partial sums of a tile: slot 0 if it is its first of the phase, 1 if its last, else 2
__device__ __forceinline__ float* slot_of(const DecodeParams& p, float* slots, const Phase& f, int cta, int tile) {
  const int lo = cta * f.q, hi = min(f.total, lo + f.q);
  const int s = tile == lo / f.L ? 0 : tile == (hi - 1) / f.L ? 1 : 2;
  return slots + ((size_t)cta * DEC_SLOTS + s) * p.ncap * 256;
}

__device__ __forceinline__ float4 ldcg4(const float* p) { return __ldcg(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ void add4(float4& a, const float4& b) { a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w; }

// Up/gate tile: sums over its CTAs in order, SwiGLU, h.  This CTA takes every
// nc-th of the tile's n rows (nc CTAs share it), a warp a row, a lane 4 columns.
__device__ void finish_up(const DecodeParams& p, const Phase& f, int tile, float* slots, bool shared, int n, int row0, int ew) {
  const int lane = threadIdx.x & 31;
  const int b = tile * f.L, half = f.L / 2;
  const int c0 = f.owner(b), c1 = f.owner(b + half - 1), d0 = f.owner(b + half), d1 = f.owner(b + f.L - 1);
  const int nc = d1 - c0 + 1, me = (int)blockIdx.x - c0;
  const int width = shared ? p.I_s : p.I, col = (tile % (width / 128)) * 128 + 4 * lane;
  for (int r = me + nc * ew; r < n; r += nc * 4) {
    float4 u = make_float4(0.f, 0.f, 0.f, 0.f), g = u;
    for (int c = c0; c <= c1; ++c) add4(u, ldcg4(slot_of(p, slots, f, c, tile) + r * 256 + 4 * lane));
    for (int c = d0; c <= d1; ++c) add4(g, ldcg4(slot_of(p, slots, f, c, tile) + r * 256 + 128 + 4 * lane));
    const float h[4] = {silu_f32(g.x) * u.x, silu_f32(g.y) * u.y, silu_f32(g.z) * u.z, silu_f32(g.w) * u.w};
    if (shared || !p.mx) {
      bf16* to = shared ? p.h_s + (size_t)r * p.I_s + col : static_cast<bf16*>(p.h) + (size_t)(row0 + r) * p.I + col;
      *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3]));
    } else {  // MX blocks of 32 columns = 8 lanes
      float m = fmaxf(fmaxf(fabsf(h[0]), fabsf(h[1])), fmaxf(fabsf(h[2]), fabsf(h[3])));
#pragma unroll
      for (int d = 4; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
      uint32_t code = 0u, scale = 0u;
      if (m != 0.0f) {
        const uint32_t eb = (__float_as_uint(m) >> 23) & 0xFFu;
        int se = (eb != 0u ? (int)eb - 127 : ilogbf(m)) - 8;
        se = max(-127, min(127, se));
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = ldexpf(h[i], -se);
        const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(v[0], v[1]), __NV_SATFINITE, __NV_E4M3);
        const uint32_t c = __nv_cvt_float2_to_fp8x2(make_float2(v[2], v[3]), __NV_SATFINITE, __NV_E4M3);
        code = a | c << 16;
        scale = (uint32_t)(se + 127);
      }
      *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.h) + (size_t)(row0 + r) * p.I + col) = code;
      if ((lane & 7) == 0) p.hs[(size_t)(row0 + r) * (p.I / 32) + col / 32] = (uint8_t)scale;
    }
  }
}

// Output tile: sums over its CTAs in order, this CTA taking every nc-th token
__device__ void finish_down(const DecodeParams& p, const Phase& f, int tile, int ew) {
  const int lane = threadIdx.x & 31;
  const int c0 = f.owner(tile * f.L), c1 = f.owner((tile + 1) * f.L - 1), nc = c1 - c0 + 1, me = (int)blockIdx.x - c0;
  for (int t = me + nc * ew; t < p.T; t += nc * 4) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = c0; c <= c1; ++c) add4(s, ldcg4(slot_of(p, p.slots, f, c, tile) + t * 128 + 4 * lane));
    *reinterpret_cast<uint2*>(p.out + (size_t)t * p.D + tile * 128 + 4 * lane) =
        make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
  }
}

// ------------------------------------------------------------------ the kernel
template <bool MX>
__global__ void __launch_bounds__(DEC_THREADS, 1) moe_decode_kernel(const __grid_constant__ DecodeMaps maps,
                                                                   const __grid_constant__ DecodeParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int NST = p.n_stages;
  uint8_t* after = smem + NST * p.stage_bytes;
  uint8_t* sf = after;  // MXFP8: per stage the scale blocks of the weights and of the tokens
  if (MX) after += NST * 2 * SF_BLOCK_BYTES;
  DecodeSched& sched = *reinterpret_cast<DecodeSched*>(after);
  uint64_t* bars = reinterpret_cast<uint64_t*>(after + sizeof(DecodeSched));
  uint64_t *full = bars, *empty = bars + DEC_MAX_STAGES, *acc_full = bars + 2 * DEC_MAX_STAGES,
           *acc_empty = acc_full + 2, *ready = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ready + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int FULL_ARRIVALS = MX ? 3 : 2;  // weights, tokens (and the tokens' scales)

  if (threadIdx.x == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(&full[i], FULL_ARRIVALS);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 128);
    }
    mbar_init(ready, 128);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc<256>(tmem_slot);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // ---- before the grid's barrier: counters and status to zero, logits, x as codes
  if (blockIdx.x == 0 && threadIdx.x < 2) p.status[threadIdx.x] = 0;
  for (int i = blockIdx.x * DEC_THREADS + threadIdx.x; i < 3 * (int)gridDim.x + 2; i += gridDim.x * DEC_THREADS) p.counters[i] = 0;
  if (MX) {
    const int blocks = p.T * (p.D / 32);
    for (int b = blockIdx.x * DEC_THREADS + threadIdx.x; b < blocks; b += gridDim.x * DEC_THREADS) {
      float v[32];
      load_bf16x32(p.x + (size_t)b * 32, v);
      uint32_t c[8];
      p.xs[b] = (uint8_t)mx_quantize32(v, c);
      uint4* d = reinterpret_cast<uint4*>(p.xq + (size_t)b * 32);
      d[0] = make_uint4(c[0], c[1], c[2], c[3]);
      d[1] = make_uint4(c[4], c[5], c[6], c[7]);
    }
    fence_proxy_async_global();  // read by TMA
  }
  if (!p.given) router_logits(p, reinterpret_cast<float2*>(&sched));
  cooperative_groups::this_grid().sync();
  if (MX) fence_proxy_async_global();

  int* const topk_done = p.counters + 3 * gridDim.x;
  int* const h_done = topk_done + 1;
  // the epilogue's 128 threads go on together or not at all
  auto agree = [](bool v) {
    uint32_t all;
    asm volatile("{\n .reg .pred a, b;\n setp.ne.u32 a, %1, 0;\n barrier.cta.red.and.pred b, 3, 128, a;\n selp.u32 %0, 1, 0, b;\n}\n"
                 : "=r"(all) : "r"((uint32_t)v) : "memory");
    return all != 0;
  };
  auto wait_bar = [&](uint64_t* bar, uint32_t parity) { return mbar_wait(bar, parity, p.status, p.timeout_ns); };

  if (warp == 0) {
    // ---------------- weights
    if (elect_one()) {
      int stage = 0;
      uint32_t parity = 1;
      bool ok = true;
      Walk w;
      for (int ph = PH_SHARED; ph <= PH_DOWN && ok; ++ph) {
        if (ph == PH_UP && !wait_bar(ready, 0)) break;
        w.enter(p, ph, ph == PH_SHARED ? 0 : sched.n_act);
        Seg s;
        while (ok && w.next(p, s)) {
          const CUtensorMap* m;
          const uint8_t* scales = nullptr;
          int row;
          bool mx = MX;
          if (ph == PH_SHARED) {
            m = s.part ? &maps.ws_gate : &maps.ws_up, row = s.tile * 128, mx = false;
          } else if (ph == PH_UP) {
            m = s.part ? &maps.w_gate : &maps.w_up;
            row = sched.act_e[s.act] * p.I + (s.tile % (p.I / 128)) * 128;
            if (MX) scales = (s.part ? p.sf_gate : p.sf_up) + (size_t)(row / 128) * (p.D / BK_MX) * SF_BLOCK_BYTES;
          } else if (s.part < 0) {
            m = &maps.ws_down, row = s.tile * 128, mx = false;
          } else {
            m = &maps.w_down, row = sched.act_e[s.act] * p.D + s.tile * 128;
            if (MX) scales = p.sf_down + (size_t)(row / 128) * (p.I / BK_MX) * SF_BLOCK_BYTES;
          }
          for (int k = s.k0; k < s.k1; ++k) {
            if (!wait_bar(&empty[stage], parity)) { ok = false; break; }
            mbar_arrive_expect_tx(&full[stage], DEC_A_BYTES + (MX && mx ? SF_BLOCK_BYTES : 0));
            tma_load_2d(smem + stage * p.stage_bytes, m, &full[stage], k * (MX && mx ? BK_MX : BK), row);
            if (MX && mx) bulk_load(sf + stage * 2 * SF_BLOCK_BYTES, scales + (size_t)k * SF_BLOCK_BYTES, SF_BLOCK_BYTES, &full[stage]);
            if (++stage == NST) stage = 0, parity ^= 1u;
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    // ---------------- tokens: the rows of x or h of a segment's tokens
    int stage = 0;
    uint32_t parity = 1;
    bool ok = true;
    Walk w;
    for (int ph = PH_SHARED; ph <= PH_DOWN && ok; ++ph) {
      if (ph == PH_UP) ok = wait_bar(ready, 0);
      if (ph == PH_DOWN && ok) {
        int go = 1;
        if (lane == 0) go = wait_counter_ge(h_done, (int)gridDim.x, p.status, p.timeout_ns);
        ok = __shfl_sync(0xffffffffu, go, 0) != 0;
        __syncwarp();
        fence_proxy_async_global();
      }
      if (!ok) break;
      w.enter(p, ph, ph == PH_SHARED ? 0 : sched.n_act);
      Seg s;
      while (ok && w.next(p, s)) {
        const bool routed = s.act >= 0, mx = MX && routed;
        const int e = routed ? sched.act_e[s.act] : 0;
        const int n = routed ? __popcll(sched.mask[e]) : p.T, off = routed ? sched.off[e] : 0;
        // lane l: the l-th load of every step
        int t[4] = {0, 0, 0, 0}, loads;
        uint32_t bytes;
        if (ph == PH_SHARED) {
          loads = 1, bytes = (uint32_t)p.ncap * 128;
        } else if (ph == PH_UP) {
          loads = (n + 3) / 4, bytes = (uint32_t)loads * 512;
#pragma unroll
          for (int j = 0; j < 4; ++j) t[j] = sched.row[off + min(4 * lane + j, n - 1)] / p.k;
        } else {
          loads = (n + 15) / 16, bytes = (uint32_t)loads * 2048;
        }
        for (int k = s.k0; k < s.k1; ++k) {
          int go = 1;
          if (lane == 0) {
            go = wait_bar(&empty[stage], parity);
            if (go) mbar_arrive_expect_tx(&full[stage], bytes);
          }
          if (!__shfl_sync(0xffffffffu, go, 0)) { ok = false; break; }
          uint8_t* b = smem + stage * p.stage_bytes + DEC_A_BYTES;
          const int kc = k * (mx ? BK_MX : BK);
          if (lane < loads) {
            if (ph == PH_SHARED) tma_load_2d(b, &maps.x, &full[stage], kc, 0);
            else if (ph == PH_UP) tma_gather4(b + lane * 512, &maps.x_rows, &full[stage], kc, t[0], t[1], t[2], t[3]);
            else tma_load_2d(b + lane * 2048, routed ? &maps.h : &maps.h_s, &full[stage], kc, off + lane * 16);
          }
          __syncwarp();
          if (++stage == NST) stage = 0, parity ^= 1u;
        }
      }
    }
  } else if (warp == 3) {
    // ---------------- MXFP8: the scale block of a step's tokens, lane l rows l and l + 32
    if (MX) {
      int stage = 0;
      uint32_t parity = 1;
      bool ok = true;
      Walk w;
      for (int ph = PH_SHARED; ph <= PH_DOWN && ok; ++ph) {
        if (ph == PH_UP) ok = wait_bar(ready, 0);
        if (ph == PH_DOWN && ok) {
          int go = 1;
          if (lane == 0) go = wait_counter_ge(h_done, (int)gridDim.x, p.status, p.timeout_ns);
          ok = __shfl_sync(0xffffffffu, go, 0) != 0;
          __syncwarp();
        }
        if (!ok) break;
        w.enter(p, ph, ph == PH_SHARED ? 0 : sched.n_act);
        Seg s;
        while (ok && w.next(p, s)) {
          const bool routed = s.act >= 0;
          const uint32_t* src[2] = {nullptr, nullptr};
          if (routed) {
            const int e = sched.act_e[s.act], n = __popcll(sched.mask[e]), off = sched.off[e];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int r = lane + 32 * j;
              if (r < n)
                src[j] = reinterpret_cast<const uint32_t*>(ph == PH_UP ? p.xs + (size_t)(sched.row[off + r] / p.k) * (p.D / 32)
                                                                      : p.hs + (size_t)(off + r) * (p.I / 32));
            }
          }
          uint32_t ahead[4][2];  // four steps' words
#pragma unroll
          for (int d = 0; d < 4; ++d)
#pragma unroll
            for (int j = 0; j < 2; ++j) ahead[d][j] = src[j] && s.k0 + d < s.k1 ? __ldcg(src[j] + s.k0 + d) : 0u;
          for (int k = s.k0; k < s.k1; k += 4) {
#pragma unroll
            for (int d = 0; d < 4; ++d) {
              if (k + d >= s.k1 || !ok) break;
              int go = 1;
              if (lane == 0) go = wait_bar(&empty[stage], parity);
              if (!__shfl_sync(0xffffffffu, go, 0)) { ok = false; break; }
              uint8_t* to = sf + stage * 2 * SF_BLOCK_BYTES + SF_BLOCK_BYTES + lane * 16;
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                *reinterpret_cast<uint32_t*>(to + 4 * j) = ahead[d][j];
                ahead[d][j] = src[j] && k + d + 4 < s.k1 ? __ldcg(src[j] + k + d + 4) : 0u;
              }
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) mbar_arrive(&full[stage]);
              if (++stage == NST) stage = 0, parity ^= 1u;
            }
          }
        }
      }
    }
  } else if (warp == 1) {
    // ---------------- products
    if (elect_one()) {
      int stage = 0, acc = 0;
      uint32_t parity = 0, acc_parity = 1;
      bool ok = true;
      Walk w;
      for (int ph = PH_SHARED; ph <= PH_DOWN && ok; ++ph) {
        if (ph == PH_UP && !wait_bar(ready, 0)) break;
        w.enter(p, ph, ph == PH_SHARED ? 0 : sched.n_act);
        Seg s;
        while (ok && w.next(p, s)) {
          const bool routed = s.act >= 0, mx = MX && routed;
          const uint32_t n = routed ? (uint32_t)(__popcll(sched.mask[sched.act_e[s.act]]) + 15) & ~15u : (uint32_t)p.ncap;
          const uint32_t idesc = mx ? idesc_mxf8_e4m3(128, n) : idesc_bf16_f32(128, n);
          if (!wait_bar(&acc_empty[acc], acc_parity)) { ok = false; break; }
          tc_fence_after();
          const uint32_t d = tmem + acc * DEC_MAX_T, sfa = tmem + 2 * DEC_MAX_T, sfb = sfa + 4;
          for (int k = s.k0; k < s.k1; ++k) {
            if (!wait_bar(&full[stage], parity)) { ok = false; break; }
            tc_fence_after();
            const uint32_t a = smem_u32(smem + stage * p.stage_bytes), b = a + DEC_A_BYTES;
            if (mx) {
              const uint32_t f = smem_u32(sf + stage * 2 * SF_BLOCK_BYTES);
              tmem_cp_32x128b_warpx4(sfa, sdesc_sf_block(f));
              tmem_cp_32x128b_warpx4(sfb, sdesc_sf_block(f + SF_BLOCK_BYTES));
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_mxf8_ss(d, sdesc_kmajor_sw128(a + kk * 32), sdesc_kmajor_sw128(b + kk * 32),
                            idesc | ((uint32_t)kk << 4) | ((uint32_t)kk << 29), sfa, sfb, k != s.k0 || kk ? 1u : 0u);
            } else {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_bf16_ss(d, sdesc_kmajor_sw128(a + kk * 32), sdesc_kmajor_sw128(b + kk * 32), idesc, k != s.k0 || kk ? 1u : 0u);
            }
            mma_commit(&empty[stage]);
            if (++stage == NST) stage = 0, parity ^= 1u;
          }
          if (!ok) break;
          mma_commit(&acc_full[acc]);
          acc ^= 1;
          if (!acc) acc_parity ^= 1u;
        }
      }
    }
    __syncwarp();
  } else {
    // ---------------- routing, then the accumulators (TMEM lanes 32 ew .. 32 ew + 31)
    const int ew = warp - 4, tid = threadIdx.x - 128, col = tid;
    bool ok = true;
    if (!p.given) {
      for (int t = blockIdx.x + ew * gridDim.x; t < p.T; t += 4 * gridDim.x) {
        token_topk(p, t);
        __syncwarp();
        if (lane == 0) red_release_add_gpu(topk_done, 1);
      }
      ok = agree(wait_counter_ge(topk_done, p.T, p.status, p.timeout_ns));
    }
    if (ok) build_schedule(p, sched, tid);
    if (ok) mbar_arrive(ready);
    const int n_act = ok ? sched.n_act : 0;
    named_bar_sync(3, 128);

    int acc = 0;
    uint32_t acc_parity = 0;
    Walk w;
    for (int ph = PH_SHARED; ph <= PH_DOWN && ok; ++ph) {
      w.enter(p, ph, ph == PH_SHARED ? 0 : n_act);
      const Phase f = w.f;
      float* slots = ph == PH_SHARED ? p.slots_s : p.slots;
      int* ctr = p.counters + ph * gridDim.x;
      Seg s;
      while (w.next(p, s)) {
        const bool routed = s.act >= 0;
        const int e = routed ? sched.act_e[s.act] : 0;
        const int n = routed ? __popcll(sched.mask[e]) : p.T, off = routed ? sched.off[e] : 0;
        float* slot = slot_of(p, slots, f, blockIdx.x, s.tile);
        if (ph == PH_DOWN && s.first)
          for (int t = 0; t < p.T; ++t) slot[t * 128 + col] = 0.0f;
        ok = agree(wait_bar(&acc_full[acc], acc_parity));
        if (!ok) break;
        tc_fence_after();
        const uint32_t taddr = tmem + acc * DEC_MAX_T + ((uint32_t)(32 * ew) << 16);
        for (int n0 = 0; n0 < n; n0 += 16) {
          uint32_t v[16];
          tmem_ld_32x32b_x16(taddr + n0, v);
          tmem_ld_wait();
          if (ph != PH_DOWN) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (n0 + j < n) slot[(n0 + j) * 256 + s.part * 128 + col] = __uint_as_float(v[j]);
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (n0 + j < n) {
                const int r = routed ? sched.row[off + n0 + j] : 0;
                const int t = routed ? r / p.k : n0 + j;
                const float g = routed ? sched.w[r] : 1.0f;
                slot[t * 128 + col] = fmaf(g, __uint_as_float(v[j]), slot[t * 128 + col]);
              }
          }
        }
        tc_fence_before();
        mbar_arrive(&acc_empty[acc]);
        acc ^= 1;
        if (!acc) acc_parity ^= 1u;
        if (s.last) {
          const int b = s.tile * f.L, c0 = f.owner(b), c1 = f.owner(b + f.L - 1);
          named_bar_sync(3, 128);
          if (c0 != c1) {  // cut: counted under its first CTA
            if (tid == 0) red_release_add_gpu(ctr + c0, 1);
          } else if (ph == PH_DOWN) {
            finish_down(p, f, s.tile, ew);
            named_bar_sync(3, 128);
          } else {
            finish_up(p, f, s.tile, slots, ph == PH_SHARED, n, off, ew);
            named_bar_sync(3, 128);
          }
        }
      }
      if (!ok) break;
      if (ph == PH_SHARED) continue;
      // the cut tiles that this CTA has a part of, of this phase (after the up/gate phase: of the shared expert's too)
      for (int q = ph == PH_UP ? PH_SHARED : PH_DOWN; q <= ph && ok; ++q) {
        Walk v;
        v.enter(p, q, q == PH_SHARED ? 0 : n_act);
        if (v.lo >= v.hi) continue;
        const int t0 = v.lo / v.f.L, t1 = (v.hi - 1) / v.f.L;
        for (int i = 0; i < (t0 == t1 ? 1 : 2) && ok; ++i) {
          const int tile = i ? t1 : t0;
          const int c0 = v.f.owner(tile * v.f.L), c1 = v.f.owner((tile + 1) * v.f.L - 1);
          if (c0 == c1) continue;
          int* const flag = p.counters + q * gridDim.x + c0;
          ok = agree(wait_counter_ge(flag, c1 - c0 + 1, p.status, p.timeout_ns));
          if (!ok) break;
          if (q == PH_DOWN) {
            finish_down(p, v.f, tile, ew);
          } else {
            const int e = q == PH_UP ? sched.act_e[tile / (p.I / 128)] : 0;
            finish_up(p, v.f, tile, q == PH_SHARED ? p.slots_s : p.slots, q == PH_SHARED,
                      q == PH_UP ? __popcll(sched.mask[e]) : p.T, q == PH_UP ? sched.off[e] : 0, ew);
          }
        }
      }
      if (ph == PH_UP) {  // h is read by TMA of every CTA; slots are used again only after all have read them
        fence_proxy_async_global();
        named_bar_sync(3, 128);
        if (tid == 0 && ok) red_release_add_gpu(h_done, 1);
        ok = agree(ok && wait_counter_ge(h_done, (int)gridDim.x, p.status, p.timeout_ns));
      } else if (w.f.total == 0) {  // no expert and no shared expert: zeros
        for (int tile = blockIdx.x; tile < p.D / 128; tile += gridDim.x)
          for (int t = ew; t < p.T; t += 4)
            *reinterpret_cast<uint2*>(p.out + (size_t)t * p.D + tile * 128 + 4 * lane) = make_uint2(0u, 0u);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  settle_after_abort(p.status);
  if (warp == 1) tmem_dealloc(tmem, 256);
}

}  // namespace moe

// ------------------------------------------------------------------ C ABI
using namespace moe;

namespace {

constexpr size_t dec_align(size_t v) { return (v + 255) / 256 * 256; }

struct DecodeLayout {
  size_t status, counters, logits, topk_idx, topk_w, xq, xs, h, hs, h_s, slots, slots_s, total;
};
DecodeLayout decode_layout(const moe_plan* pl, int64_t T) {
  const moe_config& c = pl->cfg;
  const bool mx = c.precision == MOE_PREC_MXFP8;
  const int64_t R = T * c.k, ncap = (T + 15) / 16 * 16;
  DecodeLayout L{};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at = dec_align(at + bytes);
    return here;
  };
  L.status = take(STATUS_AREA_BYTES);
  L.counters = take(sizeof(int) * (3 * pl->num_sms + 2));
  L.logits = take(sizeof(float2) * T * c.E);
  L.topk_idx = take(sizeof(int) * R);
  L.topk_w = take(sizeof(float) * R);
  L.xq = take(mx ? T * c.D : 0);
  L.xs = take(mx ? T * (c.D / 32) : 0);
  L.h = take((size_t)R * c.I * (mx ? 1 : 2));
  L.hs = take(mx ? R * (c.I / 32) : 0);
  L.h_s = take((size_t)DEC_MAX_T * c.I_s * 2);
  L.slots = take(sizeof(float) * 256 * ncap * DEC_SLOTS * pl->num_sms);
  L.slots_s = take(c.I_s ? sizeof(float) * 256 * ncap * DEC_SLOTS * pl->num_sms : 0);
  L.total = at;
  return L;
}

// rows of 128 bytes: 64 bf16 or 128 codes
int decode_map(const moe_plan* pl, CUtensorMap* m, const void* ptr, uint64_t rows, uint64_t cols, uint32_t box_rows, bool codes) {
  const cuuint64_t dims[2] = {cols, rows}, strides[1] = {cols * (codes ? 1 : 2)};
  const cuuint32_t box[2] = {codes ? 128u : 64u, box_rows}, one[2] = {1, 1};
  return pl->encode(m, codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims,
                    strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? MOE_OK
             : MOE_ERR_INVALID_ARG;
}
bool dec_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int decode(const moe_plan* pl, int64_t T, const void* x, const moe_weights* w, const int32_t* in_idx, const float* in_w,
           void* out, int32_t* topk_idx, float* topk_w, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  const moe_config& c = pl->cfg;
  const bool given = in_idx != nullptr, mx = c.precision == MOE_PREC_MXFP8;
  if (!x || !w->W_up || !w->W_gate || !w->W_down || !out || !workspace || (!given && !w->W_router)) return MOE_ERR_INVALID_ARG;
  const bool shared = w->Ws_up || w->Ws_gate || w->Ws_down;
  if (shared && (!w->Ws_up || !w->Ws_gate || !w->Ws_down || c.I_s == 0)) return MOE_ERR_INVALID_ARG;
  if (mx && (!w->W_up_scale || !w->W_gate_scale || !w->W_down_scale)) return MOE_ERR_INVALID_ARG;
  for (const void* q : {x, given ? x : w->W_router, w->W_up, w->W_gate, w->W_down, (const void*)out, w->Ws_up, w->Ws_gate, w->Ws_down,
                        mx ? (const void*)w->W_up_scale : nullptr, mx ? (const void*)w->W_gate_scale : nullptr,
                        mx ? (const void*)w->W_down_scale : nullptr})
    if (!dec_aligned(q, 16)) return MOE_ERR_INVALID_ARG;
  if (!dec_aligned(workspace, 256) || !dec_aligned(topk_idx, 4) || !dec_aligned(topk_w, 4) || !dec_aligned(given ? nullptr : w->b_router, 4))
    return MOE_ERR_INVALID_ARG;
  const DecodeLayout L = decode_layout(pl, T);
  if (workspace_bytes < L.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  int cur = -1;
  if (cudaGetDevice(&cur) != cudaSuccess || cur != pl->device) return MOE_ERR_INVALID_ARG;

  uint8_t* ws = static_cast<uint8_t*>(workspace);
  DecodeParams p{};
  p.T = (int)T, p.D = (int)c.D, p.I = (int)c.I, p.E = (int)c.E, p.k = (int)c.k, p.I_s = shared ? (int)c.I_s : 0;
  p.score_fn = c.score_fn;
  p.given = given;
  p.mx = mx;
  p.ncap = (int)((T + 15) / 16 * 16);
  p.stage_bytes = DEC_A_BYTES + p.ncap * 128;
  const int room = 227 * 1024 - dec_smem_fixed(), per = p.stage_bytes + (mx ? 2 * SF_BLOCK_BYTES : 0);
  p.n_stages = room / per < DEC_MAX_STAGES ? room / per : DEC_MAX_STAGES;
  const int smem = dec_smem_fixed() + p.n_stages * per;
  p.timeout_ns = (long long)c.timeout_ms * 1000000LL;
  p.x = static_cast<const bf16*>(x);
  p.w_router = static_cast<const bf16*>(w->W_router);
  p.b_router = w->b_router;
  p.in_idx = in_idx, p.in_w = in_w;
  p.out = static_cast<bf16*>(out);
  p.out_idx = topk_idx, p.out_w = topk_w;
  p.status = reinterpret_cast<int*>(ws + L.status);
  p.counters = reinterpret_cast<int*>(ws + L.counters);
  p.logits = reinterpret_cast<float2*>(ws + L.logits);
  p.topk_idx = reinterpret_cast<int*>(ws + L.topk_idx);
  p.topk_w = reinterpret_cast<float*>(ws + L.topk_w);
  p.xq = ws + L.xq, p.xs = ws + L.xs;
  p.h = ws + L.h, p.hs = ws + L.hs;
  p.h_s = reinterpret_cast<bf16*>(ws + L.h_s);
  p.slots = reinterpret_cast<float*>(ws + L.slots), p.slots_s = reinterpret_cast<float*>(ws + L.slots_s);
  p.sf_up = w->W_up_scale, p.sf_gate = w->W_gate_scale, p.sf_down = w->W_down_scale;

  DecodeMaps m;
  std::memset(&m, 0, sizeof(m));
  int rc = decode_map(pl, &m.x_rows, mx ? (const void*)p.xq : x, T, c.D, 1, mx);
  rc |= decode_map(pl, &m.w_up, w->W_up, c.E * c.I, c.D, 128, mx);
  rc |= decode_map(pl, &m.w_gate, w->W_gate, c.E * c.I, c.D, 128, mx);
  rc |= decode_map(pl, &m.w_down, w->W_down, c.E * c.D, c.I, 128, mx);
  rc |= decode_map(pl, &m.h, p.h, T * c.k, c.I, 16, mx);
  if (shared) {
    rc |= decode_map(pl, &m.x, x, T, c.D, (uint32_t)p.ncap, false);
    rc |= decode_map(pl, &m.ws_up, w->Ws_up, c.I_s, c.D, 128, false);
    rc |= decode_map(pl, &m.ws_gate, w->Ws_gate, c.I_s, c.D, 128, false);
    rc |= decode_map(pl, &m.ws_down, w->Ws_down, c.D, c.I_s, 128, false);
    rc |= decode_map(pl, &m.h_s, p.h_s, DEC_MAX_T, c.I_s, 16, false);
  }
  if (rc != MOE_OK) return MOE_ERR_INVALID_ARG;

  auto kernel = mx ? moe_decode_kernel<true> : moe_decode_kernel<false>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return MOE_ERR_CUDA;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)pl->num_sms);
  lc.blockDim = dim3(DEC_THREADS);
  lc.dynamicSmemBytes = (size_t)smem;
  lc.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeCooperative;  // all CTAs at once: they wait on one another
  at[0].val.cooperative = 1;
  lc.attrs = at;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, kernel, m, p) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t moe_decode_workspace_bytes(const moe_plan* plan, int64_t T) {
  if (!plan || T < 0 || T > plan->cfg.T_max || T > MOE_DECODE_MAX_TOKENS) return 0;
  return T == 0 ? 256 : decode_layout(plan, T).total;
}

int moe_decode(const moe_plan* pl, int64_t T, const void* x, const moe_weights* w, void* out, int32_t* topk_idx,
               float* topk_w, void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  if (!pl || !w || T < 0 || T > pl->cfg.T_max || T > MOE_DECODE_MAX_TOKENS) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  return decode(pl, T, x, w, nullptr, nullptr, out, topk_idx, topk_w, workspace, workspace_bytes, (cudaStream_t)stream);
}

int moe_decode_routed(const moe_plan* pl, int64_t T, const void* x, const moe_weights* w, const int32_t* topk_idx,
                      const float* topk_w, void* out, void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  if (!pl || !w || T < 0 || T > pl->cfg.T_max || T > MOE_DECODE_MAX_TOKENS) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!topk_idx || !topk_w || !dec_aligned(topk_idx, 4) || !dec_aligned(topk_w, 4)) return MOE_ERR_INVALID_ARG;
  return decode(pl, T, x, w, topk_idx, topk_w, out, nullptr, nullptr, workspace, workspace_bytes, (cudaStream_t)stream);
}

}  // extern "C"
