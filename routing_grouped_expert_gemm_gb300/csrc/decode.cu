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
//   - Work is cut into units: some steps of one weight tile for one expert, a few
//     hundred KB. SMs are not equally fast at reading memory, so units are claimed
//     from a counter, in order. A unit leaves its fp32 sums (512 bytes a token beside
//     those hundreds of KB) in a place of its own; when all of a phase are there every
//     CTA adds its share of them in a fixed order, so results do not depend on timing.
//     (With the deep queue of loads that fills the memory system a round trip to L2
//     takes microseconds: units must not wait for one, a phase may.)
//   - Three phases: the shared expert's up/gate projections, which need no
//     routing and stream while the router works (dealt out, not claimed); the routed
//     experts' up/gate projections; all down projections, one output tile at a time
//     over its experts. Weights do not depend on anything, so the loads of the next
//     phase start while its inputs are still being made.
//   - The router's products (T E D) run on the CUDA cores of all SMs first, with a bound
//     of its error beside every logit; where the k-th and the next logit are
//     closer than fp32 sums can tell apart, the undecided experts are decided in
//     fp64.
//
// D = 7168, I = 2048, 256 experts, k = 8, one shared: one token 137 us (117.6 at the copy
// rate: 18 us until the routing is known, of which the shared expert's weights hide some,
// 4 us each between the phases and at the end), 64 tokens 2.82 to 2.91 ms (all of the copy
// rate); 8 tokens of MXFP8 experts 432 us (92%).  Evicting weights from L2 first: 158 -> 150 us
// for one token, nothing for more.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cstddef>
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
enum : int { CTR_TOPK = 0, CTR_CLAIMS, CTR_UP /* units done */, CTR_H /* CTAs whose share of h is written */, CTR_DOWN, DEC_COUNTERS };
constexpr int DEC_OWN_TOPK = 4;                     // up to so many tokens every CTA makes all tokens' selection itself
constexpr int DEC_EARLY = 2;                        // steps loaded before the grid's barrier
constexpr int DEC_QUEUE = 4;                        // claimed units on their way to the roles of a CTA
constexpr int DEC_SMEM = 227 * 1024;                // shared memory of a CTA: as many stages as fit

// Steps that a unit should have, for `total` steps on `ctas` CTAs: a CTA's share in 32 units,
// though not so many that a unit is below 12 steps (4.5 us of an SM's loads), or where
// the share is small, 8 units of at least 4; and sums (ncap columns) below an eighth of its
// weights.  A projection is cut into equal units near that, so one may have down to half as
// many, and no unit has more than its tile's projection (4 steps of 256 columns: sums of 64
// tokens are then half of its weights).
__host__ __device__ inline int dec_unit_steps(int total, int ctas, int ncap) {
  const int share = (total + ctas - 1) / ctas;
  int q = share / 8;
  q = q < 4 ? 4 : q > 12 ? 12 : q;
  if (q < share / 32) q = share / 32;
  if (q < ncap / 4) q = ncap / 4;
  return q;
}

struct DecodeParams {
  int T, D, I, E, k, I_s;
  int score_fn, given, mx;
  int inv_k;      // ceil(2^16 / k)
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
  int* counters;        // [DEC_COUNTERS]
  float2* logits;       // [T, E] logit, what it may be off by
  int* topk_idx;        // [T, k]
  float* topk_w;
  uint8_t* xq;          // MXFP8: x as codes [T, D] and scales [T, D / 32]
  uint8_t* xs;
  void* h;              // [R, I] bf16, or codes
  uint8_t* hs;          // [R, I / 32]
  bf16* h_s;            // [64, I_s]
  float* sums_s;        // sums of the shared up/gate units: [tile][part][piece][T][128]
  float* sums_u;        // of the routed ones: [tile][part][piece][T k rows][128]
  float* sums_d;        // of the down units: [tile][piece][T k rows][128]
  float* sums_ds;       // of the shared expert's: [tile][piece][T][128]
  int q_s, q_ds;        // steps of a unit of the shared expert's up/gate and (where it has no others) down projections
  int most_u, most_d;   // pieces that there is room for
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
  // the units of the claimed phases
  int m_u, q_u;         // pieces of a routed up/gate part, steps of a piece
  int m_d, q_d, m_ds;   // pieces of a down projection, steps of a piece, pieces of the shared expert's
  int n_u, n_d;         // units of the two phases
  int n_rows;           // rows: routes that are not empty
};

enum : int { PH_SHARED = 0, PH_UP = 1, PH_DOWN = 2 };

// A unit as the role that loads weights hands it to the others
struct Unit {
  int phase;   // PH_*, or -1: no more
  int routed;  // 0: the shared expert
  int k0, k1;  // steps
  int n, off;  // its tokens and their first row
  int m, row;  // weights: tensor map (order of DecodeMaps) and first row
  float* sums; // where its sums go: [n][128]
  const uint8_t* scales;  // MXFP8: the weights' scale blocks of these rows
};
enum : int { M_X = 0, M_X_ROWS, M_UP, M_GATE, M_DOWN, M_S_UP, M_S_GATE, M_S_DOWN, M_H, M_H_S };

__device__ __forceinline__ int shared_pieces(const DecodeParams& p) { return (p.D / BK + p.q_s - 1) / p.q_s; }
__device__ __forceinline__ int shared_units(const DecodeParams& p) { return p.I_s / 128 * 2 * shared_pieces(p); }
// Unit i of the shared expert's up/gate phase
__device__ __forceinline__ void shared_unit(const DecodeParams& p, int i, Unit& u) {
  const int m = shared_pieces(p), piece = i % m, tp = i / m;  // tp: tile and part
  u.phase = PH_SHARED;
  u.routed = 0;
  u.n = p.T, u.off = 0;
  u.m = tp & 1 ? M_S_GATE : M_S_UP;
  u.row = (tp >> 1) * 128;
  u.k0 = piece * p.q_s;
  u.k1 = min(p.D / BK, u.k0 + p.q_s);
  u.sums = p.sums_s + (size_t)i * p.T * 128;
  u.scales = nullptr;
}
// Claimed unit i
__device__ __noinline__ void claimed_unit(const DecodeParams& p, const DecodeSched& s, int i, Unit& u) {
  const size_t R = (size_t)p.T * p.k;
  int act = -1, kd;
  if (i < s.n_u) {  // (active expert, tile, part, piece)
    u.phase = PH_UP;
    const int piece = i % s.m_u, tp = i / s.m_u % (p.I / 64), tile = tp >> 1;
    act = i / s.m_u / (p.I / 64);
    kd = p.D;
    u.k0 = piece * s.q_u, u.k1 = u.k0 + s.q_u;
    u.m = tp & 1 ? M_GATE : M_UP;
    u.row = s.act_e[act] * p.I + tile * 128;
    u.scales = tp & 1 ? p.sf_gate : p.sf_up;
    u.sums = p.sums_u + (size_t)(tp * s.m_u + piece) * R * 128;
  } else {  // (output tile, shared expert's pieces, (active expert, piece))
    i -= s.n_u;
    u.phase = PH_DOWN;
    const int per = s.m_ds + s.n_act * s.m_d, tile = i / per;
    i -= tile * per;
    int piece = i;
    if (i < s.m_ds) {
      kd = p.I_s;
      u.m = M_S_DOWN, u.row = tile * 128;
      u.sums = p.sums_ds + (size_t)(tile * s.m_ds + piece) * p.T * 128;
    } else {
      i -= s.m_ds;
      act = i / s.m_d, piece = i % s.m_d;
      kd = p.I;
      u.m = M_DOWN, u.row = s.act_e[act] * p.D + tile * 128;
      u.sums = p.sums_d + (size_t)(tile * s.m_d + piece) * R * 128;
    }
    u.scales = p.sf_down;
    u.k0 = piece * s.q_d, u.k1 = u.k0 + s.q_d;
  }
  u.routed = act >= 0;
  const int step = p.mx && u.routed ? BK_MX : BK;
  u.k1 = min(u.k1, kd / step);
  if (u.routed) {
    const int e = s.act_e[act];
    u.n = __popcll(s.mask[e]);
    u.off = s.off[e];
    u.sums += (size_t)u.off * 128;
    u.scales = p.mx ? u.scales + (size_t)(u.row / 128) * (kd / BK_MX) * SF_BLOCK_BYTES : nullptr;
  } else {
    u.n = p.T, u.off = 0;
    u.scales = nullptr;
  }
}

// Everything of a CTA in shared memory but the stages
struct DecodeShared {
  DecodeSched sched;
  DecodeParams p;  // (here its fields cost 30 cycles, not a miss of the constant cache each)
  Unit queue[DEC_QUEUE];
  uint64_t full[DEC_MAX_STAGES], empty[DEC_MAX_STAGES], acc_full[2], acc_empty[2], ready, q_full[DEC_QUEUE], q_empty[DEC_QUEUE];
  uint32_t tmem;
};
constexpr int dec_smem_fixed() { return (int)sizeof(DecodeShared) + 1024 /* alignment */; }

// Bounded waits (as in common.cuh), out of line: a launch runs most of this kernel's
// code once, and what it costs then is fetching it
__device__ __noinline__ bool dec_wait_slow(uint64_t* bar, uint32_t parity, const DecodeParams& p) {
  return mbar_wait(bar, parity, p.status, p.timeout_ns);
}
__device__ __forceinline__ bool dec_wait(uint64_t* bar, uint32_t parity, const DecodeParams& p) {
  return mbar_try_wait(bar, parity) || dec_wait_slow(bar, parity, p);
}
__device__ __noinline__ bool dec_wait_count(int ctr, int need, const DecodeParams& p) {
  return wait_counter_ge(p.counters + ctr, need, p.status, p.timeout_ns);
}
// the epilogue's 128 threads go on together or not at all
__device__ __forceinline__ bool agree(bool v) {
  uint32_t all;
  asm volatile("{\n .reg .pred a, b;\n setp.ne.u32 a, %1, 0;\n barrier.cta.red.and.pred b, 3, 128, a;\n selp.u32 %0, 1, 0, b;\n}\n"
               : "=r"(all) : "r"((uint32_t)v) : "memory");
  return all != 0;
}

__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// ------------------------------------------------------------------ router
// Logits of all tokens: a team of four warps takes four experts (so that x comes from
// L2 once for them; one where that leaves teams without work) and 4 tokens, each warp a quarter of D in chunks
// of 256 (8 elements a lane).  Beside a logit what fp32 may be off by: a product
// passes through at most `depth` additions, each of half an ulp (2^-24) of a sum that
// is at most the sum of magnitudes, which is at most |x| |w|; and the bias through one.
// (1 + 2^-8 covers the norms' own roundings.)  Below 2^-126 a rounding loses up to 2^-150
// whatever the value: squares of elements below 2^-75 come to nothing, so a lane whose
// elements are not all zeros adds 2^-149 for every one of them to the squares, which does
// nothing to those of ordinary size; and a logit may lose as much with every product.
constexpr int RT_E = 4, RT_T = 4, RT_N = RT_E * RT_T + RT_E + RT_T;
__device__ __forceinline__ float dec_depth(int D) { return (float)((D / 256 + 3) / 4 + 8 + 10 + 4); }

__device__ __forceinline__ void unpack8(const uint4& q, float (&f)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(w[i] << 16), f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
}

__device__ __forceinline__ uint32_t any_bits(const uint4& q) { return (q.x | q.y) | (q.z | q.w); }

__device__ __noinline__ void router_logits(const DecodeParams& p, float* part /* [8 warps][RT_N][33] */, float* red /* [8][RT_N] */) {
  constexpr int NV = RT_N, AHEAD = 3;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, team = warp >> 2, quarter = warp & 3;
  const int groups = (p.T + RT_T - 1) / RT_T, chunks = p.D / 256;
  const int per = p.E * groups <= 4 * (int)gridDim.x ? 1 : RT_E, items = (p.E + per - 1) / per * groups;
  const uint4 none = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
  for (int first = blockIdx.x; first < items; first += 2 * gridDim.x) {
    const int item = first + (1 - team) * (int)gridDim.x;  // (a thread of team 0 starts the loads first)
    const bool on = item < items;
    const int e0 = on ? item / groups * per : 0, t0 = on ? item % groups * RT_T : 0;
    const int ne = min(per, p.E - e0), nt = min(RT_T, p.T - t0);
    float v[NV];  // logits, then |w|^2, then |x|^2
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = 0.0f;
    uint32_t bits[RT_E + RT_T];  // of this lane's elements of w and x: whether one of them is not zero
#pragma unroll
    for (int i = 0; i < RT_E + RT_T; ++i) bits[i] = 0u;
    const uint4* w = reinterpret_cast<const uint4*>(p.w_router + (size_t)e0 * p.D) + lane;
    const uint4* x = reinterpret_cast<const uint4*>(p.x + (size_t)t0 * p.D) + lane;
    const int d8 = p.D / 8;
    uint4 wq[AHEAD][RT_E], xq[RT_T];  // weights three chunks ahead, tokens one
    auto get = [&](int c, uint4 (&q)[RT_E]) {
#pragma unroll
      for (int e = 0; e < RT_E; ++e) q[e] = on && c < chunks && e < ne ? __ldg(w + (size_t)e * d8 + c * 32) : none;
    };
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) get(quarter + 4 * a, wq[a]);
#pragma unroll
    for (int t = 0; t < RT_T; ++t) xq[t] = on && quarter < chunks && t < nt ? __ldg(x + (size_t)t * d8 + quarter * 32) : none;
#pragma unroll 1
    for (int c = quarter; on && c < chunks; c += 4) {
      float wf[RT_E][8];
#pragma unroll
      for (int e = 0; e < RT_E; ++e) {
        unpack8(wq[0][e], wf[e]);
        bits[e] |= any_bits(wq[0][e]);
#pragma unroll
        for (int a = 0; a + 1 < AHEAD; ++a) wq[a][e] = wq[a + 1][e];
      }
      get(c + 4 * AHEAD, wq[AHEAD - 1]);
#pragma unroll
      for (int e = 0; e < RT_E; ++e)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[RT_E * RT_T + e] = fmaf(wf[e][j], wf[e][j], v[RT_E * RT_T + e]);
#pragma unroll
      for (int t = 0; t < RT_T; ++t) {
        if (t >= nt) break;
        float xf[8], of[RT_E];  // (a chunk's sum by itself: fewer additions behind one another)
        unpack8(xq[t], xf);
        bits[RT_E + t] |= any_bits(xq[t]);
        if (c + 4 < chunks) xq[t] = __ldg(x + (size_t)t * d8 + (c + 4) * 32);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[RT_E * RT_T + RT_E + t] = fmaf(xf[j], xf[j], v[RT_E * RT_T + RT_E + t]);
#pragma unroll
          for (int e = 0; e < RT_E; ++e) of[e] = j ? fmaf(xf[j], wf[e][j], of[e]) : xf[0] * wf[e][0];
        }
#pragma unroll
        for (int e = 0; e < RT_E; ++e) v[t * RT_E + e] += of[e];
      }
    }
#pragma unroll
    for (int i = 0; i < RT_E + RT_T; ++i)
      if (bits[i] & 0x7fff7fffu) v[RT_E * RT_T + i] += __int_as_float(8 * ((chunks + 3) / 4));  // 2^-149 each
    // the lanes' sums through shared memory: lane l adds those of value l
    float* mine = part + warp * (NV * 33);
#pragma unroll
    for (int i = 0; i < NV; ++i) mine[i * 33 + lane] = v[i];
    __syncwarp();
    if (lane < NV) {
      float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
      for (int l = 0; l < 32; l += 4)
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] += mine[lane * 33 + l + i];
      red[warp * NV + lane] = (sum[0] + sum[1]) + (sum[2] + sum[3]);
    }
    __syncwarp();
    named_bar_sync(1 + team, 128);
    if (quarter == 0 && on && lane < RT_E * RT_T && lane / RT_E < nt && lane % RT_E < ne) {  // lane: a token and an expert
      const int t = lane / RT_E, e = lane % RT_E;
      const float* r = red + team * 4 * NV;
      float2 s = make_float2(0.0f, 0.0f);
      float ww = 0.0f, xx = 0.0f;
#pragma unroll
      for (int q = 0; q < 4; ++q) s.x += r[q * NV + lane], ww += r[q * NV + RT_E * RT_T + e], xx += r[q * NV + RT_E * RT_T + RT_E + t];
      s.y = 0.0f;  // (of zeros)
      if (ww > 0.0f && xx > 0.0f) s.y = sqrtf(ww) * sqrtf(xx) * dec_depth(p.D) * (257.0f / 256.0f / 16777216.0f) + __int_as_float(p.D);
      if (p.b_router) {
        s.x += p.b_router[e0 + e];
        s.y += fabsf(s.x) * (1.0f / 16777216.0f);
      }
      if (!(s.x - s.x == 0.0f)) s.y = 0.0f;  // infinite or NaN: nothing to decide
      p.logits[(size_t)(t0 + t) * p.E + e0 + e] = s;
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

struct TopkScratch {
  uint32_t key[E_MAX];
  uint32_t words[E_MAX / 32], open[E_MAX / 32];  // a bit an expert
  float range[3][4];
  float logit[TOPK_MAX];
  int idx[DEC_OWN_TOPK * TOPK_MAX];
  float w[DEC_OWN_TOPK * TOPK_MAX];
};
static_assert(offsetof(DecodeSched, scan) - offsetof(DecodeSched, row) >= E_MAX * sizeof(float2), "the logits lie where rows and experts come to lie");
static_assert(sizeof(DecodeSched::w) >= E_MAX * 8, "keys in fp64 lie where the weights come to lie");
static_assert(DEC_OWN_TOPK * TOPK_MAX <= 128, "a thread a route");
static_assert(sizeof(TopkScratch) <= sizeof(DecodeSched::mask), "scratch of the selection lies where the masks come to lie");

// What a selected logit may be off by, besides its own rounding to fp32, before fp64
// sums take its place for the weight's sake.  The bound holds for any order of signs; sums
// whose parts cancel from 10^5 to 1 are off by a 220th of it at most (2^14 of them), so
// 2^-6 means weights within 10^-4.  Unit tokens and router rows have bounds of 10^-4.  At
// 2^-9 rows of 16 times that length pay for it already (one token of 256 experts 136 -> 196 us).
constexpr float DEC_LOGIT_TOL = 1.0f / 64.0f;
__device__ __forceinline__ bool too_far_off(float2 q) { return fmaf(fabsf(q.x), -1.0f / 16777216.0f, q.y) > DEC_LOGIT_TOL; }

// The selection of token t where fp32 left it open, by the epilogue's 128 threads:
// the experts that may be in or out, given what every logit may be off by, are ranked
// by their logits in fp64 (as integers of the same order, NaN lowest), which take the
// place of the fp32 ones; and so do those of experts that are in, but too far off.
__device__ __noinline__ void decide_fp64(const DecodeParams& p, int t, int tid, float lo, float hi, TopkScratch& s, float2* val,
                                         unsigned long long* dkey /* [E], shared memory */) {
  const int lane = tid & 31, ew = tid >> 5, words = (p.E + 31) / 32;
#pragma unroll 1
  for (int e = tid; e < ((p.E + 127) & ~127); e += 128) {
    const bool in = s.words[e >> 5] >> lane & 1;
    const float2 q = val[e];
    const bool open = e < p.E && (in ? q.x - q.y <= hi || too_far_off(q) : q.x + q.y >= lo);
    const uint32_t o = __ballot_sync(0xffffffffu, open), w = __ballot_sync(0xffffffffu, in && !open);
    if (lane == 0) s.open[e >> 5] = o, s.words[e >> 5] = w;
  }
  named_bar_sync(3, 128);
  int n = 0, want = p.k;
#pragma unroll 1
  for (int w = 0; w < words; ++w) {
    want -= __popc(s.words[w]);
    uint32_t who = s.open[w];
#pragma unroll 1
    for (; who; who &= who - 1, ++n) {  // a warp every fourth
      if ((n & 3) != ew) continue;
      const int e = 32 * w + __ffs(who) - 1;
      const bf16 *x = p.x + (size_t)t * p.D + 8 * lane, *v = p.w_router + (size_t)e * p.D + 8 * lane;
      double sum = 0.0;
#pragma unroll 2
      for (int d = 0; d < p.D; d += 256) {
        float a[8], b[8];
        unpack8(__ldg(reinterpret_cast<const uint4*>(x + d)), a);
        unpack8(__ldg(reinterpret_cast<const uint4*>(v + d)), b);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = fma((double)a[j], (double)b[j], sum);
      }
#pragma unroll 1
      for (int m = 16; m >= 1; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
      if (p.b_router) sum += (double)p.b_router[e];
      const long long bits = __double_as_longlong(sum + 0.0);
      if (lane == 0) {
        dkey[e] = sum != sum ? 0ull : (unsigned long long)(bits ^ (bits >> 63 | (long long)0x8000000000000000ull));
        val[e].x = (float)sum;
      }
    }
  }
  named_bar_sync(3, 128);
#pragma unroll 1
  for (int e = tid; e < ((p.E + 127) & ~127); e += 128) {
    bool in = s.words[e >> 5] >> lane & 1;
    if (s.open[e >> 5] >> lane & 1) {
      const unsigned long long key = dkey[e];
      int rank = 0;
#pragma unroll 1
      for (int w = 0; w < words; ++w)
#pragma unroll 1
        for (uint32_t who = s.open[w]; who; who &= who - 1) {
          const int f = 32 * w + __ffs(who) - 1;
          rank += dkey[f] > key || (dkey[f] == key && f < e);
        }
      in = rank < want;
    }
    const uint32_t w = __ballot_sync(0xffffffffu, in);
    if (lane == 0) s.words[e >> 5] = w;  // (this warp alone reads this word here)
  }
  named_bar_sync(3, 128);
}

// Experts and weights of token t, by the epilogue's 128 threads (thread i has
// experts i + 128 j): an expert's rank is the number of keys before its own, counted
// in a short loop over all of them (selecting the largest k times over took 15 us of a
// call at 256 experts).  Loops stay rolled: every line of code is a miss.
__device__ __noinline__ void token_topk(const DecodeParams& p, int t, int tid, TopkScratch& s, float2* val /* [E], shared memory */,
                                       unsigned long long* dkey, int* idx, float* wt) {
  const int lane = tid & 31, ew = tid >> 5, k = p.k;
  const float2* from = p.logits + (size_t)t * p.E;
#pragma unroll 1
  for (int e = tid; e < ((p.E + 127) & ~127); e += 128) {
    const float2 q = e < p.E ? __ldcg(from + e) : make_float2(0.0f, 0.0f);
    val[e] = q;
    s.key[e] = e < p.E ? dec_key(q.x) : 0u;
  }
  named_bar_sync(3, 128);
  // the rank of an expert among all: four keys a look, two experts at once
  // lowest that a selected logit may be, highest that another may be
  float lo = INFINITY, hi = -INFINITY, most = 0.0f;  // (most: the error, infinite where a selected one is too far off)
#pragma unroll 1
  for (int e = tid; e < ((p.E + 127) & ~127); e += 256) {
    const int e2 = e + 128;
    const bool two = e2 < ((p.E + 127) & ~127);
    const uint32_t key = s.key[e], key2 = two ? s.key[e2] : 0u;
    int rank = 0, rank2 = 0;
#pragma unroll 2
    for (int j = 0; j < p.E; j += 4) {  // (keys past the last expert are 0 and behind it in every tie)
      const uint4 o = *reinterpret_cast<const uint4*>(s.key + j);
      const int d = e - j, d2 = e2 - j;  // ties: the lower id is before
      rank += (o.x >= key + (d <= 0)) + (o.y >= key + (d <= 1)) + (o.z >= key + (d <= 2)) + (o.w >= key + (d <= 3));
      rank2 += (o.x >= key2 + (d2 <= 0)) + (o.y >= key2 + (d2 <= 1)) + (o.z >= key2 + (d2 <= 2)) + (o.w >= key2 + (d2 <= 3));
    }
#pragma unroll 1
    for (int i = 0; i < (two ? 2 : 1); ++i) {
      const int at = i ? e2 : e;
      const float2 q = val[at];
      const bool in = at < p.E && (i ? rank2 : rank) < k;
      if (in) lo = fminf(lo, q.x - q.y);
      else if (at < p.E) hi = fmaxf(hi, q.x + q.y);
      most = fmaxf(most, in && too_far_off(q) ? INFINITY : q.y);
      const uint32_t w = __ballot_sync(0xffffffffu, in);
      if (lane == 0) s.words[at >> 5] = w;
    }
  }
#pragma unroll 1
  for (int d = 16; d >= 1; d >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, d));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, d));
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
  }
  if (lane == 0) s.range[0][ew] = lo, s.range[1][ew] = hi, s.range[2][ew] = most;
  named_bar_sync(3, 128);
#pragma unroll 1
  for (int w = 0; w < 4; ++w) lo = fminf(lo, s.range[0][w]), hi = fmaxf(hi, s.range[1][w]), most = fmaxf(most, s.range[2][w]);
  if (most > 0.0f && (lo <= hi || most == INFINITY)) {  // (exact logits that are equal are ties, decided above)
    decide_fp64(p, t, tid, lo, hi, s, val, dkey);
  }
  // slots in ascending order: the selected experts below
#pragma unroll 1
  for (int e = tid; e < p.E; e += 128) {
    if (!(s.words[e >> 5] >> lane & 1)) continue;
    int slot = __popc(s.words[e >> 5] & ((1u << lane) - 1u));
#pragma unroll 1
    for (int w = 0; w < e >> 5; ++w) slot += __popc(s.words[w]);
    s.logit[slot] = val[e].x;
    idx[slot] = e;
    if (p.out_idx && (int)blockIdx.x == t % (int)gridDim.x) p.out_idx[(size_t)t * k + slot] = e;
  }
  named_bar_sync(3, 128);
  // weights over their sum.  Softmax: exp(l - m); sigmoid: exp(min(l, 0)) / (1 + exp(-|l|)), both factors scaled so
  // that the largest is near 1 (logits far below 0 leave fp32's range otherwise)
  if (ew == 0) {
    const float l = lane < k ? s.logit[lane] : -INFINITY;
    const bool soft = p.score_fn == MOE_SCORE_SOFTMAX;
    const float a = soft ? l : fminf(l, 0.0f);
    float m = a;
#pragma unroll 1
    for (int d = 16; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    float w = lane < k ? expf(a - m) : 0.0f;
    if (!soft && lane < k) w /= 1.0f + expf(-fabsf(l));
    float sum = w;
#pragma unroll 1
    for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane < k) {
      wt[lane] = w / sum;
      if (p.out_w && (int)blockIdx.x == t % (int)gridDim.x) p.out_w[(size_t)t * k + lane] = w / sum;
    }
  }
}

// r / k for a route r, by a reciprocal: r (k ceil(2^16 / k) - 2^16) < 2^16 for r < 1024
__device__ __forceinline__ int token_of(const DecodeParams& p, int r) { return (int)((unsigned)r * (unsigned)p.inv_k >> 16); }

// The routing into shared memory, by the 128 threads of the epilogue warps
__device__ __noinline__ void build_schedule(const DecodeParams& p, DecodeSched& s, int tid) {
  const int R = p.T * p.k;
#pragma unroll 1
  for (int e = tid; e < p.E; e += 128) s.mask[e] = 0ull;
  if (p.given || p.T > DEC_OWN_TOPK) {
    const int* idx = p.given ? p.in_idx : p.topk_idx;
    const float* wt = p.given ? p.in_w : p.topk_w;
#pragma unroll 1
    for (int r = tid; r < R; r += 128) {
      const int e = __ldcg(idx + r);
      s.w[r] = __ldcg(wt + r);
      const bool ok = e >= 0 && e < p.E;
      if (!ok && e != -1 && blockIdx.x == 0) atomicOr(p.status + 1, FLAG_ROUTES_INVALID);
      s.idx[r] = ok ? (uint16_t)e : (uint16_t)0xffffu;
    }
  }
  named_bar_sync(3, 128);
  if (p.given) {  // a second slot of a token with the same expert is an empty one
#pragma unroll 1
    for (int r = tid; r < R; r += 128) {
      const int t = token_of(p, r);
      const uint16_t e = s.idx[r];
      bool twice = false;
#pragma unroll 1
      for (int q = t * p.k; q < r; ++q) twice |= e != 0xffffu && s.idx[q] == e;
      if (twice && blockIdx.x == 0) atomicOr(p.status + 1, FLAG_ROUTES_INVALID);
      if (!twice && e != 0xffffu) atomicOr(&s.mask[e], 1ull << t);
      s.row[r] = twice;  // (marked; the slots before it still have to be seen)
    }
    named_bar_sync(3, 128);
#pragma unroll 1
    for (int r = tid; r < R; r += 128)
      if (s.row[r]) s.idx[r] = 0xffffu;
  } else {
#pragma unroll 1
    for (int r = tid; r < R; r += 128) atomicOr(&s.mask[s.idx[r]], 1ull << token_of(p, r));
  }
  named_bar_sync(3, 128);
  // rows and active experts before every expert: thread i takes experts 4 i .. 4 i + 3
  int rows = 0, act = 0;
#pragma unroll 1
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
#pragma unroll 1
  for (int j = 0; j < 4; ++j) {
    const int e = 4 * tid + j;
    if (e < p.E) {
      const int n = __popcll(s.mask[e]);
      s.off[e] = (uint16_t)rows;
      if (n) s.act_e[act++] = (uint16_t)e;
      rows += n;
    }
  }
  if (tid == 127) {
    s.n_act = act;
    s.n_rows = rows;
    const int kd = p.D / (p.mx ? BK_MX : BK), ki = p.I / (p.mx ? BK_MX : BK), ks = p.I_s / BK;
    const int q = dec_unit_steps(act * (p.I / 128) * 2 * kd, gridDim.x, p.ncap);
    s.m_u = min(max((kd + q - 1) / q, 1), p.most_u);
    s.q_u = (kd + s.m_u - 1) / s.m_u;
    s.m_u = (kd + s.q_u - 1) / s.q_u;
    s.n_u = act * (p.I / 128) * 2 * s.m_u;
    const int r = dec_unit_steps(p.D / 128 * (ks + act * ki), gridDim.x, p.ncap);
    s.m_d = min(max((ki + r - 1) / r, 1), p.most_d);
    s.q_d = max((ki + s.m_d - 1) / s.m_d, p.q_ds);
    s.m_d = (ki + s.q_d - 1) / s.q_d;
    s.m_ds = (ks + s.q_d - 1) / s.q_d;
    s.n_d = p.D / 128 * (s.m_ds + act * s.m_d);
  }
  named_bar_sync(3, 128);
#pragma unroll 1
  for (int r = tid; r < R; r += 128) {
    const uint16_t e = s.idx[r];
    if (e != 0xffffu) s.row[s.off[e] + __popcll(s.mask[e] & ((1ull << token_of(p, r)) - 1ull))] = (uint16_t)r;
  }
}

// ------------------------------------------------------------------ finished tiles
__device__ __forceinline__ float4 ldcg4(const float* p) { return __ldcg(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ void add4(float4& a, const float4& b) { a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w; }
__device__ __forceinline__ void fma4(float4& a, float g, const float4& b) {
  a.x = fmaf(g, b.x, a.x), a.y = fmaf(g, b.y, a.y), a.z = fmaf(g, b.z, a.z), a.w = fmaf(g, b.w, a.w);
}

// The sums that follow are a few rows of 512 bytes out of L2 an output, and what they
// cost is the trips there, each with up to four rows on its way.  A warp takes 128
// columns, a lane 4; or, where that makes fewer trips (few items, many rows each), 32
// columns: 8 lanes a row of 128 bytes, each quarter of the warp every fourth row, and
// the quarters are added in the end (one token's last sums 10 -> 3 us; 64 tokens' h the
// other way round, 13 -> 48).
struct Split {
  int quarter, of, lane, blocks;  // this lane's quarter, quarters, lane in it, items' columns
  __device__ __forceinline__ Split(int items /* of 128 columns */, int rows) {
    const int l = threadIdx.x & 31, warps = 4 * gridDim.x;
    const bool split = (4 * items + warps - 1) / warps * ((rows + 15) / 16) < (items + warps - 1) / warps * ((rows + 3) / 4);
    quarter = split ? l >> 3 : 0, of = split ? 4 : 1, lane = split ? l & 7 : l, blocks = split ? 32 : 128;
  }
};
__device__ __forceinline__ float4 quarters(float4 a) {
#pragma unroll
  for (int d = 8; d <= 16; d <<= 1) {
    a.x += __shfl_xor_sync(0xffffffffu, a.x, d), a.y += __shfl_xor_sync(0xffffffffu, a.y, d);
    a.z += __shfl_xor_sync(0xffffffffu, a.z, d), a.w += __shfl_xor_sync(0xffffffffu, a.w, d);
  }
  return a;
}

// h of all rows, this CTA's share: an item is a row (token) and 32 or 128 columns: the
// sums of its pieces, SwiGLU.
__device__ __noinline__ void finish_up(const DecodeParams& p, const DecodeSched& sc, int ew) {
  const Split sp(p.T * (p.I_s / 128) + sc.n_rows * (p.I / 128), max(shared_pieces(p), sc.m_u));
  const int blocks_s = p.I_s / sp.blocks, blocks_u = p.I / sp.blocks, of_s = p.T * blocks_s, items = of_s + sc.n_rows * blocks_u;
#pragma unroll 1
  for (int it = blockIdx.x + ew * gridDim.x; it < items; it += 4 * gridDim.x) {
    const bool shared = it < of_s;
    const int blocks = shared ? blocks_s : blocks_u, r = (shared ? it : it - of_s) / blocks, block = (shared ? it : it - of_s) % blocks;
    const int m = shared ? shared_pieces(p) : sc.m_u, col = block * sp.blocks + 4 * sp.lane, tile = col >> 7;
    const size_t rows = shared ? p.T : (size_t)p.T * p.k;
    const float* su = (shared ? p.sums_s : p.sums_u) + ((size_t)tile * 2 * m * rows + r) * 128 + (col & 127);
    const float* sg = su + (size_t)m * rows * 128;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), g = a;
#pragma unroll 1
    for (int c0 = sp.quarter; c0 < m; c0 += 4 * sp.of) {
      float4 q[2][4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const bool in = c0 + sp.of * c < m;
        q[0][c] = in ? ldcg4(su + (c0 + sp.of * c) * rows * 128) : make_float4(0.f, 0.f, 0.f, 0.f);
        q[1][c] = in ? ldcg4(sg + (c0 + sp.of * c) * rows * 128) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) add4(a, q[0][c]), add4(g, q[1][c]);
    }
    if (sp.of > 1) a = quarters(a), g = quarters(g);
    const float h[4] = {silu_f32(g.x) * a.x, silu_f32(g.y) * a.y, silu_f32(g.z) * a.z, silu_f32(g.w) * a.w};
    if (shared || !p.mx) {
      bf16* to = shared ? p.h_s + (size_t)r * p.I_s + col : static_cast<bf16*>(p.h) + (size_t)r * p.I + col;
      if (sp.quarter == 0) *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3]));
    } else {  // an MX block is 8 lanes
      float most = fmaxf(fmaxf(fabsf(h[0]), fabsf(h[1])), fmaxf(fabsf(h[2]), fabsf(h[3])));
#pragma unroll
      for (int d = 4; d >= 1; d >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
      uint32_t code = 0u, scale = 0u;
      if (most != 0.0f) {
        const uint32_t eb = (__float_as_uint(most) >> 23) & 0xFFu;
        int se = (eb != 0u ? (int)eb - 127 : ilogbf(most)) - 8;
        se = max(-127, min(127, se));
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = ldexpf(h[i], -se);
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[0], v[1]), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[2], v[3]), __NV_SATFINITE, __NV_E4M3);
        code = lo | hi << 16;
        scale = (uint32_t)(se + 127);
      }
      if (sp.quarter == 0) *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.h) + (size_t)r * p.I + col) = code;
      if (sp.quarter == 0 && (sp.lane & 7) == 0) p.hs[(size_t)r * (p.I / 32) + col / 32] = (uint8_t)scale;
    }
  }
}

// The output, this CTA's share: an item is a token and 32 or 128 columns; its terms are the
// pieces of the shared expert's output and of its slots' outputs, these times the slot's weight.
__device__ __noinline__ void finish_down(const DecodeParams& p, const DecodeSched& sc, int ew) {
  const int terms = sc.m_ds + p.k * sc.m_d;
  const Split sp(p.T * (p.D / 128), terms);
  const int blocks = p.D / sp.blocks;
  const size_t R = (size_t)p.T * p.k;
#pragma unroll 1
  for (int it = blockIdx.x + ew * gridDim.x; it < p.T * blocks; it += 4 * gridDim.x) {
    const int t = it / blocks, at = it % blocks * sp.blocks + 4 * sp.lane, tile = at >> 7, col = at & 127;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int i0 = sp.quarter; i0 < terms; i0 += 4 * sp.of) {
      float4 q[4];
      float w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int term = i0 + sp.of * i;
        const float* from = nullptr;
        w[i] = 1.0f;
        if (term < sc.m_ds) {
          from = p.sums_ds + ((size_t)(tile * sc.m_ds + term) * p.T + t) * 128;
        } else if (term < terms) {
          const int j = (term - sc.m_ds) / sc.m_d, c = term - sc.m_ds - j * sc.m_d, r = t * p.k + j, e = sc.idx[r];
          if (e != 0xffff) {
            from = p.sums_d + ((size_t)(tile * sc.m_d + c) * R + sc.off[e] + __popcll(sc.mask[e] & ((1ull << t) - 1ull))) * 128;
            w[i] = sc.w[r];
          }
        }
        q[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (from) q[i] = ldcg4(from + col);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) fma4(s, w[i], q[i]);
    }
    if (sp.of > 1) s = quarters(s);
    if (sp.quarter == 0)
      *reinterpret_cast<uint2*>(p.out + (size_t)t * p.D + at) =
          make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
  }
}

// ------------------------------------------------------------------ the kernel
static_assert(3 * (DEC_A_BYTES + DEC_MAX_T * 128) >= 8 * RT_N * 33 * 4, "the router's sums fit into the stages without early loads");
template <bool MX>
__global__ void __launch_bounds__(DEC_THREADS, 1) moe_decode_kernel(const __grid_constant__ DecodeMaps maps,
                                                                   const __grid_constant__ DecodeParams params) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int NST = params.n_stages, stage_bytes = params.stage_bytes;
  uint8_t* sf = smem + NST * stage_bytes;  // MXFP8: per stage the scale blocks of the weights and of the tokens
  DecodeShared& sh = *reinterpret_cast<DecodeShared*>(sf + (MX ? NST * 2 * SF_BLOCK_BYTES : 0));
  DecodeSched& sched = sh.sched;
  const DecodeParams& p = sh.p;
  const CUtensorMap* const map = &maps.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int FULL_ARRIVALS = MX ? 3 : 2;  // weights, tokens (and the tokens' scales)

  // ---- before the grid's barrier
  if (threadIdx.x < sizeof(DecodeParams) / 4)
    reinterpret_cast<uint32_t*>(&sh.p)[threadIdx.x] = reinterpret_cast<const uint32_t*>(&params)[threadIdx.x];
  if (threadIdx.x >= 128 && threadIdx.x < 128 + (int)(sizeof(DecodeMaps) / sizeof(CUtensorMap))) prefetch_tensormap(map + (threadIdx.x - 128));
  if (threadIdx.x == 0) {
#pragma unroll 1
    for (int i = 0; i < NST; ++i) {
      mbar_init(&sh.full[i], FULL_ARRIVALS);
      mbar_init(&sh.empty[i], 1);
    }
#pragma unroll 1
    for (int i = 0; i < DEC_QUEUE; ++i) {
      mbar_init(&sh.q_full[i], 1);
      mbar_init(&sh.q_empty[i], 128 + (MX ? 3 : 2));  // epilogue, tokens, (scales,) products
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.acc_full[i], 1);
      mbar_init(&sh.acc_empty[i], 128);
    }
    mbar_init(&sh.ready, 128);
    fence_barrier_init();
  }
  __syncthreads();
  // Loads of one step: 128 rows of weights; the rows of x or h of the unit's tokens.  Weights are read once: they are
  // the first to leave L2, and do not push out what is used again (tokens, sums, the kernel's own code)
  const uint64_t once = l2_policy_evict_first();
  auto load_weights = [&](const Unit& u, int k, int stage) {
    const bool mx = MX && u.routed;
    mbar_arrive_expect_tx(&sh.full[stage], DEC_A_BYTES + (mx ? SF_BLOCK_BYTES : 0));
    tma_load_2d_hint(smem + stage * stage_bytes, map + u.m, &sh.full[stage], k * (mx ? BK_MX : BK), u.row, once);
    if (mx) bulk_load(sf + stage * 2 * SF_BLOCK_BYTES, u.scales + (size_t)k * SF_BLOCK_BYTES, SF_BLOCK_BYTES, &sh.full[stage]);
  };
  auto load_x = [&](int k, int stage) {
    mbar_arrive_expect_tx(&sh.full[stage], (uint32_t)p.ncap * 128);
    tma_load_2d(smem + stage * stage_bytes + DEC_A_BYTES, map + M_X, &sh.full[stage], k * BK, 0);
  };
  // The first loads of the shared expert's weights, which wait for nothing, by one thread while the others are at the
  // router's weights; counters and status to zero, logits, x as codes
  const int n_shared = shared_units(p);
  if (threadIdx.x == 0) {
    int stage = 0;
#pragma unroll 1
    for (int i = blockIdx.x; i < n_shared && stage < DEC_EARLY; i += gridDim.x) {
      Unit u;
      shared_unit(p, i, u);
#pragma unroll 1
      for (int k = u.k0; k < u.k1 && stage < DEC_EARLY; ++k, ++stage) {
        load_weights(u, k, stage);
        load_x(k, stage);
      }
    }
  }
  if (blockIdx.x == 0 && threadIdx.x < 2) p.status[threadIdx.x] = 0;
  if (blockIdx.x == 0 && threadIdx.x < DEC_COUNTERS) p.counters[threadIdx.x] = 0;
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
  if (warp == 1) {
    tmem_alloc<256>(&sh.tmem);
    tmem_relinquish();
  }
  __syncwarp();
  if (!p.given) {  // (its sums in stages that have no loads yet)
    router_logits(p, reinterpret_cast<float*>(smem + DEC_EARLY * stage_bytes), reinterpret_cast<float*>(&sched));
    fence_proxy_async_smem();
  }
  tc_fence_before();
  cooperative_groups::this_grid().sync();  // (of this CTA's threads too)
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  if (MX) fence_proxy_async_global();

  // position in the ring of stages, and in the queue of units
  int stage = 0, at = 0;
  uint32_t parity = 0;
  auto advance = [&]() {
    if (++stage == NST) stage = 0, parity ^= 1u;
  };
  auto q_slot = [&]() { return at % DEC_QUEUE; };
  auto q_parity = [&]() { return (uint32_t)(at / DEC_QUEUE) & 1u; };

  if (warp == 0) {
    // ---------------- units and their weights: the shared expert's up/gate units by number, then claimed ones
    if (elect_one()) {
      bool ok = true;
      int mine = blockIdx.x, next = 0, early = 0, units = 0;
      bool claiming = false;
#pragma unroll 1
      for (; ok; ++at) {
        const bool shared = mine < n_shared;
        if (!shared && !claiming) {
          if (!dec_wait(&sh.ready, 0, p)) break;
          claiming = true;
          units = sched.n_u + sched.n_d;
          next = atomicAdd(p.counters + CTR_CLAIMS, 1);
        }
        if (!dec_wait(&sh.q_empty[q_slot()], q_parity() ^ 1u, p)) break;
        Unit& u = sh.queue[q_slot()];
        if (shared) {
          shared_unit(p, mine, u);
          mine += gridDim.x;
        } else if (next < units) {
          const int id = next;
          next = atomicAdd(p.counters + CTR_CLAIMS, 1);  // (the answer is not needed before this unit's loads are issued)
          claimed_unit(p, sched, id, u);
        } else {
          u.phase = -1;
        }
        mbar_arrive(&sh.q_full[q_slot()]);
        if (u.phase < 0) break;
        const Unit v = u;
#pragma unroll 1
        for (int k = v.k0; k < v.k1; ++k, advance()) {
          if (shared && early < DEC_EARLY) { ++early; continue; }
          if (!(ok = dec_wait(&sh.empty[stage], parity ^ 1u, p))) break;
          load_weights(v, k, stage);
        }
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    // ---------------- tokens
    bool ok = true, have_h = false;
    int early = 0;
#pragma unroll 1
    for (; ok; ++at) {
      int go = 1;
      if (lane == 0) go = dec_wait(&sh.q_full[q_slot()], q_parity(), p);
      if (!__shfl_sync(0xffffffffu, go, 0)) break;
      __syncwarp();
      const Unit u = sh.queue[q_slot()];
      // lane l: the l-th load of every step
      int t[4] = {0, 0, 0, 0}, loads = 1;
      uint32_t bytes = (uint32_t)p.ncap * 128;
      if (u.phase == PH_UP) {
        loads = (u.n + 3) / 4, bytes = (uint32_t)loads * 512;
#pragma unroll
        for (int j = 0; j < 4; ++j) t[j] = token_of(p, sched.row[u.off + min(4 * lane + j, u.n - 1)]);
      } else if (u.phase == PH_DOWN) {
        loads = (u.n + 15) / 16, bytes = (uint32_t)loads * 2048;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_empty[q_slot()]);
      if (u.phase < 0) break;
      if (u.phase == PH_DOWN && !have_h) {
        if (lane == 0) go = dec_wait_count(CTR_H, (int)gridDim.x, p);
        if (!__shfl_sync(0xffffffffu, go, 0)) break;
        __syncwarp();
        fence_proxy_async_global();
        have_h = true;
      }
      const bool mx = MX && u.routed;
#pragma unroll 1
      for (int k = u.k0; k < u.k1; ++k, advance()) {
        if (u.phase == PH_SHARED && early < DEC_EARLY) { ++early; continue; }
        if (lane == 0) {
          go = dec_wait(&sh.empty[stage], parity ^ 1u, p);
          if (go) mbar_arrive_expect_tx(&sh.full[stage], bytes);
        }
        if (!(ok = __shfl_sync(0xffffffffu, go, 0) != 0)) break;
        uint8_t* b = smem + stage * stage_bytes + DEC_A_BYTES;
        const int kc = k * (mx ? BK_MX : BK);
        if (lane < loads) {
          if (u.phase == PH_UP) tma_gather4(b + lane * 512, map + M_X_ROWS, &sh.full[stage], kc, t[0], t[1], t[2], t[3]);
          else tma_load_2d(b + lane * 2048, map + (u.phase == PH_SHARED ? M_X : u.routed ? M_H : M_H_S), &sh.full[stage], kc, u.off + lane * 16);
        }
        __syncwarp();
      }
    }
  } else if (warp == 3) {
    // ---------------- MXFP8: the scale block of a step's tokens, lane l rows l and l + 32 (for other steps only the arrival)
    if (MX) {
      bool ok = true, have_h = false;
#pragma unroll 1
      for (; ok; ++at) {
        int go = 1;
        if (lane == 0) go = dec_wait(&sh.q_full[q_slot()], q_parity(), p);
        if (!__shfl_sync(0xffffffffu, go, 0)) break;
        __syncwarp();
        const Unit u = sh.queue[q_slot()];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.q_empty[q_slot()]);
        if (u.phase < 0) break;
        if (u.phase == PH_DOWN && !have_h) {
          if (lane == 0) go = dec_wait_count(CTR_H, (int)gridDim.x, p);
          if (!__shfl_sync(0xffffffffu, go, 0)) break;
          __syncwarp();
          have_h = true;
        }
        const uint32_t* src[2] = {nullptr, nullptr};
        if (u.routed) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int r = lane + 32 * j;
            if (r < u.n)
              src[j] = reinterpret_cast<const uint32_t*>(u.phase == PH_UP ? p.xs + (size_t)token_of(p, sched.row[u.off + r]) * (p.D / 32)
                                                                         : p.hs + (size_t)(u.off + r) * (p.I / 32));
          }
        }
        uint32_t ahead[4][2];  // four steps' words
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
          for (int j = 0; j < 2; ++j) ahead[d][j] = src[j] && u.k0 + d < u.k1 ? __ldcg(src[j] + u.k0 + d) : 0u;
#pragma unroll 1
        for (int k = u.k0; k < u.k1; ++k, advance()) {
          if (lane == 0) go = dec_wait(&sh.empty[stage], parity ^ 1u, p);
          if (!(ok = __shfl_sync(0xffffffffu, go, 0) != 0)) break;
          uint8_t* to = sf + stage * 2 * SF_BLOCK_BYTES + SF_BLOCK_BYTES + lane * 16;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (u.routed) *reinterpret_cast<uint32_t*>(to + 4 * j) = ahead[0][j];
#pragma unroll
            for (int d = 0; d < 3; ++d) ahead[d][j] = ahead[d + 1][j];
            ahead[3][j] = src[j] && k + 4 < u.k1 ? __ldcg(src[j] + k + 4) : 0u;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.full[stage]);
        }
      }
    }
  } else if (warp == 1) {
    // ---------------- products
    if (elect_one()) {
      int acc = 0;
      uint32_t acc_parity = 1;
      bool ok = true;
#pragma unroll 1
      for (; ok; ++at) {
        if (!dec_wait(&sh.q_full[q_slot()], q_parity(), p)) break;
        const Unit& q = sh.queue[q_slot()];
        const int phase = q.phase, k0 = q.k0, k1 = q.k1;
        const bool mx = MX && q.routed;
        const uint32_t n = (uint32_t)(q.n + 15) & ~15u;
        mbar_arrive(&sh.q_empty[q_slot()]);
        if (phase < 0) break;
        const uint32_t idesc = mx ? idesc_mxf8_e4m3(128, n) : idesc_bf16_f32(128, n);
        if (!dec_wait(&sh.acc_empty[acc], acc_parity, p)) break;
        tc_fence_after();
        const uint32_t d = tmem + acc * DEC_MAX_T, sfa = tmem + 2 * DEC_MAX_T, sfb = sfa + 4;
#pragma unroll 1
        for (int k = k0; k < k1; ++k, advance()) {
          if (!(ok = dec_wait(&sh.full[stage], parity, p))) break;
          tc_fence_after();
          const uint32_t a = smem_u32(smem + stage * stage_bytes), b = a + DEC_A_BYTES;
          if (mx) {
            const uint32_t f = smem_u32(sf + stage * 2 * SF_BLOCK_BYTES);
            tmem_cp_32x128b_warpx4(sfa, sdesc_sf_block(f));
            tmem_cp_32x128b_warpx4(sfb, sdesc_sf_block(f + SF_BLOCK_BYTES));
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_mxf8_ss(d, sdesc_kmajor_sw128(a + kk * 32), sdesc_kmajor_sw128(b + kk * 32),
                          idesc | ((uint32_t)kk << 4) | ((uint32_t)kk << 29), sfa, sfb, k != k0 || kk ? 1u : 0u);
          } else {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_bf16_ss(d, sdesc_kmajor_sw128(a + kk * 32), sdesc_kmajor_sw128(b + kk * 32), idesc, k != k0 || kk ? 1u : 0u);
          }
          mma_commit(&sh.empty[stage]);
        }
        if (!ok) break;
        mma_commit(&sh.acc_full[acc]);
        acc ^= 1;
        if (!acc) acc_parity ^= 1u;
      }
    }
    __syncwarp();
  } else {
    // ---------------- routing, then the accumulators (TMEM lanes 32 ew .. 32 ew + 31)
    const int ew = warp - 4, tid = threadIdx.x - 128;
    bool ok = true;
    if (!p.given) {
      TopkScratch& scratch = *reinterpret_cast<TopkScratch*>(sched.mask);
      const bool own = p.T <= DEC_OWN_TOPK;
      int done = 0;
#pragma unroll 1
      for (int t = own ? 0 : blockIdx.x; t < p.T; t += own ? 1 : gridDim.x, ++done) {
        token_topk(p, t, tid, scratch, reinterpret_cast<float2*>(sched.row), reinterpret_cast<unsigned long long*>(sched.w),
                   own ? scratch.idx + t * p.k : p.topk_idx + (size_t)t * p.k, own ? scratch.w + t * p.k : p.topk_w + (size_t)t * p.k);
        named_bar_sync(3, 128);
      }
      if (own) {
        if (tid < p.T * p.k) sched.idx[tid] = (uint16_t)scratch.idx[tid], sched.w[tid] = scratch.w[tid];
        named_bar_sync(3, 128);
      }
      if (!own) {
        if (tid == 0 && done) red_release_add_gpu(p.counters + CTR_TOPK, done);
        // (one thread asks: the others' loads would be in the way of those that work)
        ok = agree(tid != 0 || dec_wait_count(CTR_TOPK, p.T, p));
      }
    }
    if (ok) build_schedule(p, sched, tid);
    named_bar_sync(3, 128);
    if (ok) mbar_arrive(&sh.ready);

    // all units of a phase are done: `mine` of them here.  (One thread asks.)
    auto all_done = [&](int ctr, int mine, int all) {
      named_bar_sync(3, 128);
      if (tid == 0) red_release_add_gpu(p.counters + ctr, mine);
      return agree(tid != 0 || dec_wait_count(ctr, all, p));
    };
    int acc = 0, units[2] = {0, 0};  // up/gate and down units
    uint32_t acc_parity = 0;
    bool have_h = false;
#pragma unroll 1
    for (; ok; ++at) {
      if (!(ok = agree(dec_wait(&sh.q_full[q_slot()], q_parity(), p)))) break;
      const Unit& q = sh.queue[q_slot()];
      const int phase = q.phase, n = q.n;
      float* to = q.sums + tid;
      mbar_arrive(&sh.q_empty[q_slot()]);
      if (!have_h && (phase < 0 || phase == PH_DOWN)) {  // the last of this CTA's up/gate units is done
        if (!(ok = all_done(CTR_UP, units[0], n_shared + sched.n_u))) break;
        finish_up(p, sched, ew);
        fence_proxy_async_global();  // h is read by TMA
        named_bar_sync(3, 128);
        if (tid == 0) red_release_add_gpu(p.counters + CTR_H, 1);
        have_h = true;
      }
      if (phase < 0) break;
      ++units[phase == PH_DOWN];
      if (!(ok = agree(dec_wait(&sh.acc_full[acc], acc_parity, p)))) break;
      tc_fence_after();
      const uint32_t taddr = tmem + acc * DEC_MAX_T + ((uint32_t)(32 * ew) << 16);
#pragma unroll 1
      for (int n0 = 0; n0 < n; n0 += 16) {
        uint32_t v[16];
        tmem_ld_32x32b_x16(taddr + n0, v);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          if (n0 + j >= n) break;
          to[(n0 + j) * 128] = __uint_as_float(v[j]);
        }
      }
      tc_fence_before();
      mbar_arrive(&sh.acc_empty[acc]);
      acc ^= 1;
      if (!acc) acc_parity ^= 1u;
    }
    if (ok && all_done(CTR_DOWN, units[1], sched.n_d)) finish_down(p, sched, ew);  // (without any expert: zeros)
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
  size_t status, counters, logits, topk_idx, topk_w, xq, xs, h, hs, h_s, sums_s, sums_u, sums_d, sums_ds, total;
  int q_s, q_ds, most_u, most_d;
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
  const int64_t step = mx ? BK_MX : BK, kd = c.D / step, ki = c.I / step;
  auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  // units: the shared expert's up/gate projections are cut here, the others when the
  // experts are known, into at most so many pieces (fewer for more tokens, whose sums are larger).
  // Rows times pieces would now and then be fewer for one token more; the room for them is not, so
  // that a workspace for some tokens does for any fewer
  auto steps = [&](int64_t cap) { return dec_unit_steps((int)(c.I_s / 128 * 2 * (c.D / BK)), pl->num_sms, (int)cap); };
  L.q_s = steps(ncap);
  int64_t rows_s = 0;
  for (int64_t cap = 16; cap <= ncap; cap += 16) {
    const int64_t rows = (T < cap ? T : cap) * up(c.D / BK, steps(cap));
    rows_s = rows > rows_s ? rows : rows_s;
  }
  const int64_t most = T <= 8 ? 16 : 128 / T, rows_most = T <= 8 ? 16 * T : 128;  // (at least T most)
  auto rows_of = [&](int64_t pieces) { return T * pieces < rows_most ? T * pieces : rows_most; };
  L.most_u = (int)(most < up(kd, 4) ? most : up(kd, 4));
  L.most_d = (int)(most < up(ki, 4) ? most : up(ki, 4));
  L.q_ds = (int)up(c.I_s / BK, most);
  L.counters = take(sizeof(int) * DEC_COUNTERS);
  L.logits = take(sizeof(float2) * T * c.E);
  L.topk_idx = take(sizeof(int) * R);
  L.topk_w = take(sizeof(float) * R);
  L.xq = take(mx ? T * c.D : 0);
  L.xs = take(mx ? T * (c.D / 32) : 0);
  L.h = take((size_t)R * c.I * (mx ? 1 : 2));
  L.hs = take(mx ? R * (c.I / 32) : 0);
  L.h_s = take((size_t)DEC_MAX_T * c.I_s * 2);
  L.sums_s = take((size_t)(c.I_s / 128) * 2 * rows_s * 512);
  L.sums_u = take((size_t)(c.I / 128) * 2 * rows_of(up(kd, 4)) * c.k * 512);
  L.sums_d = take((size_t)(c.D / 128) * rows_of(up(ki, 4)) * c.k * 512);
  L.sums_ds = take((size_t)(c.D / 128) * (c.I_s ? rows_most : 0) * 512);
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
  p.inv_k = (65536 + p.k - 1) / p.k;
  p.score_fn = c.score_fn;
  p.given = given;
  p.mx = mx;
  p.ncap = (int)((T + 15) / 16 * 16);
  p.stage_bytes = DEC_A_BYTES + p.ncap * 128;
  const int room = DEC_SMEM - dec_smem_fixed(), per = p.stage_bytes + (mx ? 2 * SF_BLOCK_BYTES : 0);
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
  p.sums_s = reinterpret_cast<float*>(ws + L.sums_s), p.sums_u = reinterpret_cast<float*>(ws + L.sums_u);
  p.sums_d = reinterpret_cast<float*>(ws + L.sums_d), p.sums_ds = reinterpret_cast<float*>(ws + L.sums_ds);
  p.q_s = L.q_s, p.q_ds = L.q_ds, p.most_u = L.most_u, p.most_d = L.most_d;
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
  // (the limit belongs to the kernel, not to the launch, and another thread's call may set it in between: the same for all)
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, DEC_SMEM) != cudaSuccess) return MOE_ERR_CUDA;
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
