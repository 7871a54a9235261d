// Momentum and orthogonalised updates of stacked weight matrices
// (moe_muon_update in include/moe.h).
//
// Newton-Schulz steps on X = U / |U|_F, m = min(rows, cols), n = max(rows, cols):
//   A = X X^T (rows <= cols; else X^T X),  B = b A + c A^2,  X <- a X + B X (else a X + X B).
// Every product is one tcgen05 GEMM over the whole stack (grid of CTA pairs,
// M = N = 256 tiles); A and A^2 are symmetric, so only the tiles on and below
// the diagonal are computed and the others are written as their transposes.
//
// Precision.  Operands are fp16 (11 bits; bf16's 8 leave errors of 1e-2 to
// 1e-1 in the result), sums fp32.  A polynomial step multiplies a small
// singular value by a and leaves a large one near 1, so an error made in X in
// all directions grows against the small ones: rounding X itself to fp16 each
// step costs 1e-2 on decaying spectra.  X is therefore held as hi + lo, two
// fp16 numbers (22 bits); the term a X is taken from both, and only B X, which
// lies in the directions of the large singular values, from hi.  The diagonals
// of A and B, which carry most of them where the rows are nearly orthogonal,
// are kept in fp32 beside fp16 matrices without a diagonal (A = D + O gives
// A^2 = O^2 + D O + O D + D^2) and are applied to the fp32 sums.  B's diagonal
// multiplies hi in the early steps, so that it cancels against the other
// elements' share in the small directions, and hi + lo in the last two, after
// which nothing grows any more.  Left against fp64 (relative Frobenius norm,
// over flat, decaying and rank-deficient spectra): 2e-4 to 1.4e-3, with 16 rows
// up to 1.9e-3, before the result's own rounding to bf16 (1.7e-3).
//
// Scales.  fp16 has 5 exponent bits, so X_0 is U 2^k with |U 2^k|_F in
// [2^14, 2^15): no element overflows, and those down to 2^-28 of the norm keep
// their 11 bits.  Later iterates, A and B are held times 2^12, so they must stay
// below 16 (|X|_2 < 1.3 for the default coefficients; others are checked when the
// plan is made, ns_in_range); the factors, and what is left of 1 / |U|_F, are
// applied to the fp32 sums.
#include <cuda_fp16.h>

#include <cmath>
#include <cstring>
#include <new>
#include <type_traits>

#include "../../include/moe.h"
#include "common.cuh"
#include "plan.cuh"

namespace moe {

constexpr int NS_THREADS = 352;       // producer, MMA issuer, eight epilogue warps, the epilogue's loads and stores
constexpr int NS_TILE = 256;          // of a CTA pair: 256 x 256, or 256 x 128 (narrow), 128 rows in each CTA
constexpr int NS_BOX = 8192;          // one {64, 64} fp16 box
constexpr int NS_STAGE = 4 * NS_BOX;  // per CTA: 128 rows of A and half of B's 256, 64 of K
constexpr int NS_STAGES = 5;
constexpr int NS_EBUF = 4 * NS_BOX;   // epilogue buffer: two tiles of 128 rows x 64 columns
constexpr int NS_SMEM = NS_STAGES * NS_STAGE + 2 * NS_EBUF + 1024 + 256;
constexpr float NS_S = 4096.0f;       // scale of the held iterates, A and B
constexpr int NS_PREP_BLOCKS = 1024;  // partial sums per matrix, at most

enum : int { NS_GRAM = 0, NS_POLY = 1, NS_STEP = 2 };

struct NsMaps {
  CUtensorMap a, b, b64;    // operands; b64: the second for narrow tiles (box of 64 rows; MN-major the same as b)
  CUtensorMap in0, in1;     // box {64, 128}: POLY: A; STEP: X's hi and lo
  CUtensorMap out0, out1;   // box {64, 128}: A or B, and (box {64, 64}) its transposed tiles; STEP: hi and lo, or the update
};

struct NsParams {
  int M, N, K;             // of one matrix's product
  int nb;                  // matrices
  int tiles_n, n_tiles;    // column tiles; tiles per matrix (symmetric: the lower ones)
  int n_wide, n_units;     // the first tiles of the launch, whole; and with the others' halves
  int first, last;         // Newton-Schulz step
  int diag_full;           // STEP: B's diagonal multiplies hi + lo, not hi
  int tall;                // STEP: X B, B's diagonal belongs to the columns
  int out_vec;             // the update goes out through its tensor map (16-byte aligned rows)
  int ldd;                 // matrix stride of the diagonals
  float ca, cb;            // POLY: B = ca A + cb A^2; STEP: X <- ca X + diag(B) X + cb sum
  float scale;             // of the final update
  const float* rho;        // [nb] 1 / |U 2^k|_F
  float* diag_a;           // [nb, ldd] A's diagonal times NS_S
  float* diag_b;           // [nb, ldd] B's diagonal
  bf16* out_final;
  int* status;
  long long timeout_ns;
};

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* smem_src, int32_t c0, int32_t c1, int32_t c2) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(smem_src)), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}

__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t smem_addr) {  // MN-major, {64, 64} boxes 8192 B apart
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(NS_BOX >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}
// .kind::f16 with fp16 A and B (format 0), fp32 D
constexpr uint32_t ns_idesc(int tn, bool a_mn, bool b_mn) {
  return (1u << 4) | ((uint32_t)(tn >> 3) << 17) | ((NS_TILE >> 4) << 24) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u);
}

struct NsTile {
  int mat, m0, n0, w;  // w: columns, 256 or 128
};
// Unit u: a whole tile, or from n_wide on half of one.  Symmetric products: the
// tiles on and below the diagonal, row by row.
template <int KIND>
__device__ __forceinline__ NsTile ns_tile(const NsParams& p, int u) {
  NsTile t;
  const bool wide = u < p.n_wide;
  const int g = wide ? u : p.n_wide + (u - p.n_wide) / 2;
  t.mat = g / p.n_tiles;
  const int v = g - t.mat * p.n_tiles;
  int i, j;
  if (KIND == NS_STEP) {
    i = v / p.tiles_n;
    j = v - i * p.tiles_n;
  } else {
    i = (int)((sqrtf(8.0f * (float)v + 1.0f) - 1.0f) * 0.5f);
    while (i * (i + 1) / 2 > v) --i;
    while ((i + 1) * (i + 2) / 2 <= v) ++i;
    j = v - i * (i + 1) / 2;
  }
  t.m0 = i * NS_TILE;
  t.n0 = j * NS_TILE + (wide ? 0 : ((u - p.n_wide) & 1) * 128);
  t.w = wide ? 256 : 128;
  return t;
}

__device__ __forceinline__ void unpack8(const uint4& w, float* v) {
  const __half2* h = reinterpret_cast<const __half2*>(&w);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float2 f = __half22float2(h[q]);
    v[2 * q] = f.x;
    v[2 * q + 1] = f.y;
  }
}
__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint4 pack8(const __half* h) {
  return make_uint4((uint32_t)__half_as_ushort(h[0]) | ((uint32_t)__half_as_ushort(h[1]) << 16),
                    (uint32_t)__half_as_ushort(h[2]) | ((uint32_t)__half_as_ushort(h[3]) << 16),
                    (uint32_t)__half_as_ushort(h[4]) | ((uint32_t)__half_as_ushort(h[5]) << 16),
                    (uint32_t)__half_as_ushort(h[6]) | ((uint32_t)__half_as_ushort(h[7]) << 16));
}

// One row (TMEM lane) of half an epilogue chunk (32 of 64 columns, from i0 * 8):
// `main` holds this row's inputs and takes its outputs in place (POLY: A -> B;
// STEP: hi), `aux` is lo, or takes the chunk transposed (symmetric products'
// tiles below the diagonal).  Rows of 128 bytes, 16-byte pieces swizzled as the
// tensor maps'.
// g: the row's diagonal element (POLY: A's; STEP, not tall: B's).
template <int KIND>
__device__ __forceinline__ void ns_chunk(const NsParams& p, const NsTile& t, uint8_t* main, uint8_t* aux, int rl, int r,
                                         int c0, int i0, float rho, float g, uint32_t taddr) {
  const int cw = c0 + 8 * i0;  // this warp's columns: cw .. cw + 31
  // the columns' diagonal (the same for the whole warp), on its way while TMEM is read
  float4 dv[KIND == NS_GRAM ? 1 : 8];
  const bool by_column = KIND == NS_POLY || (KIND == NS_STEP && p.tall);
  if (by_column) {
    const float4* d4 = reinterpret_cast<const float4*>((KIND == NS_POLY ? p.diag_a : p.diag_b) + (size_t)t.mat * p.ldd + cw);
#pragma unroll
    for (int i = 0; i < (KIND == NS_GRAM ? 1 : 8); ++i) dv[i] = d4[i];
  }
  uint32_t acc[32];
  tmem_ld_32x32b_x32(taddr + 8u * (uint32_t)i0, acc);
  tmem_ld_wait();
  const bool mirror = KIND != NS_STEP && t.n0 < t.m0;  // (the halves of a diagonal tile are both computed)
  // the diagonal crosses a warp's 32 x 32 elements from corner to corner or not at all
  const int lane = rl & 31, diag = KIND != NS_STEP && r - lane == cw ? lane : -1;
  float f = 1.0f, cb = p.cb;
  if (KIND == NS_GRAM) f = p.first ? rho * rho * NS_S : 1.0f / NS_S;
  if (KIND == NS_STEP && p.first) f = NS_S * rho, cb = rho;
  const float fa = KIND == NS_POLY ? p.ca + cb * g : f * p.ca;
#pragma unroll
  for (int ii = 0; ii < 4; ++ii) {
    const int i = i0 + ii;
    uint4* at = reinterpret_cast<uint4*>(main + rl * 128 + ((i ^ (rl & 7)) << 4));
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(acc[8 * ii + j]);
    if (KIND == NS_GRAM) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= f;
      float on = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        on = 8 * ii + j == diag ? v[j] : on;
        v[j] = 8 * ii + j == diag ? 0.0f : v[j];
      }
      if (diag >> 3 == ii && r < p.M) p.diag_a[(size_t)t.mat * p.ldd + r] = on;
    } else {
      float x[8], d[8];
      unpack8(*at, x);
      if (by_column) {
        const float4 w0 = dv[KIND == NS_GRAM ? 0 : 2 * ii], w1 = dv[KIND == NS_GRAM ? 0 : 2 * ii + 1];
        d[0] = w0.x, d[1] = w0.y, d[2] = w0.z, d[3] = w0.w, d[4] = w1.x, d[5] = w1.y, d[6] = w1.z, d[7] = w1.w;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = g;
      }
      if (KIND == NS_POLY) {  // b O + c (O^2 + (D_r + D_c) O); on the diagonal b D + c (O^2 + D^2)
        float on = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) on = 8 * ii + j == diag ? v[j] : on;
        if (diag >> 3 == ii && r < p.M) p.diag_b[(size_t)t.mat * p.ldd + r] = (p.ca * g + cb * (on + g * g)) / NS_S;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 8 * ii + j == diag ? 0.0f : x[j] * (fa + cb * d[j]) + cb * v[j];
      } else {
        uint4* al = reinterpret_cast<uint4*>(aux + rl * 128 + ((i ^ (rl & 7)) << 4));
        float lo[8];
        unpack8(*al, lo);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float both = x[j] + lo[j];
          v[j] = both * fa + ((p.diag_full ? both : x[j]) * (f * d[j]) + cb * v[j]);
        }
        if (p.last) {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] *= p.scale;
          *at = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
          continue;
        }
        uint32_t l[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 h = __half22float2(__floats2half2_rn(v[2 * j], v[2 * j + 1]));
          l[j] = pack_half2(v[2 * j] - h.x, v[2 * j + 1] - h.y);
        }
        *al = make_uint4(l[0], l[1], l[2], l[3]);
      }
    }
    uint32_t h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = pack_half2(v[2 * j], v[2 * j + 1]);
    *at = make_uint4(h[0], h[1], h[2], h[3]);
    if (mirror) {  // element (r, c) goes to row c, column r; two 64-column boxes
      uint8_t* b = aux + (rl >> 6) * NS_BOX;
      const int rc = rl & 63;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        *reinterpret_cast<uint16_t*>(b + (8 * i + j) * 128 + (((rc >> 3) ^ j) << 4) + (rc & 7) * 2) =
            (uint16_t)(h[j / 2] >> (16 * (j & 1)));
    }
  }
  if (KIND == NS_STEP && p.last && !p.out_vec) {
    // rows that no tensor map can describe: from shared memory, a row of the
    // warp's 32 at a time (each thread storing its own row took 35 us more for
    // 3 x 777 x 1001)
    __syncwarp();
    const int col = 8 * i0 + (int)lane_id(), rl0 = rl & ~31, r0 = r - (rl & 31);
    bf16* o = p.out_final + (size_t)t.mat * (size_t)p.M * p.N + c0 + col;
#pragma unroll 4
    for (int k = 0; k < 32; ++k) {
      const int q = rl0 + k;
      if (r0 + k < p.M && c0 + col < p.N)
        o[(size_t)(r0 + k) * p.N] =
            *reinterpret_cast<const bf16*>(main + q * 128 + (((col >> 3) ^ (q & 7)) << 4) + (col & 7) * 2);
    }
  }
}

// Persistent CTA pairs, one per SM pair; pair u takes tiles u, u + pairs, ...
// Warp 0: TMA producer of this CTA's operands (counted on the even CTA's full
// barrier); warp 1 of the even CTA: tcgen05.mma for both; warps 2-9: epilogue
// of this CTA's 128 rows, 64 columns at a time, two warps to 32 rows; warp 10:
// loads the epilogue's inputs into the two epilogue buffers and stores its
// outputs from them, both by TMA, the loads ahead of the accumulator.  Two
// accumulators of 256 columns in TMEM alternate, so a tile's epilogue runs under
// the next tile's products.
// (Rows read and written by the threads themselves, 32 rows of 16 bytes at a
// time, took 30 us a tile of X against 12 us of products.)
// 16 x 2048 x 7168, against 1715 TFLOP/s of a sustained library product: A 322
// us (1680 TFLOP/s), A^2 100 us (1550), X 644 us (1494: its tiles also move
// 128 KB in and 128 KB out per CTA).  The card is at its power limit there, at
// 1.5 GHz.
template <int KIND, bool A_MN, bool B_MN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NS_THREADS, 1)
    ns_gemm(const __grid_constant__ NsMaps mp, const NsParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ebuf = smem + NS_STAGES * NS_STAGE;
  uint64_t* full = reinterpret_cast<uint64_t*>(ebuf + 2 * NS_EBUF);           // [NS_STAGES]
  uint64_t* empty = full + NS_STAGES;                                         // [NS_STAGES]
  uint64_t* tfull = empty + NS_STAGES;                                        // [2]
  uint64_t* tempty = tfull + 2;                                               // [2]
  uint64_t* eload = tempty + 2;                                               // [2] inputs landed (or buffer free)
  uint64_t* edone = eload + 2;                                                // [2] outputs written
  uint64_t* drain = edone + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  static_assert((2 * NS_STAGES + 9) * 8 + 4 <= 256, "barrier area");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)(cluster_ctarank() & 1u);
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int n_units = p.n_units;
  const int nk = (p.K + BK - 1) / BK;
  // epilogue chunks of this CTA's part of a tile
  auto chunks = [&](const NsTile& t) { return t.m0 + rank * 128 < p.M ? (min(t.w, p.N - t.n0) + 63) / 64 : 0; };
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS_STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 16);  // one arrival per epilogue warp of both CTAs
      mbar_init(&eload[a], 1);
      mbar_init(&edone[a], 8);    // one per epilogue warp
    }
    mbar_init(drain, 1);
    fence_barrier_init();
    prefetch_tensormap(&mp.a);
    prefetch_tensormap(&mp.b);
    prefetch_tensormap(&mp.b64);
  }
  if (warp == 1) {
    tmem_alloc_pair<512>(tmem_slot);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // the other CTA's barriers exist before anything targets them
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the inputs are the last launch's results
  int failed = 0;  // a wait of this thread ran out

  if (warp == 0) {
    if (lane == 0) {
      const uint32_t full_even = mapa_shared(full, 0);
      uint32_t stage = 0, phase = 0;
      int issued = 0;
      bool ok = true;
      for (int u = pair; u < n_units && ok; u += pairs) {
        const NsTile t = ns_tile<KIND>(p, u);
        const int ar = t.m0 + rank * 128, br = t.n0 + rank * (t.w / 2);
        const bool wide = t.w == 256;
        for (int s = 0; s < nk; ++s) {
          if (!mbar_wait_cluster(&empty[stage], phase ^ 1u, p.status, p.timeout_ns)) { ok = false; failed = 1; break; }
          uint8_t* sa = smem + stage * NS_STAGE;
          uint8_t* sb = sa + 2 * NS_BOX;
          if (leader) mbar_arrive_expect_tx(&full[stage], 2u * (wide ? 4u : 3u) * NS_BOX);
          const uint32_t fb = full_even + 8u * stage;
          if (A_MN) {
            tma_load_3d_pair(sa, &mp.a, fb, ar, s * BK, t.mat);
            tma_load_3d_pair(sa + NS_BOX, &mp.a, fb, ar + 64, s * BK, t.mat);
          } else {
            tma_load_3d_pair(sa, &mp.a, fb, s * BK, ar, t.mat);
          }
          if (B_MN) {
            tma_load_3d_pair(sb, &mp.b, fb, br, s * BK, t.mat);
            if (wide) tma_load_3d_pair(sb + NS_BOX, &mp.b, fb, br + 64, s * BK, t.mat);
          } else {
            tma_load_3d_pair(sb, wide ? &mp.b : &mp.b64, fb, s * BK, br, t.mat);
          }
          ++issued;
          if (++stage == NS_STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      // both CTAs' last loads have landed before either leaves (the odd CTA
      // waits for the even one at the cluster barrier below)
      if (leader)
        for (int i = (issued > NS_STAGES ? issued - NS_STAGES : 0); i < issued; ++i)
          mbar_wait_drain(&full[i % NS_STAGES], (uint32_t)(i / NS_STAGES) & 1u, p.timeout_ns);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (leader && elect_one()) {
      uint32_t stage = 0, phase = 0;
      int i = 0;
      bool ok = true;
      for (int u = pair; u < n_units && ok; u += pairs, ++i) {
        const uint32_t acc = (uint32_t)i & 1u;
        const uint32_t id = u < p.n_wide ? ns_idesc(256, A_MN, B_MN) : ns_idesc(128, A_MN, B_MN);
        if (!mbar_wait_cluster(&tempty[acc], (((uint32_t)i >> 1) & 1u) ^ 1u, p.status, p.timeout_ns)) { failed = 1; break; }
        tc_fence_after();
        const uint32_t d = tmem + acc * 256u;
        for (int s = 0; s < nk; ++s) {
          if (!mbar_wait_cluster(&full[stage], phase, p.status, p.timeout_ns)) { ok = false; failed = 1; break; }
          tc_fence_after();
          const uint32_t a_addr = smem_u32(smem + stage * NS_STAGE);
          const uint32_t b_addr = a_addr + 2 * NS_BOX;
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk) {
            const uint64_t ad = A_MN ? sdesc_mn_sw128(a_addr + kk * 2048) : sdesc_kmajor_sw128(a_addr + kk * 32);
            const uint64_t bd = B_MN ? sdesc_mn_sw128(b_addr + kk * 2048) : sdesc_kmajor_sw128(b_addr + kk * 32);
            mma_bf16_pair(d, ad, bd, id, (s | kk) != 0 ? 1u : 0u);
          }
          mma_commit_pair(&empty[stage], 0x3);
          if (++stage == NS_STAGES) { stage = 0; phase ^= 1u; }
        }
        if (ok) mma_commit_pair(&tfull[acc], 0x3);
      }
      mma_commit_pair(drain, 0x1);
      mbar_wait_drain(drain, 0, p.timeout_ns);  // every MMA issued has completed before TMEM is freed
    }
    __syncwarp();
  } else if (warp < 10) {
    const int q = warp & 3, rl = q * 32 + lane, half = (warp - 2) >> 2;
    const uint32_t tempty_even = mapa_shared(tempty, 0);
    int i = 0, n = 0;
    bool ok = true;
    for (int u = pair; u < n_units && ok; u += pairs, ++i) {
      const NsTile t = ns_tile<KIND>(p, u);
      const uint32_t acc = (uint32_t)i & 1u;
      const int nc = chunks(t);
      const float rho = p.first ? p.rho[t.mat] : 0.0f;
      float g = 0.0f;
      if (KIND == NS_POLY) g = p.diag_a[(size_t)t.mat * p.ldd + t.m0 + rank * 128 + rl];
      if (KIND == NS_STEP && !p.tall) g = p.diag_b[(size_t)t.mat * p.ldd + t.m0 + rank * 128 + rl];
      if (!__all_sync(0xffffffffu, mbar_wait_cluster(&tfull[acc], ((uint32_t)i >> 1) & 1u, p.status, p.timeout_ns))) { failed = 1; break; }
      tc_fence_after();
      const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + acc * 256u;
#pragma unroll 1
      for (int c = 0; c < nc; ++c, ++n) {
        const int b = n & 1;
        if (!__all_sync(0xffffffffu, mbar_wait(&eload[b], ((uint32_t)n >> 1) & 1u, p.status, p.timeout_ns))) { ok = false; failed = 1; break; }
        uint8_t* e = ebuf + b * NS_EBUF;
        ns_chunk<KIND>(p, t, e, e + 2 * NS_BOX, rl, t.m0 + rank * 128 + rl, t.n0 + 64 * c, 4 * half, rho, g,
                       taddr + 64u * (uint32_t)c);
        fence_proxy_async_smem();  // these writes, before the TMA store that follows the arrival
        __syncwarp();
        if (lane == 0) mbar_arrive(&edone[b]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && ok) mbar_arrive_remote(tempty_even + acc * 8u);
    }
  } else if (lane == 0) {
    // chunk n uses buffer n & 1: loaded two chunks ahead, once the chunk before
    // in that buffer has been stored
    int lu = pair, lc = 0, ln = 0;  // next chunk to load: unit, chunk of its tile, number
    auto load_next = [&]() {
      while (lu < n_units) {
        const NsTile t = ns_tile<KIND>(p, lu);
        if (lc >= chunks(t)) {
          lu += pairs;
          lc = 0;
          continue;
        }
        const int b = ln & 1, row = t.m0 + rank * 128, col = t.n0 + 64 * lc;
        uint8_t* e = ebuf + b * NS_EBUF;
        if (KIND == NS_GRAM) {
          mbar_arrive(&eload[b]);
        } else {
          mbar_arrive_expect_tx(&eload[b], (KIND == NS_STEP ? 4u : 2u) * NS_BOX);
          tma_load_3d(e, &mp.in0, &eload[b], col, row, t.mat);
          if (KIND == NS_STEP) tma_load_3d(e + 2 * NS_BOX, &mp.in1, &eload[b], col, row, t.mat);
        }
        ++lc;
        ++ln;
        return;
      }
    };
    load_next();
    load_next();
    int n = 0;
    bool ok = true;
    for (int u = pair; u < n_units && ok; u += pairs) {
      const NsTile t = ns_tile<KIND>(p, u);
      const int nc = chunks(t), row = t.m0 + rank * 128;
      for (int c = 0; c < nc; ++c, ++n) {
        const int b = n & 1, col = t.n0 + 64 * c;
        if (!mbar_wait(&edone[b], ((uint32_t)n >> 1) & 1u, p.status, p.timeout_ns)) { ok = false; failed = 1; break; }
        const uint8_t* e = ebuf + b * NS_EBUF;
        if (KIND == NS_STEP) {
          if (!p.last || p.out_vec) tma_store_3d(&mp.out0, e, col, row, t.mat);
          if (!p.last) tma_store_3d(&mp.out1, e + 2 * NS_BOX, col, row, t.mat);
        } else {
          tma_store_3d(&mp.out0, e, col, row, t.mat);
          if (t.n0 < t.m0) {
            tma_store_3d(&mp.out1, e + 2 * NS_BOX, row, col, t.mat);
            if (row + 64 < p.M) tma_store_3d(&mp.out1, e + 3 * NS_BOX, row + 64, col, t.mat);
          }
        }
        bulk_commit_group();
        bulk_wait_group_read<0>();
        load_next();
      }
    }
    bulk_wait_group_all();
    // (after a wait that ran out: the inputs still on their way have landed)
    for (int k = ln > 2 ? ln - 2 : 0; k < ln; ++k) mbar_wait_drain(&eload[k & 1], ((uint32_t)k >> 1) & 1u, p.timeout_ns);
  }
  __syncwarp();
  tc_fence_before();
  // (the status word is read only if a wait of this CTA ran out: 0.7 us a launch)
  if (__syncthreads_or(failed)) settle_after_abort(p.status);
  // neither CTA frees TMEM or leaves while the other may still issue into its
  // TMEM, arrive on its barriers or load into its shared memory
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ------------------------------------------------------------------ momentum, norm, first iterate
struct PrepParams {
  const void* grad;
  int64_t grs, gms;        // gradient's row and matrix strides, elements
  int dtype, R, C, nesterov, nblk;
  int64_t ld;              // of the first iterate
  float mu;
  float* momentum;         // or NULL
  float* part;             // [nb, NS_PREP_BLOCKS, 4]
  float* rho;              // [nb]
  __half* hi;
  __half* lo;
  int* status;             // cleared by the call's first launch (NULL in the others)
};

// V consecutive values of the gradient (V = 8: 16-byte loads) or of fp32 memory
template <int V>
__device__ __forceinline__ void load_f32(const float* s, float (&v)[V]) {
  if constexpr (V == 8) {
    const float4 a = reinterpret_cast<const float4*>(s)[0], b = reinterpret_cast<const float4*>(s)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    v[0] = *s;
  }
}
template <int V>
__device__ __forceinline__ void load_grad(const void* g, int dtype, size_t i, float (&v)[V]) {
  if (dtype == MOE_DTYPE_FP32) {
    load_f32<V>(static_cast<const float*>(g) + i, v);
    return;
  }
  const uint16_t* s = static_cast<const uint16_t*>(g) + i;
  uint32_t w[(V + 1) / 2];
  if constexpr (V == 8) {
    const uint4 q = *reinterpret_cast<const uint4*>(s);
    w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
  } else {
    w[0] = *s;
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const uint16_t h = (uint16_t)(w[j / 2] >> (16 * (j & 1)));
    v[j] = dtype == MOE_DTYPE_BF16 ? __uint_as_float((uint32_t)h << 16) : __half2float(__ushort_as_half(h));
  }
}
// vectors of a thread in flight (of 8 values: 4 were 1 to 4% slower on large stacks)
__host__ __device__ constexpr int prep_unroll(int V) { return V == 8 ? 2 : 8; }

// Sums of squares in three sums of their own: values far from 1 are squared
// in scaled form, so that no finite matrix has an infinite norm and none that
// is not zero has a zero one.  (Squares up to 2^96, and up to 2^30 of them: below
// 2^126.  The smallest, of 2^-149, is 2^-106.)
__device__ __forceinline__ void add_square(float (&f)[3], float u) {
  const float a = fabsf(u);
  const bool big = a >= 0x1p48f, small = a < 0x1p-48f;
  const float v = u * (big ? 0x1p-80f : small ? 0x1p96f : 1.0f);
  f[0] += small ? v * v : 0.0f;
  f[1] += big || small ? 0.0f : v * v;
  f[2] += big ? v * v : 0.0f;
}
// The three sums over the block (256 threads), valid in thread 0, in a fixed order.
__device__ __forceinline__ void block_sum3(float (&f)[3], float (*s)[8]) {
#pragma unroll
  for (int q = 0; q < 3; ++q) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) f[q] += __shfl_xor_sync(0xffffffffu, f[q], o);
    if ((threadIdx.x & 31) == 0) s[q][threadIdx.x >> 5] = f[q];
  }
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int q = 0; q < 3; ++q) f[q] = ((s[q][0] + s[q][1]) + (s[q][2] + s[q][3])) + ((s[q][4] + s[q][5]) + (s[q][6] + s[q][7]));
  }
}
// U 2^k = (u f1) f2 has a norm in [2^14, 2^15); rho = 1 / that norm (0 for a
// matrix of zeros, NaN where the norm is not finite, which makes every element
// of that matrix's result NaN).
__device__ __forceinline__ void norm_scale(const float (&f)[3], float* f1, float* f2, float* rho) {
  const double norm = sqrt((double)f[0] * 0x1p-192 + (double)f[1] + (double)f[2] * 0x1p160);
  *f1 = *f2 = *rho = 0.0f;
  if (!(norm < (double)INFINITY)) {
    *rho = NAN;
  } else if (norm > 0.0) {
    int e;
    const double m = frexp(norm, &e);  // norm = m 2^e, m in [0.5, 1)
    const int k = 15 - e;
    *f1 = ldexpf(1.0f, k / 2);
    *f2 = ldexpf(1.0f, k - k / 2);
    *rho = (float)(0x1p-15 / m);
  }
}

// Advance the momentum and sum U's squares.  (16 x 2048 x 7168: 350 us, and
// ns_prep_first 410 to 450 us, 2.35 GB each: 6.7 and 5.2 to 5.7 TB/s.  The two passes
// over the same gradient and momentum cannot be one, as the first iterate needs the
// norm; a matrix at a time, so that the second would find them in L2, took 5% longer.)
template <int V>
__global__ void __launch_bounds__(256) ns_prep_norm(const PrepParams p) {
  constexpr int NS_PREP_U = prep_unroll(V);
  __shared__ float s[3][8];
  const int mat = blockIdx.y, cv = p.C / V, n = p.R * cv;
  const bool flat = p.grs == p.C;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (p.status && blockIdx.x == 0 && mat == 0 && threadIdx.x == 0) p.status[0] = 0;
  float* mom = p.momentum ? p.momentum + (size_t)mat * p.R * p.C : nullptr;
  float f[3] = {0.0f, 0.0f, 0.0f};
  for (int64_t i0 = (int64_t)blockIdx.x * (256 * NS_PREP_U) + threadIdx.x; i0 < n; i0 += (int64_t)gridDim.x * (256 * NS_PREP_U)) {
    float u[NS_PREP_U][V], m[NS_PREP_U][V];
#pragma unroll
    for (int q = 0; q < NS_PREP_U; ++q) {
      const int64_t i = i0 + 256 * q;
      if (i < n) {
        const size_t o = flat ? (size_t)i * V : (size_t)((int)i / cv) * p.grs + (size_t)((int)i % cv) * V;
        load_grad<V>(p.grad, p.dtype, (size_t)mat * p.gms + o, u[q]);
        if (mom) load_f32<V>(mom + (size_t)i * V, m[q]);
      }
    }
#pragma unroll
    for (int q = 0; q < NS_PREP_U; ++q) {
      const int64_t i = i0 + 256 * q;
      if (i >= n) break;
      if (mom) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          m[q][j] = p.mu * m[q][j] + u[q][j];
          u[q][j] = p.nesterov ? u[q][j] + p.mu * m[q][j] : m[q][j];
        }
        float* d = mom + (size_t)i * V;
        if constexpr (V == 8) {
          reinterpret_cast<float4*>(d)[0] = make_float4(m[q][0], m[q][1], m[q][2], m[q][3]);
          reinterpret_cast<float4*>(d)[1] = make_float4(m[q][4], m[q][5], m[q][6], m[q][7]);
        } else {
          d[0] = m[q][0];
        }
      }
#pragma unroll
      for (int j = 0; j < V; ++j) add_square(f, u[q][j]);
    }
  }
  block_sum3(f, s);
  if (threadIdx.x == 0)
    *reinterpret_cast<float4*>(p.part + ((size_t)mat * NS_PREP_BLOCKS + blockIdx.x) * 4) = make_float4(f[0], f[1], f[2], 0.0f);
}

// X_0 = U 2^k as hi + lo.
template <int V>
__global__ void __launch_bounds__(256) ns_prep_first(const PrepParams p) {
  constexpr int NS_PREP_U = prep_unroll(V);
  __shared__ float s[3][8];
  __shared__ float s_f[2];
  const int mat = blockIdx.y, cv = p.C / V, n = p.R * cv;
  const bool flat = p.grs == p.C;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float f[3] = {0.0f, 0.0f, 0.0f};
  for (int b = threadIdx.x; b < p.nblk; b += 256) {
    const float4 w = *reinterpret_cast<const float4*>(p.part + ((size_t)mat * NS_PREP_BLOCKS + b) * 4);
    f[0] += w.x, f[1] += w.y, f[2] += w.z;
  }
  block_sum3(f, s);
  if (threadIdx.x == 0) {
    float rho;
    norm_scale(f, &s_f[0], &s_f[1], &rho);
    if (blockIdx.x == 0) p.rho[mat] = rho;
  }
  __syncthreads();
  const float f1 = s_f[0], f2 = s_f[1];
  const float* mom = p.momentum ? p.momentum + (size_t)mat * p.R * p.C : nullptr;
  for (int64_t i0 = (int64_t)blockIdx.x * (256 * NS_PREP_U) + threadIdx.x; i0 < n; i0 += (int64_t)gridDim.x * (256 * NS_PREP_U)) {
    float u[NS_PREP_U][V], m[NS_PREP_U][V];
#pragma unroll
    for (int q = 0; q < NS_PREP_U; ++q) {
      const int64_t i = i0 + 256 * q;
      if (i < n) {
        const size_t o = flat ? (size_t)i * V : (size_t)((int)i / cv) * p.grs + (size_t)((int)i % cv) * V;
        if (!mom || p.nesterov) load_grad<V>(p.grad, p.dtype, (size_t)mat * p.gms + o, u[q]);
        if (mom) load_f32<V>(mom + (size_t)i * V, m[q]);
      }
    }
#pragma unroll
    for (int q = 0; q < NS_PREP_U; ++q) {
      const int64_t i = i0 + 256 * q;
      if (i >= n) break;
      __half h[8], l[8];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float x = (mom ? p.nesterov ? u[q][j] + p.mu * m[q][j] : m[q][j] : u[q][j]) * f1 * f2;
        h[j] = __float2half_rn(x);
        l[j] = __float2half_rn(x - __half2float(h[j]));
      }
      if constexpr (V == 8) {  // (rows of multiples of 8 are not padded)
        const size_t o = (size_t)mat * p.R * p.C + (size_t)i * V;
        *reinterpret_cast<uint4*>(p.hi + o) = pack8(h);
        *reinterpret_cast<uint4*>(p.lo + o) = pack8(l);
      } else {
        const size_t o = ((size_t)mat * p.R + (int)i / cv) * p.ld + (int)i % cv;
        p.hi[o] = h[0];
        p.lo[o] = l[0];
      }
    }
  }
}

// ------------------------------------------------------------------ small matrices: one launch
// min(rows, cols) <= 128: a cluster of CTAs keeps one matrix on chip from the
// gradient to the update.  Held as m x n with m the smaller side (so a tall
// matrix transposed), CTA r has columns r W .. r W + W - 1: x in registers
// (fp32, one row of 4 W / 16 columns per thread), its hi part in shared memory
// as the operand of both products -- K-major for X X^T, and, the same bytes,
// MN-major for B X.  The parts of A = X X^T are summed over the cluster through
// distributed shared memory, each CTA reducing 1 / cluster of the matrix and
// writing the sums to all; everything else is local.  16 x 128 x 256: 48 us,
// 10 of them for the gradient and the momentum and 6.5 a step, against 111 us
// in the general form's 17 launches.  What bounds it is the chain of a step:
// three products (1 us each from the barrier to the sums in TMEM) and what
// follows each of them.
constexpr int SM_THREADS = 512;
constexpr int SM_BLK = 16384;                       // 128 rows x 64 fp16, swizzled
constexpr int SM_PITCH = 132;                       // floats per row of a CTA's part of A
constexpr int SM_BYTES = 4 * SM_BLK + 2 * SM_BLK + 128 * SM_PITCH * 4 + 4096 + 1024;  // X, A or B, part; one CTA per SM

struct SmallParams {
  PrepParams in;
  bf16* out;
  int steps, tall, m, n, mp;  // mp: m rounded up to 16
  int vec;                    // rows of the stored matrix are 16-byte aligned vectors of 8
  float a, b, c, scale;
  int* status;
  long long timeout_ns;
};

__device__ __forceinline__ uint32_t sw_at(int r, int c) {  // byte of element (r, c) in 64-column blocks
  return (uint32_t)((c >> 6) * SM_BLK + r * 128 + ((((c & 63) >> 3) ^ (r & 7)) << 4) + (c & 7) * 2);
}
__device__ __forceinline__ uint64_t sdesc_mn_blocks(uint32_t smem_addr) {  // MN-major, 64-wide blocks SM_BLK apart
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(SM_BLK >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}
// 32 lanes x 16 consecutive 32-bit columns (lane base in taddr)
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ void st_cluster_u2(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

// WC: columns per thread (W = 4 WC)
template <int WC>
__global__ void __launch_bounds__(SM_THREADS, 1) ns_small(const __grid_constant__ SmallParams p) {
  constexpr int W = 4 * WC;
  // sums over the columns (the norm, A) are made of slabs of 128 columns, then of pairs of slabs, whatever W is: a
  // matrix's update does not depend on how many CTAs share it
  constexpr int HB = W == 256 ? 2 : 1, HW = W / HB;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* xs = smem;                                                   // hi of X: W / 64 blocks
  uint8_t* ab = smem + 4 * SM_BLK;                                      // A, then B, without diagonals
  float* part = reinterpret_cast<float*>(ab + 2 * SM_BLK);              // [128, SM_PITCH]
  float* s_da = part + 128 * SM_PITCH;                                  // [128] A's diagonal times NS_S
  float* s_db = s_da + 128;                                             // [128] B's diagonal
  float* s_sum = s_db + 128;                                            // [32][4] sums of squares by slab
  float(*s_red)[16] = reinterpret_cast<float(*)[16]>(s_sum + 128);      // [3 HB][16]
  float* s_f = s_sum + 128 + 96;                                        // f1, f2, rho
  uint64_t* bar = reinterpret_cast<uint64_t*>(s_f + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t cs, rank;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(cs));
  rank = cluster_ctarank();
  const int mat = blockIdx.x / cs;
  const int i = (warp & 3) * 32 + lane;      // row of the m x n matrix
  const int j0 = (warp >> 2) * WC;           // first column in the slab
  const bool tall = p.tall != 0;
  uint32_t phase = 0;

  if (threadIdx.x == 0) {
    mbar_init(bar, 1);
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc<512>(tmem_slot);
    tmem_relinquish();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // what is before this launch on the stream
  if (blockIdx.x == 0 && threadIdx.x == 0) p.status[0] = 0;
  // gradient and momentum -> U: read in the matrix's own order, 8 values a
  // thread, and turned to this thread's row of columns through shared memory
  float x[WC];
  float f[HB][3];
  {
    constexpr int PITCH = W + 4;
    float* stage = reinterpret_cast<float*>(smem);  // [128][PITCH], before X and A are there
    const PrepParams& in = p.in;
    float* mom = in.momentum ? in.momentum + (size_t)mat * in.R * in.C : nullptr;
    const int s0 = (int)rank * W;  // the first column
    if (p.m < 128 || p.n - s0 < W) {
      for (int u = threadIdx.x; u < 128 * PITCH / 4; u += SM_THREADS) reinterpret_cast<float4*>(stage)[u] = make_float4(0, 0, 0, 0);
      __syncthreads();
    }
    const bool vec = p.vec != 0;
    constexpr int U = 4;  // units of a thread in flight
#pragma unroll
    for (int h = 0; h < HB; ++h) {
    f[h][0] = f[h][1] = f[h][2] = 0.0f;
    const int first = s0 + h * HW, width = min(HW, p.n - first);                     // the slab
    const int lead = tall ? width : p.m, cols = tall ? p.m : width;                  // rows of the stored matrix, columns
    const int r_at = tall ? first : 0, c_at = tall ? 0 : first;
    const int per = cols > 0 ? (cols + 7) / 8 : 0, units = lead > 0 ? lead * per : 0;
    for (int u0 = threadIdx.x; u0 < units; u0 += U * SM_THREADS) {
      float g[U][8], m[U][8];
#pragma unroll
      for (int q = 0; q < U; ++q) {
        const int u = u0 + q * SM_THREADS;
        if (u < units) {
          const int r = u / per, c = (u - r * per) * 8;
          const size_t gi = (size_t)mat * in.gms + (size_t)(r_at + r) * in.grs + c_at + c;
          const float* mi = mom + (size_t)(r_at + r) * in.C + c_at + c;
          if (vec) {
            load_grad<8>(in.grad, in.dtype, gi, g[q]);
            if (mom) load_f32<8>(mi, m[q]);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              float v[1] = {0.0f};
              if (c + j < cols) load_grad<1>(in.grad, in.dtype, gi + j, v);
              g[q][j] = v[0];
              m[q][j] = mom && c + j < cols ? mi[j] : 0.0f;
            }
          }
        }
      }
#pragma unroll
      for (int q = 0; q < U; ++q) {
        const int u = u0 + q * SM_THREADS;
        if (u < units) {
          const int r = u / per, c = (u - r * per) * 8;
          if (mom) {
            float* mi = mom + (size_t)(r_at + r) * in.C + c_at + c;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              m[q][j] = in.mu * m[q][j] + g[q][j];
              g[q][j] = in.nesterov ? g[q][j] + in.mu * m[q][j] : m[q][j];
            }
            if (vec) {
              reinterpret_cast<float4*>(mi)[0] = make_float4(m[q][0], m[q][1], m[q][2], m[q][3]);
              reinterpret_cast<float4*>(mi)[1] = make_float4(m[q][4], m[q][5], m[q][6], m[q][7]);
            } else {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                if (c + j < cols) mi[j] = m[q][j];
            }
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (c + j >= cols) break;
            add_square(f[h], g[q][j]);
            stage[tall ? (c + j) * PITCH + h * HW + r : r * PITCH + h * HW + c + j] = g[q][j];
          }
        }
      }
    }
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < WC; c += 4) {
      const float4 v = *reinterpret_cast<const float4*>(stage + i * PITCH + j0 + c);
      x[c] = v.x, x[c + 1] = v.y, x[c + 2] = v.z, x[c + 3] = v.w;
    }
  }
#pragma unroll
  for (int h = 0; h < HB; ++h)
#pragma unroll
    for (int q = 0; q < 3; ++q) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) f[h][q] += __shfl_xor_sync(0xffffffffu, f[h][q], o);
      if (lane == 0) s_red[3 * h + q][warp] = f[h][q];
    }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // every CTA runs: its shared memory may be written
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (threadIdx.x < 3 * HB * cs) {  // this CTA's sums, to every CTA
    const uint32_t q = threadIdx.x % (3 * HB), to = threadIdx.x / (3 * HB);
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; ++w) v += s_red[q][w];
    st_shared_cluster_u32(mapa_shared(s_sum + (rank * HB + q / 3) * 4 + q % 3, to), __float_as_uint(v));
  }
  __syncwarp();
  cluster_sync_all();
  if (threadIdx.x == 0) {
    float v[3] = {0.0f, 0.0f, 0.0f};
    for (uint32_t r = 0; r < cs * HB; ++r)
#pragma unroll
      for (int q = 0; q < 3; ++q) v[q] += s_sum[r * 4 + q];
    norm_scale(v, &s_f[0], &s_f[1], &s_f[2]);
  }
  __syncthreads();
  const float f1 = s_f[0], f2 = s_f[1], rho = s_f[2];
  auto put_hi = [&]() {  // X's hi part as operand
#pragma unroll
    for (int c = 0; c < WC; c += 8) {
      *reinterpret_cast<uint4*>(xs + sw_at(i, j0 + c)) =
          make_uint4(pack_half2(x[c], x[c + 1]), pack_half2(x[c + 2], x[c + 3]), pack_half2(x[c + 4], x[c + 5]),
                     pack_half2(x[c + 6], x[c + 7]));
    }
  };
#pragma unroll
  for (int c = 0; c < WC; ++c) x[c] = x[c] * f1 * f2;
  put_hi();

  const uint32_t xa = smem_u32(xs), aa = smem_u32(ab);
  const uint32_t row_tmem = tmem + ((uint32_t)((warp & 3) * 32) << 16);
  const int c32 = (warp >> 2) * 32;  // this thread's columns of A and B: c32 .. c32 + 31
  // what all threads wrote is the tensor core's to read; then the products, then everyone
  auto products = [&](auto issue) {
    fence_proxy_async_all();
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0) {
      tc_fence_after();
      fence_proxy_async_all();
      issue();
      mma_commit(bar);
    }
    __syncwarp();
    // (on a time limit the status says so and the barriers below go on; the
    // status word is not read here: another CTA may not have cleared it yet)
    if (!mbar_wait_drain(bar, phase, p.timeout_ns)) raise_status(p.status, STATUS_TIMEOUT);
    phase ^= 1u;
    __syncwarp();
    tc_fence_after();
  };
  constexpr uint32_t ID = (1u << 4) | (8u << 24);  // fp16 x fp16 -> fp32, M = 128
  for (int s = 0; s < p.steps; ++s) {
    const bool first = s == 0, last = s == p.steps - 1;
    // A = X X^T: this CTA's columns' part
    products([&]() {
      for (int k = 0; k < W; k += 16) {
        const uint64_t d = sdesc_kmajor_sw128(xa + (uint32_t)((k >> 6) * SM_BLK + (k & 63) * 2));
        mma_bf16_ss(tmem + (uint32_t)(k / HW) * 128u, d, d, ID | ((uint32_t)(p.mp >> 3) << 17), k % HW != 0 ? 1u : 0u);
      }
    });
    const float fa = first ? rho * rho * NS_S : 1.0f / NS_S;
    // one row of 8 columns of A: the diagonal apart, the rest as operand
    auto put_a = [&](int r, int c, float (&v)[8]) {
      float d = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] *= fa;
        d = c + j == r ? v[j] : d;
        v[j] = c + j == r ? 0.0f : v[j];
      }
      *reinterpret_cast<uint4*>(ab + sw_at(r, c)) =
          make_uint4(pack_half2(v[0], v[1]), pack_half2(v[2], v[3]), pack_half2(v[4], v[5]), pack_half2(v[6], v[7]));
      if ((r & ~7) == c) s_da[r] = d;
    };
    if (c32 < p.mp) {
      uint32_t acc[32];
      tmem_ld_32x32b_x32(row_tmem + (uint32_t)c32, acc);
      tmem_ld_wait();
      if (HB == 2) {
        uint32_t more[32];
        tmem_ld_32x32b_x32(row_tmem + 128u + (uint32_t)c32, more);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 32; ++c) acc[c] = __float_as_uint(__uint_as_float(acc[c]) + __uint_as_float(more[c]));
      }
#pragma unroll
      for (int c = 0; c < 32; c += 8) {
        if (c32 + c >= p.mp) break;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(acc[c + j]);
        if (cs == 1) {
          put_a(i, c32 + c, v);
        } else if (i < p.mp) {
          float4* d = reinterpret_cast<float4*>(part + i * SM_PITCH + c32 + c);
          d[0] = make_float4(v[0], v[1], v[2], v[3]);
          d[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
      }
    }
    if (cs > 1) {
      __syncwarp();
      cluster_sync_all();
      // 4 columns a thread, consecutive threads side by side (no bank conflicts), CTA r the r-th share
      const int per_row = p.mp / 4, share = (p.mp * per_row + (int)cs - 1) / (int)cs;
      const int u_to = min(p.mp * per_row, ((int)rank + 1) * share);
      for (int u = (int)rank * share + (int)threadIdx.x; u < u_to; u += SM_THREADS) {
        const int r = u / per_row, c = (u - r * per_row) * 4;
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
        for (uint32_t q = 0; q < cs; q += 3 - HB) {  // in the CTAs' order, whoever sums
          float4 w = ld_cluster_f4(mapa_shared(part + r * SM_PITCH + c, q));
          if (HB == 1) {  // (clusters are even)
            const float4 w1 = ld_cluster_f4(mapa_shared(part + r * SM_PITCH + c, q + 1));
            w.x += w1.x, w.y += w1.y, w.z += w1.z, w.w += w1.w;
          }
          v[0] += w.x, v[1] += w.y, v[2] += w.z, v[3] += w.w;
        }
        float d = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[j] *= fa;
          d = c + j == r ? v[j] : d;
          v[j] = c + j == r ? 0.0f : v[j];
        }
        const uint32_t h0 = pack_half2(v[0], v[1]), h1 = pack_half2(v[2], v[3]);
        for (uint32_t q = 0; q < cs; ++q) {
          st_cluster_u2(mapa_shared(ab + sw_at(r, c), q), h0, h1);
          if ((r & ~3) == c) st_shared_cluster_u32(mapa_shared(s_da + r, q), __float_as_uint(d));
        }
      }
      fence_proxy_async_all();
      __syncwarp();
      cluster_sync_all();
    }
    // B = b A + c A^2, with A = D + O: A^2 = O^2 + D O + O D + D^2
    products([&]() {
      for (int k = 0; k < p.mp; k += 16) {
        const uint64_t d = sdesc_kmajor_sw128(aa + (uint32_t)((k >> 6) * SM_BLK + (k & 63) * 2));
        mma_bf16_ss(tmem + 128u, d, d, ID | ((uint32_t)(p.mp >> 3) << 17), k != 0 ? 1u : 0u);
      }
    });
    if (c32 < p.mp) {
      uint32_t acc[32];
      tmem_ld_32x32b_x32(row_tmem + 128u + (uint32_t)c32, acc);
      tmem_ld_wait();
      const float di = s_da[i], cb = p.c / NS_S;
#pragma unroll
      for (int c = 0; c < 32; c += 8) {
        if (c32 + c >= p.mp || i >= p.mp) break;
        uint4* at = reinterpret_cast<uint4*>(ab + sw_at(i, c32 + c));
        float o[8];
        unpack8(*at, o);
        float on = 0.0f, v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float w = __uint_as_float(acc[c + j]);
          const bool diag = c32 + c + j == i;
          on = diag ? w : on;
          v[j] = diag ? 0.0f : o[j] * (p.b + cb * (di + s_da[c32 + c + j])) + cb * w;
        }
        if ((i & ~7) == c32 + c) s_db[i] = (p.b * di + cb * (on + di * di)) / NS_S;
        *at = make_uint4(pack_half2(v[0], v[1]), pack_half2(v[2], v[3]), pack_half2(v[4], v[5]), pack_half2(v[6], v[7]));
      }
    }
    // X <- a X + B X
    products([&]() {
      for (int k = 0; k < p.mp; k += 16)
        mma_bf16_ss(tmem + 256u, sdesc_kmajor_sw128(aa + (uint32_t)((k >> 6) * SM_BLK + (k & 63) * 2)),
                    sdesc_mn_blocks(xa + (uint32_t)k * 128u), ID | (1u << 16) | ((uint32_t)(W >> 3) << 17), k != 0 ? 1u : 0u);
    });
    const float db = i < p.mp ? s_db[i] : 0.0f, fx = first ? NS_S * rho : 1.0f, cb = first ? rho : 1.0f / NS_S;
    const bool diag_full = s >= p.steps - 2;
#pragma unroll
    for (int c = 0; c < WC; c += 16) {
      uint32_t acc[16];
      tmem_ld_32x32b_x16(row_tmem + 256u + (uint32_t)(j0 + c), acc);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float v = x[c + j], y = diag_full ? v : __half2float(__float2half_rn(v));
        x[c + j] = fx * (p.a * v + db * y) + cb * __uint_as_float(acc[j]);
      }
    }
    if (!last) put_hi();
  }

  // the update, through shared memory into the matrix's own order: this CTA's
  // part is `lead` rows of `cols` values, rows `pitch` apart in the matrix
  {
    const int s0 = (int)rank * W, width = min(W, p.n - s0);
    const int lead = tall ? width : p.m, cols = tall ? p.m : width, pitch = tall ? p.m : p.n;
    bf16* out = p.out + (size_t)mat * p.m * p.n + (tall ? (size_t)s0 * p.m : (size_t)s0);
    constexpr int SP = (W > 128 ? W : 128) + 8;  // elements between rows in shared memory
    bf16* stage = reinterpret_cast<bf16*>(smem);
#pragma unroll
    for (int c = 0; c < WC; c += 8) {
      if (tall) {
#pragma unroll
        for (int j = 0; j < 8; ++j) stage[(j0 + c + j) * SP + i] = __float2bfloat16_rn(x[c + j] * p.scale);
      } else {
        *reinterpret_cast<uint4*>(stage + i * SP + j0 + c) =
            make_uint4(pack_bf16x2(x[c] * p.scale, x[c + 1] * p.scale), pack_bf16x2(x[c + 2] * p.scale, x[c + 3] * p.scale),
                       pack_bf16x2(x[c + 4] * p.scale, x[c + 5] * p.scale), pack_bf16x2(x[c + 6] * p.scale, x[c + 7] * p.scale));
      }
    }
    __syncthreads();
    if (cols % 8 == 0 && pitch % 8 == 0 && (reinterpret_cast<uintptr_t>(p.out) & 15u) == 0) {
      const int per = cols / 8;
      for (int u = threadIdx.x; u < lead * per; u += SM_THREADS) {
        const int r = u / per, c = (u - r * per) * 8;
        *reinterpret_cast<uint4*>(out + (size_t)r * pitch + c) = *reinterpret_cast<const uint4*>(stage + r * SP + c);
      }
    } else {
      for (int u = threadIdx.x; u < lead * cols; u += SM_THREADS) {
        const int r = u / cols, c = u - r * cols;
        out[(size_t)r * pitch + c] = stage[r * SP + c];
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  __syncwarp();
  cluster_sync_all();  // no CTA leaves while another may still read its shared memory
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace moe

// ------------------------------------------------------------------ C ABI
using namespace moe;

struct moe_muon_plan {
  moe_muon_config cfg;
  int device, num_sms;
  int64_t chunk;  // matrices in flight
  int small_cs, small_wc;  // the one-launch form: CTAs per matrix (0: not used) and columns per thread
  encode_tiled_fn encode;
};

namespace {

// Whether every iterate, A and B stay in range: held as fp16 times 4096, they
// must not reach 16.  A singular value of X is at most 1 at the start and goes
// through s -> a s + b s^3 + c s^5 each step; an element of X is at most the
// largest, one of A or B beside the diagonal (which is kept in fp32) half of the
// spread of the eigenvalues.  1% a step for the products' own errors, and 15 of 16.
bool ns_in_range(const moe_muon_config& cfg) {
  const double a = cfg.a, b = cfg.b, c = cfg.c, most = 15.0;
  double S = 1.01;  // bound of the singular values
  for (int i = 0; i < cfg.steps; ++i) {
    const double t = S * S;  // of A's eigenvalues, 0 .. t
    auto poly = [&](double u) { return u * (b + c * u); };  // of B's
    const double turn = c != 0.0 ? -b / (2.0 * c) : -1.0, inner = turn > 0.0 && turn < t ? poly(turn) : 0.0;
    const double hi = fmax(fmax(0.0, poly(t)), inner), lo = fmin(fmin(0.0, poly(t)), inner);
    if (!(t <= 2.0 * most) || !(hi - lo <= 2.0 * most)) return false;
    // |s (a + b u + c u^2)|, u = s^2: at the end, or where a + 3 b u + 5 c u^2 = 0
    auto at = [&](double u) { return u > 0.0 && u < t ? fabs(sqrt(u) * (a + u * (b + c * u))) : 0.0; };
    double next = fabs(S * (a + t * (b + c * t)));
    if (c != 0.0) {
      const double d = 9.0 * b * b - 20.0 * a * c;
      if (d >= 0.0) next = fmax(next, fmax(at((-3.0 * b + sqrt(d)) / (10.0 * c)), at((-3.0 * b - sqrt(d)) / (10.0 * c))));
    } else if (b != 0.0) {
      next = fmax(next, at(-a / (3.0 * b)));
    }
    S = 1.01 * next;
    if (i + 1 < cfg.steps && !(S <= most)) return false;  // (the last one is the update, in bf16)
  }
  return true;
}

int64_t up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }
bool ns_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct NsLayout {
  size_t rho, part, hi[2], lo[2], a, b, da, db, total;
  int64_t m, n, ldx, lda, ldd;
};

NsLayout ns_layout(const moe_muon_plan* pl) {
  const moe_muon_config& c = pl->cfg;
  NsLayout L{};
  if (pl->small_cs) {  // on chip but for the status word
    L.total = 256;
    return L;
  }
  L.m = c.rows < c.cols ? c.rows : c.cols;
  L.n = c.rows < c.cols ? c.cols : c.rows;
  L.ldx = up(c.cols, 8);
  L.lda = up(L.m, 8);
  L.ldd = up(L.m, NS_TILE);  // the epilogue reads whole tiles' diagonals
  size_t off = 256;  // status word
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = (size_t)up((int64_t)(off + bytes), 256);
    return at;
  };
  L.rho = take(sizeof(float) * pl->chunk);
  L.part = take(sizeof(float) * 4 * NS_PREP_BLOCKS * pl->chunk);
  for (int i = 0; i < 2; ++i) {
    L.hi[i] = take(sizeof(__half) * pl->chunk * c.rows * L.ldx);
    L.lo[i] = take(sizeof(__half) * pl->chunk * c.rows * L.ldx);
  }
  L.a = take(sizeof(__half) * pl->chunk * L.m * L.lda);
  L.b = take(sizeof(__half) * pl->chunk * L.m * L.lda);
  L.da = take(sizeof(float) * pl->chunk * L.ldd);
  L.db = take(sizeof(float) * pl->chunk * L.ldd);
  L.total = off;
  return L;
}

// [nb, rows, cols] of 16-bit elements, rows ld apart; box {64, box_rows, 1}; elements outside a matrix read as zero
int ns_encode(const moe_muon_plan* pl, CUtensorMap* m, const void* ptr, int64_t nb, int64_t rows, int64_t cols, int64_t ld,
              uint32_t box_rows, CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_FLOAT16) {
  cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)nb};
  cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)(ld * rows) * 2};
  cuuint32_t box[3] = {64, box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = pl->encode(m, type, 3, const_cast<void*>(ptr), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MOE_OK : MOE_ERR_INVALID_ARG;
}

// Launch; the grid may be set up while the launch before it on the stream still
// runs (the kernels wait for that one's results themselves)
template <typename P, typename... A>
cudaError_t launch_after(void (*kernel)(P, A...), dim3 grid, int threads, size_t smem, cudaStream_t st,
                         const std::remove_const_t<P>& p, const std::remove_const_t<A>&... a) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = grid;
  lc.blockDim = dim3((unsigned)threads);
  lc.dynamicSmemBytes = smem;
  lc.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = at;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, kernel, p, a...);
}

// The one-launch form's shape for a plan, if it applies: m <= 128 and up to 16
// CTAs of at most 256 columns.
using SmallKernel = void (*)(SmallParams);
SmallKernel small_kernel(int wc) { return wc == 16 ? ns_small<16> : wc == 32 ? ns_small<32> : ns_small<64>; }
cudaLaunchConfig_t small_launch(const moe_muon_plan* pl, cudaLaunchAttribute (&at)[2], cudaStream_t st) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)(pl->cfg.count * pl->small_cs));
  lc.blockDim = dim3(SM_THREADS);
  lc.dynamicSmemBytes = SM_BYTES;
  lc.stream = st;
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)pl->small_cs;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = at;
  lc.numAttrs = 2;
  return lc;
}
int small_prepare(moe_muon_plan* pl) {
  const moe_muon_config& c = pl->cfg;
  const int64_t m = c.rows < c.cols ? c.rows : c.cols, n = c.rows < c.cols ? c.cols : c.rows;
  pl->small_cs = pl->small_wc = 0;
  if (m > 128 || n > 16 * 256) return MOE_OK;
  int wc = 64, cs = 1;
  while (cs * 256 < n) cs *= 2;
  while (wc > 16 && (int64_t)cs * 2 * wc >= n) wc /= 2;  // (as narrow as the columns are)
  // Twice the CTAs with half the columns each, where all of them still run at
  // once: less work per CTA for the same exchanges (2 x 128 x 1024: 4 CTAs 64
  // us, 8 54 us; 8 x 100 x 600: 60 and 50 us).  A CTA that needs no exchange
  // stays alone (16 x 128 x 256: 47.5 us, two CTAs 48.8 us).  Both give the same bits.
  if (cs > 1 && cs < 8 && wc == 64 && c.count * cs * 2 <= pl->num_sms) cs *= 2, wc = 32;
  pl->small_cs = cs;
  pl->small_wc = wc;
  const SmallKernel k = small_kernel(wc);
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SM_BYTES) != cudaSuccess ||
      cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
    return MOE_ERR_CUDA;
  cudaLaunchAttribute at[2];
  const cudaLaunchConfig_t lc = small_launch(pl, at, nullptr);
  int fit = 0;
  if (cudaOccupancyMaxActiveClusters(&fit, k, &lc) != cudaSuccess) return MOE_ERR_CUDA;
  // Few clusters of 16 run at once (SMs of one GPC), so with many matrices the
  // general form catches up and passes it (n x 117 x 3051: 9 matrices 151 us and
  // 205 us, 40 449 and 477, 80 1011 and 943).  The form goes by the matrices' size alone
  // all the same, so that a matrix's update does not depend on the others.
  if (fit < 1) pl->small_cs = 0;
  return MOE_OK;
}

template <int KIND, bool A_MN, bool B_MN>
bool ns_prepare() {
  return cudaFuncSetAttribute(ns_gemm<KIND, A_MN, B_MN>, cudaFuncAttributeMaxDynamicSharedMemorySize, NS_SMEM) == cudaSuccess;
}
// One product of every matrix, M and N of one given.  Every CTA pair takes
// whole tiles, round by round; tiles that would fill less than half of a last
// round are halved for it, a half taking about 0.6 of a tile's time (2 x 700 x
// 650, all of them halves: 189 us, whole 259 us; 8 x 1024 x 4096, whose A has 80
// tiles for 76 pairs: 748 us, two whole rounds 777 us).
template <int KIND, bool A_MN, bool B_MN>
cudaError_t ns_launch(const moe_muon_plan* pl, const NsMaps& mp, NsParams p, cudaStream_t st) {
  const int64_t pairs = pl->num_sms / 2, mt = up(p.M, NS_TILE) / NS_TILE;
  p.tiles_n = (int)(up(p.N, NS_TILE) / NS_TILE);
  p.n_tiles = (int)(KIND == NS_STEP ? mt * p.tiles_n : mt * (mt + 1) / 2);
  const int64_t tiles = (int64_t)p.nb * p.n_tiles, rest = tiles % pairs;
  p.n_wide = (int)(2 * rest <= pairs ? tiles - rest : tiles);
  p.n_units = (int)(p.n_wide + 2 * (tiles - p.n_wide));
  const int64_t grid = p.n_units < pairs ? p.n_units : pairs;
  return launch_after(ns_gemm<KIND, A_MN, B_MN>, dim3((unsigned)(2 * grid)), NS_THREADS, NS_SMEM, st, mp, p);
}

}  // namespace

extern "C" {

int moe_muon_plan_create(const moe_muon_config* cfg, moe_muon_plan** out) {
  if (!cfg || !out) return MOE_ERR_INVALID_ARG;
  *out = nullptr;
  moe_muon_config c = *cfg;
  if (c.steps == 0) c.steps = 5;
  if (c.timeout_ms <= 0) c.timeout_ms = 2000;
  if (c.a == 0.0f && c.b == 0.0f && c.c == 0.0f) c.a = 3.4445f, c.b = -4.7750f, c.c = 2.0315f;
  if (c.grad_dtype < MOE_DTYPE_FP32 || c.grad_dtype > MOE_DTYPE_FP16 || c.steps < 1 || c.steps > 32) return MOE_ERR_INVALID_ARG;
  if (!(c.a - c.a == 0.0f) || !(c.b - c.b == 0.0f) || !(c.c - c.c == 0.0f)) return MOE_ERR_INVALID_ARG;  // finite
  if (!ns_in_range(c)) return MOE_ERR_INVALID_ARG;
  if (c.count < 1 || c.count > 65536 || c.rows < 1 || c.rows > 65536 || c.cols < 1 || c.cols > 65536 ||
      c.rows * c.cols > (int64_t)1 << 30)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  int dev = 0, sms = 0, major = 0, minor = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
    return MOE_ERR_CUDA;
  if (major != 10 || minor != 3) return MOE_ERR_UNSUPPORTED_DEVICE;
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess || !fn)
    return MOE_ERR_CUDA;
  if (!ns_prepare<NS_GRAM, false, false>() || !ns_prepare<NS_GRAM, true, true>() || !ns_prepare<NS_POLY, false, false>() ||
      !ns_prepare<NS_STEP, false, false>() || !ns_prepare<NS_STEP, false, true>())
    return MOE_ERR_CUDA;
  moe_muon_plan* pl = new (std::nothrow) moe_muon_plan;
  if (!pl) return MOE_ERR_INVALID_ARG;
  pl->cfg = c;
  pl->device = dev;
  pl->num_sms = sms;
  pl->encode = reinterpret_cast<encode_tiled_fn>(fn);
  // matrices in flight: the smallest product (A, half of m / 256 squared tiles)
  // fills the CTA pairs eight times over, so its last, part-filled round costs
  // little, and the workspace does not grow with the stack
  const int64_t mt = up(c.rows < c.cols ? c.rows : c.cols, NS_TILE) / NS_TILE, tiles = mt * (mt + 1) / 2;
  const int64_t want = (8 * (int64_t)(sms / 2) + tiles - 1) / tiles;
  pl->chunk = want < c.count ? want : c.count;
  const int rc = small_prepare(pl);
  if (rc != MOE_OK) {
    delete pl;
    return rc;
  }
  *out = pl;
  return MOE_OK;
}

int moe_muon_plan_destroy(moe_muon_plan* plan) {
  delete plan;
  return MOE_OK;
}

size_t moe_muon_workspace_bytes(const moe_muon_plan* plan) { return plan ? ns_layout(plan).total : 0; }

int moe_muon_update(const moe_muon_plan* pl, const void* grad, int64_t grad_row_stride, int64_t grad_stride,
                    float* momentum, float mu, int32_t nesterov, float scale, void* update, void* workspace,
                    size_t workspace_bytes, moe_stream_t stream_) {
  if (!pl || !grad || !update || !workspace) return MOE_ERR_INVALID_ARG;
  const moe_muon_config& c = pl->cfg;
  const size_t gsize = c.grad_dtype == MOE_DTYPE_FP32 ? 4 : 2;
  if (grad_row_stride == 0) grad_row_stride = c.cols;
  if (grad_stride == 0) grad_stride = c.rows * grad_row_stride;
  if (grad_row_stride < c.cols || grad_row_stride > (int64_t)1 << 31 || grad_stride < 0 || grad_stride > (int64_t)1 << 40)
    return MOE_ERR_INVALID_ARG;
  if (!ns_aligned(grad, gsize) || !ns_aligned(momentum, 4) || !ns_aligned(update, 2) || !ns_aligned(workspace, 256))
    return MOE_ERR_INVALID_ARG;
  if (!(mu - mu == 0.0f) || !(scale - scale == 0.0f) || (nesterov != 0 && nesterov != 1)) return MOE_ERR_INVALID_ARG;
  const NsLayout L = ns_layout(pl);
  if (workspace_bytes < L.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  int cur = -1;
  if (cudaGetDevice(&cur) != cudaSuccess || cur != pl->device) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream_;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const bool tall = c.rows > c.cols;
  PrepParams pp{};
  pp.grad = grad;
  pp.grs = grad_row_stride;
  pp.gms = grad_stride;
  pp.dtype = c.grad_dtype;
  pp.R = (int)c.rows;
  pp.C = (int)c.cols;
  pp.nesterov = nesterov;
  pp.mu = mu;
  pp.momentum = momentum;
  if (pl->small_cs) {
    SmallParams sp{};
    sp.in = pp;
    sp.out = static_cast<bf16*>(update);
    sp.steps = c.steps;
    sp.tall = tall;
    sp.m = (int)(tall ? c.cols : c.rows);
    sp.n = (int)(tall ? c.rows : c.cols);
    sp.mp = (int)up(sp.m, 16);
    sp.vec = c.cols % 8 == 0 && grad_row_stride % 8 == 0 && grad_stride % 8 == 0 && ns_aligned(grad, 16) && ns_aligned(momentum, 16);
    sp.a = c.a;
    sp.b = c.b;
    sp.c = c.c;
    sp.scale = scale / NS_S;
    sp.status = reinterpret_cast<int*>(ws);
    sp.timeout_ns = (long long)c.timeout_ms * 1000000LL;
    cudaLaunchAttribute at[2];
    const cudaLaunchConfig_t lc = small_launch(pl, at, st);
    return cudaLaunchKernelEx(&lc, small_kernel(pl->small_wc), sp) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  }
  auto half_at = [&](size_t o) { return reinterpret_cast<__half*>(ws + o); };

  // K-major operands and the epilogue's tiles are 128 rows at a time, MN-major
  // operands and transposed tiles {64, 64} boxes
  CUtensorMap xk[2], xm[2], xl[2], ak, am, bk, bm, uk;
  int rc = MOE_OK;
  for (int i = 0; i < 2; ++i) {
    rc |= ns_encode(pl, &xk[i], half_at(L.hi[i]), pl->chunk, c.rows, c.cols, L.ldx, 128);
    rc |= ns_encode(pl, &xm[i], half_at(L.hi[i]), pl->chunk, c.rows, c.cols, L.ldx, 64);
    rc |= ns_encode(pl, &xl[i], half_at(L.lo[i]), pl->chunk, c.rows, c.cols, L.ldx, 128);
  }
  rc |= ns_encode(pl, &ak, half_at(L.a), pl->chunk, L.m, L.m, L.lda, 128);
  rc |= ns_encode(pl, &am, half_at(L.a), pl->chunk, L.m, L.m, L.lda, 64);
  rc |= ns_encode(pl, &bk, half_at(L.b), pl->chunk, L.m, L.m, L.lda, 128);
  rc |= ns_encode(pl, &bm, half_at(L.b), pl->chunk, L.m, L.m, L.lda, 64);
  if (rc != MOE_OK) return MOE_ERR_INVALID_ARG;

  pp.ld = L.ldx;
  pp.part = reinterpret_cast<float*>(ws + L.part);
  pp.rho = reinterpret_cast<float*>(ws + L.rho);
  pp.hi = half_at(L.hi[0]);
  pp.lo = half_at(L.lo[0]);
  const bool vec = c.cols % 8 == 0 && grad_row_stride % 8 == 0 && grad_stride % 8 == 0 && ns_aligned(grad, 16) &&
                   ns_aligned(momentum, 16);
  const int64_t per = 256 * prep_unroll(vec ? 8 : 1), nblk = up(c.rows * c.cols / (vec ? 8 : 1), per) / per;
  // blocks per matrix: 256, more where few matrices would leave SMs idle (1 x
  // 1500 x 2500: 337 us with 256, 319 with 1024; 8 x 1024 x 4096: 836 and 859 us)
  int64_t most = 8 * (int64_t)pl->num_sms / pl->chunk;
  most = most < 256 ? 256 : most < NS_PREP_BLOCKS ? most : NS_PREP_BLOCKS;
  pp.nblk = (int)(nblk < most ? nblk : most);

  NsParams g{};
  g.rho = pp.rho;
  g.status = reinterpret_cast<int*>(ws);
  g.timeout_ns = (long long)c.timeout_ms * 1000000LL;
  g.scale = scale / NS_S;
  g.tall = tall;
  g.ldd = (int)L.ldd;
  g.diag_a = reinterpret_cast<float*>(ws + L.da);
  g.diag_b = reinterpret_cast<float*>(ws + L.db);
  for (int64_t c0 = 0; c0 < c.count; c0 += pl->chunk) {
    const int nb = (int)(c.count - c0 < pl->chunk ? c.count - c0 : pl->chunk);
    pp.grad = static_cast<const uint8_t*>(grad) + (size_t)c0 * grad_stride * gsize;
    pp.status = c0 == 0 ? g.status : nullptr;
    pp.momentum = momentum ? momentum + (size_t)c0 * c.rows * c.cols : nullptr;
    bf16* out = static_cast<bf16*>(update) + (size_t)c0 * c.rows * c.cols;
    const dim3 pgrid((unsigned)pp.nblk, (unsigned)nb);
    if (launch_after(vec ? ns_prep_norm<8> : ns_prep_norm<1>, pgrid, 256, 0, st, pp) != cudaSuccess ||
        launch_after(vec ? ns_prep_first<8> : ns_prep_first<1>, pgrid, 256, 0, st, pp) != cudaSuccess)
      return MOE_ERR_CUDA;
    g.nb = nb;
    g.out_final = out;
    g.out_vec = c.cols % 8 == 0 && ns_aligned(out, 16);
    uk = xk[0];
    if (g.out_vec && ns_encode(pl, &uk, out, nb, c.rows, c.cols, c.cols, 128, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16) != MOE_OK)
      return MOE_ERR_INVALID_ARG;
    for (int s = 0; s < c.steps; ++s) {
      const int x = s & 1;
      cudaError_t err;
      g.first = s == 0;
      g.last = s == c.steps - 1;
      g.diag_full = s >= c.steps - 2;
      // A = X X^T or X^T X
      g.M = g.N = (int)L.m;
      g.K = (int)L.n;
      const CUtensorMap& xx = tall ? xm[x] : xk[x];
      const NsMaps gram = {xx, xx, xm[x], ak, ak, ak, am};
      err = tall ? ns_launch<NS_GRAM, true, true>(pl, gram, g, st) : ns_launch<NS_GRAM, false, false>(pl, gram, g, st);
      if (err != cudaSuccess) return MOE_ERR_CUDA;
      // B = b A + c A^2
      g.K = (int)L.m;
      g.ca = c.b;
      g.cb = c.c / NS_S;
      const NsMaps poly = {ak, ak, am, ak, ak, bk, bm};
      if (ns_launch<NS_POLY, false, false>(pl, poly, g, st) != cudaSuccess) return MOE_ERR_CUDA;
      // X <- a X + B X or a X + X B
      g.M = (int)c.rows;
      g.N = (int)c.cols;
      g.ca = c.a;
      g.cb = 1.0f / NS_S;
      const NsMaps step = {tall ? xk[x] : bk, tall ? bk : xm[x], tall ? bm : xm[x], xk[x], xl[x], g.last ? uk : xk[x ^ 1], xl[x ^ 1]};
      err = tall ? ns_launch<NS_STEP, false, false>(pl, step, g, st) : ns_launch<NS_STEP, false, true>(pl, step, g, st);
      if (err != cudaSuccess) return MOE_ERR_CUDA;
    }
  }
  return MOE_OK;
}

int moe_muon_get_status(const moe_muon_plan* plan, const void* workspace, int* device_status, moe_stream_t stream) {
  if (!plan || !workspace || !device_status) return MOE_ERR_INVALID_ARG;
  int v = 0;
  if (cudaMemcpyAsync(&v, workspace, sizeof(v), cudaMemcpyDeviceToHost, (cudaStream_t)stream) != cudaSuccess)
    return MOE_ERR_CUDA;
  if (cudaStreamSynchronize((cudaStream_t)stream) != cudaSuccess) return MOE_ERR_CUDA;
  *device_status = v;
  return MOE_OK;
}

}  // extern "C"
