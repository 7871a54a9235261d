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
// over flat, decaying and rank-deficient spectra, 16 to 2048 rows): 2e-4 to
// 1.4e-3, before the result's own rounding to bf16 (1.7e-3).
//
// Scales.  fp16 has 5 exponent bits, so X_0 is U 2^k with |U 2^k|_F in
// [2^14, 2^15): no element overflows and those 2^-28 of the norm keep their
// bits.  Later iterates, A and B are held times 2^12 (|X|_2 < 1.3 for the
// default coefficients, so below 16 on their side too); the factors, and what
// is left of 1 / |U|_F, are applied to the fp32 sums.
#include <cuda_fp16.h>

#include <cstring>
#include <new>

#include "../../include/moe.h"
#include "common.cuh"
#include "plan.cuh"

namespace moe {

constexpr int NS_THREADS = 224;       // producer, MMA issuer, four epilogue warps, the epilogue's loads and stores
constexpr int NS_TILE = 256;          // of a CTA pair: 256 x 256, 128 rows in each CTA
constexpr int NS_BOX = 8192;          // one {64, 64} fp16 box
constexpr int NS_STAGE = 4 * NS_BOX;  // per CTA: 128 rows of A and half of B's 256, 64 of K
constexpr int NS_STAGES = 5;
constexpr int NS_EBUF = 4 * NS_BOX;   // epilogue buffer: two tiles of 128 rows x 64 columns
constexpr int NS_SMEM = NS_STAGES * NS_STAGE + 2 * NS_EBUF + 1024 + 256;
constexpr float NS_S = 4096.0f;       // scale of the held iterates, A and B
constexpr int NS_PREP_BLOCKS = 256;   // partial sums per matrix, at most

enum : int { NS_GRAM = 0, NS_POLY = 1, NS_STEP = 2 };

struct NsMaps {
  CUtensorMap a, b;         // operands
  CUtensorMap in0, in1;     // box {64, 128}: POLY: A; STEP: X's hi and lo
  CUtensorMap out0, out1;   // box {64, 128}: A or B, and (box {64, 64}) its transposed tiles; STEP: hi and lo, or the update
};

struct NsParams {
  int M, N, K;             // of one matrix's product
  int nb;                  // matrices
  int tiles_n, n_tiles;    // column tiles; tiles per matrix (symmetric: the lower ones)
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
constexpr uint32_t ns_idesc(bool a_mn, bool b_mn) {
  return (1u << 4) | ((NS_TILE >> 3) << 17) | ((NS_TILE >> 4) << 24) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u);
}

struct NsTile {
  int mat, m0, n0;
};
template <int KIND>
__device__ __forceinline__ NsTile ns_tile(const NsParams& p, int u) {
  NsTile t;
  t.mat = u / p.n_tiles;
  const int v = u - t.mat * p.n_tiles;
  int i, j;
  if (KIND == NS_STEP) {
    i = v / p.tiles_n;
    j = v - i * p.tiles_n;
  } else {  // lower triangle, row by row
    i = (int)((sqrtf(8.0f * (float)v + 1.0f) - 1.0f) * 0.5f);
    while (i * (i + 1) / 2 > v) --i;
    while ((i + 1) * (i + 2) / 2 <= v) ++i;
    j = v - i * (i + 1) / 2;
  }
  t.m0 = i * NS_TILE;
  t.n0 = j * NS_TILE;
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
__device__ __forceinline__ uint4 pack8(const __half* h) {
  return make_uint4((uint32_t)__half_as_ushort(h[0]) | ((uint32_t)__half_as_ushort(h[1]) << 16),
                    (uint32_t)__half_as_ushort(h[2]) | ((uint32_t)__half_as_ushort(h[3]) << 16),
                    (uint32_t)__half_as_ushort(h[4]) | ((uint32_t)__half_as_ushort(h[5]) << 16),
                    (uint32_t)__half_as_ushort(h[6]) | ((uint32_t)__half_as_ushort(h[7]) << 16));
}

// One row (TMEM lane) of an epilogue chunk, 64 columns: `main` holds this row's
// inputs and takes its outputs in place (POLY: A -> B; STEP: hi), `aux` is lo,
// or takes the chunk transposed (symmetric products' tiles below the
// diagonal).  Rows of 128 bytes, 16-byte pieces swizzled as the tensor maps'.
template <int KIND>
__device__ __forceinline__ void ns_chunk(const NsParams& p, const NsTile& t, uint8_t* main, uint8_t* aux, int rl, int r,
                                         int c0, float rho, uint32_t taddr) {
  uint32_t acc[2][32];
  tmem_ld_32x32b_x32(taddr, acc[0]);
  tmem_ld_32x32b_x32(taddr + 32u, acc[1]);
  tmem_ld_wait();
  const bool mirror = KIND != NS_STEP && t.m0 != t.n0;
  const float* da = p.diag_a + (size_t)t.mat * p.ldd;
  const float* db = p.diag_b + (size_t)t.mat * p.ldd;
  float f = 1.0f, g = 0.0f, cb = p.cb;
  if (KIND == NS_GRAM) f = p.first ? rho * rho * NS_S : 1.0f / NS_S;
  if (KIND == NS_POLY) g = da[r];
  if (KIND == NS_STEP) {
    if (p.first) f = NS_S * rho, cb = rho;
    if (!p.tall) g = db[r];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = c0 + 8 * i;
    uint4* at = reinterpret_cast<uint4*>(main + rl * 128 + ((i ^ (rl & 7)) << 4));
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(acc[i / 4][(8 * i + j) & 31]);
    __half h[8];
    if (KIND == NS_GRAM) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] *= f;
        if (c + j == r) {
          if (r < p.M) p.diag_a[(size_t)t.mat * p.ldd + r] = v[j];
          v[j] = 0.0f;
        }
        h[j] = __float2half_rn(v[j]);
      }
    } else {
      float x[8], d[8];
      unpack8(*at, x);
      if (KIND == NS_POLY || p.tall) {  // the columns' diagonal: the same 32 bytes for the whole warp
        const float4* s4 = reinterpret_cast<const float4*>((KIND == NS_POLY ? da : db) + c);
        const float4 w0 = s4[0], w1 = s4[1];
        d[0] = w0.x, d[1] = w0.y, d[2] = w0.z, d[3] = w0.w, d[4] = w1.x, d[5] = w1.y, d[6] = w1.z, d[7] = w1.w;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = g;
      }
      if (KIND == NS_POLY) {  // b O + c (O^2 + (D_r + D_c) O); on the diagonal b D + c (O^2 + D^2)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (c + j == r) {
            if (r < p.M) p.diag_b[(size_t)t.mat * p.ldd + r] = (p.ca * g + cb * (v[j] + g * g)) / NS_S;
            h[j] = __float2half_rn(0.0f);
          } else {
            h[j] = __float2half_rn(p.ca * x[j] + cb * (v[j] + (g + d[j]) * x[j]));
          }
        }
      } else {
        uint4* al = reinterpret_cast<uint4*>(aux + rl * 128 + ((i ^ (rl & 7)) << 4));
        float lo[8];
        unpack8(*al, lo);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float both = x[j] + lo[j], y = p.diag_full ? both : x[j];
          v[j] = f * (p.ca * both + d[j] * y) + cb * v[j];
        }
        if (p.last) {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] *= p.scale;
          if (p.out_vec) {
            *at = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                             pack_bf16x2(v[6], v[7]));
          } else if (r < p.M) {
            bf16* o = p.out_final + (size_t)t.mat * (size_t)p.M * p.N + (size_t)r * p.N + c;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (c + j < p.N) o[j] = __float2bfloat16_rn(v[j]);
          }
          continue;
        }
        __half l[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          h[j] = __float2half_rn(v[j]);
          l[j] = __float2half_rn(v[j] - __half2float(h[j]));
        }
        *al = pack8(l);
      }
    }
    *at = pack8(h);
    if (mirror) {  // element (r, c) goes to row c, column r; two 64-column boxes
      uint8_t* b = aux + (rl >> 6) * NS_BOX;
      const int rc = rl & 63;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        *reinterpret_cast<__half*>(b + (8 * i + j) * 128 + (((rc >> 3) ^ j) << 4) + (rc & 7) * 2) = h[j];
    }
  }
}

// Persistent CTA pairs, one per SM pair; pair u takes tiles u, u + pairs, ...
// Warp 0: TMA producer of this CTA's operands (counted on the even CTA's full
// barrier); warp 1 of the even CTA: tcgen05.mma for both; warps 2-5: epilogue
// of this CTA's 128 rows, 64 columns at a time; warp 6: loads the epilogue's
// inputs into the two epilogue buffers and stores its outputs from them, both
// by TMA, the loads ahead of the accumulator.  Two 256-column accumulators in
// TMEM alternate, so a tile's epilogue runs under the next tile's products.
// (Rows read and written by the threads themselves, 32 rows of 16 bytes at a
// time, took 30 us a tile of X against 12 us of products.)
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
  const int n_units = p.nb * p.n_tiles;
  const int nk = (p.K + BK - 1) / BK;
  // epilogue chunks of this CTA's part of a tile
  auto chunks = [&](const NsTile& t) { return t.m0 + rank * 128 < p.M ? (min(NS_TILE, p.N - t.n0) + 63) / 64 : 0; };
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS_STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 8);  // one arrival per epilogue warp of both CTAs
      mbar_init(&eload[a], 1);
      mbar_init(&edone[a], 4);   // one per epilogue warp
    }
    mbar_init(drain, 1);
    fence_barrier_init();
    prefetch_tensormap(&mp.a);
    prefetch_tensormap(&mp.b);
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

  if (warp == 0) {
    if (lane == 0) {
      const uint32_t full_even = mapa_shared(full, 0);
      uint32_t stage = 0, phase = 0;
      int issued = 0;
      bool ok = true;
      for (int u = pair; u < n_units && ok; u += pairs) {
        const NsTile t = ns_tile<KIND>(p, u);
        const int ar = t.m0 + rank * 128, br = t.n0 + rank * 128;
        for (int s = 0; s < nk; ++s) {
          if (!mbar_wait_cluster(&empty[stage], phase ^ 1u, p.status, p.timeout_ns)) { ok = false; break; }
          uint8_t* sa = smem + stage * NS_STAGE;
          uint8_t* sb = sa + 2 * NS_BOX;
          if (leader) mbar_arrive_expect_tx(&full[stage], 2u * NS_STAGE);
          const uint32_t fb = full_even + 8u * stage;
          if (A_MN) {
            tma_load_3d_pair(sa, &mp.a, fb, ar, s * BK, t.mat);
            tma_load_3d_pair(sa + NS_BOX, &mp.a, fb, ar + 64, s * BK, t.mat);
          } else {
            tma_load_3d_pair(sa, &mp.a, fb, s * BK, ar, t.mat);
          }
          if (B_MN) {
            tma_load_3d_pair(sb, &mp.b, fb, br, s * BK, t.mat);
            tma_load_3d_pair(sb + NS_BOX, &mp.b, fb, br + 64, s * BK, t.mat);
          } else {
            tma_load_3d_pair(sb, &mp.b, fb, s * BK, br, t.mat);
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
        if (!mbar_wait_cluster(&tempty[acc], (((uint32_t)i >> 1) & 1u) ^ 1u, p.status, p.timeout_ns)) break;
        tc_fence_after();
        const uint32_t d = tmem + acc * 256u;
        for (int s = 0; s < nk; ++s) {
          if (!mbar_wait_cluster(&full[stage], phase, p.status, p.timeout_ns)) { ok = false; break; }
          tc_fence_after();
          const uint32_t a_addr = smem_u32(smem + stage * NS_STAGE);
          const uint32_t b_addr = a_addr + 2 * NS_BOX;
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk) {
            const uint64_t ad = A_MN ? sdesc_mn_sw128(a_addr + kk * 2048) : sdesc_kmajor_sw128(a_addr + kk * 32);
            const uint64_t bd = B_MN ? sdesc_mn_sw128(b_addr + kk * 2048) : sdesc_kmajor_sw128(b_addr + kk * 32);
            mma_bf16_pair(d, ad, bd, ns_idesc(A_MN, B_MN), (s | kk) != 0 ? 1u : 0u);
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
  } else if (warp < 6) {
    const int q = warp & 3, rl = q * 32 + lane;
    const uint32_t tempty_even = mapa_shared(tempty, 0);
    int i = 0, n = 0;
    bool ok = true;
    for (int u = pair; u < n_units && ok; u += pairs, ++i) {
      const NsTile t = ns_tile<KIND>(p, u);
      const uint32_t acc = (uint32_t)i & 1u;
      const int nc = chunks(t);
      const float rho = p.first ? p.rho[t.mat] : 0.0f;
      if (!__all_sync(0xffffffffu, mbar_wait_cluster(&tfull[acc], ((uint32_t)i >> 1) & 1u, p.status, p.timeout_ns))) break;
      tc_fence_after();
      const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + acc * 256u;
#pragma unroll 1
      for (int c = 0; c < nc; ++c, ++n) {
        const int b = n & 1;
        if (!__all_sync(0xffffffffu, mbar_wait(&eload[b], ((uint32_t)n >> 1) & 1u, p.status, p.timeout_ns))) { ok = false; break; }
        uint8_t* e = ebuf + b * NS_EBUF;
        ns_chunk<KIND>(p, t, e, e + 2 * NS_BOX, rl, t.m0 + rank * 128 + rl, t.n0 + 64 * c, rho, taddr + 64u * (uint32_t)c);
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
        if (!mbar_wait(&edone[b], ((uint32_t)n >> 1) & 1u, p.status, p.timeout_ns)) { ok = false; break; }
        const uint8_t* e = ebuf + b * NS_EBUF;
        if (KIND == NS_STEP) {
          if (!p.last || p.out_vec) tma_store_3d(&mp.out0, e, col, row, t.mat);
          if (!p.last) tma_store_3d(&mp.out1, e + 2 * NS_BOX, col, row, t.mat);
        } else {
          tma_store_3d(&mp.out0, e, col, row, t.mat);
          if (t.m0 != t.n0) {
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
  settle_after_abort(p.status);
  tc_fence_before();
  __syncthreads();
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
  double* part;            // [nb, NS_PREP_BLOCKS, 3]
  float* rho;              // [nb]
  __half* hi;
  __half* lo;
  int* status;             // cleared by the call's first launch (NULL in the others)
};

__device__ __forceinline__ float load_grad(const void* g, int dtype, size_t i) {
  if (dtype == MOE_DTYPE_FP32) return static_cast<const float*>(g)[i];
  if (dtype == MOE_DTYPE_BF16) return __bfloat162float(static_cast<const bf16*>(g)[i]);
  return __half2float(static_cast<const __half*>(g)[i]);
}
// The V values U (V = 4: 16 or 8 bytes of the gradient at once) at row r,
// columns c .. c + V - 1; `advance` takes the momentum one step first.
template <int V>
__device__ __forceinline__ void load_u(const PrepParams& p, int mat, int r, int c, bool advance, float (&u)[V]) {
  const size_t gi = (size_t)mat * p.gms + (size_t)r * p.grs + c;
  if constexpr (V == 4) {
    if (p.dtype == MOE_DTYPE_FP32) {
      const float4 w = *reinterpret_cast<const float4*>(static_cast<const float*>(p.grad) + gi);
      u[0] = w.x, u[1] = w.y, u[2] = w.z, u[3] = w.w;
    } else {
      const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.grad) + gi);
      const uint16_t h[4] = {(uint16_t)w.x, (uint16_t)(w.x >> 16), (uint16_t)w.y, (uint16_t)(w.y >> 16)};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        u[j] = p.dtype == MOE_DTYPE_BF16 ? __uint_as_float((uint32_t)h[j] << 16) : __half2float(__ushort_as_half(h[j]));
    }
  } else {
    u[0] = load_grad(p.grad, p.dtype, gi);
  }
  if (!p.momentum) return;
  float* mp = p.momentum + ((size_t)mat * p.R + r) * p.C + c;
  float m[V];
  if constexpr (V == 4) {
    const float4 w = *reinterpret_cast<const float4*>(mp);
    m[0] = w.x, m[1] = w.y, m[2] = w.z, m[3] = w.w;
  } else {
    m[0] = *mp;
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if (advance) m[j] = p.mu * m[j] + u[j];
    u[j] = p.nesterov ? u[j] + p.mu * m[j] : m[j];
  }
  if (advance) {
    if constexpr (V == 4) *reinterpret_cast<float4*>(mp) = make_float4(m[0], m[1], m[2], m[3]);
    else *mp = m[0];
  }
}

// Advance the momentum and sum U's squares: fp32 runs of at most a few hundred
// per thread, fp64 across threads.  Values far from 1 are summed in scaled
// form in sums of their own, so that no finite matrix has an infinite norm and
// none that is not zero has a zero one.
template <int V>
__global__ void __launch_bounds__(256) ns_prep_norm(const PrepParams p) {
  __shared__ double s[3][8];
  const int mat = blockIdx.y, cv = p.C / V;
  const int n = p.R * cv;
  if (p.status && blockIdx.x == 0 && mat == 0 && threadIdx.x == 0) p.status[0] = 0;
  double tot[3] = {0.0, 0.0, 0.0};
  float f[3] = {0.0f, 0.0f, 0.0f};
  int run = 0;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
    const int r = (int)i / cv, c = ((int)i - r * cv) * V;
    float u[V];
    load_u<V>(p, mat, r, c, true, u);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float a = fabsf(u[j]);
      const bool big = a >= 0x1p50f, small = a < 0x1p-50f;
      const float v = u[j] * (big ? 0x1p-80f : small ? 0x1p100f : 1.0f);
      f[0] += small ? v * v : 0.0f;
      f[1] += big || small ? 0.0f : v * v;
      f[2] += big ? v * v : 0.0f;
    }
    if (++run == 64) {
#pragma unroll
      for (int q = 0; q < 3; ++q) tot[q] += (double)f[q], f[q] = 0.0f;
      run = 0;
    }
  }
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    tot[q] += (double)f[q];
    for (int o = 16; o > 0; o >>= 1) tot[q] += __shfl_xor_sync(0xffffffffu, tot[q], o);
    if ((threadIdx.x & 31) == 0) s[q][threadIdx.x >> 5] = tot[q];
  }
  __syncthreads();
  if (threadIdx.x < 3) {
    double v = 0.0;
    for (int w = 0; w < 8; ++w) v += s[threadIdx.x][w];
    p.part[((size_t)mat * NS_PREP_BLOCKS + blockIdx.x) * 3 + threadIdx.x] = v;
  }
}

// X_0 = U 2^k as hi + lo, |U 2^k|_F in [2^14, 2^15); rho = 1 / |U 2^k|_F (0 for
// a matrix of zeros, NaN where the norm is not finite, which makes every
// element of that matrix's result NaN).
template <int V>
__global__ void __launch_bounds__(256) ns_prep_first(const PrepParams p) {
  __shared__ double s[3][8];
  __shared__ float s_f[2];
  const int mat = blockIdx.y, cv = p.C / V;
  const int n = p.R * cv;
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    double v = (int)threadIdx.x < p.nblk ? p.part[((size_t)mat * NS_PREP_BLOCKS + threadIdx.x) * 3 + q] : 0.0;
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) s[q][threadIdx.x >> 5] = v;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    double v[3];
    for (int q = 0; q < 3; ++q) {
      v[q] = 0.0;
      for (int w = 0; w < 8; ++w) v[q] += s[q][w];
    }
    const double norm = sqrt(v[0] * 0x1p-200 + v[1] + v[2] * 0x1p160);
    float f1 = 0.0f, f2 = 0.0f, rho = 0.0f;
    if (!(norm < (double)INFINITY)) {
      rho = NAN;
    } else if (norm > 0.0) {
      int e;
      frexp(norm, &e);  // norm = [0.5, 1) 2^e
      const int k = 15 - e;
      f1 = ldexpf(1.0f, k / 2);
      f2 = ldexpf(1.0f, k - k / 2);
      rho = (float)(1.0 / ldexp(norm, k));
    }
    s_f[0] = f1;
    s_f[1] = f2;
    if (blockIdx.x == 0) p.rho[mat] = rho;
  }
  __syncthreads();
  const float f1 = s_f[0], f2 = s_f[1];
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
    const int r = (int)i / cv, c = ((int)i - r * cv) * V;
    float u[V];
    load_u<V>(p, mat, r, c, false, u);
    __half h[V], l[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float x = u[j] * f1 * f2;
      h[j] = __float2half_rn(x);
      l[j] = __float2half_rn(x - __half2float(h[j]));
    }
    const size_t o = ((size_t)mat * p.R + r) * p.ld + c;
    if constexpr (V == 4) {
      *reinterpret_cast<uint2*>(p.hi + o) = make_uint2((uint32_t)__half_as_ushort(h[0]) | ((uint32_t)__half_as_ushort(h[1]) << 16),
                                                       (uint32_t)__half_as_ushort(h[2]) | ((uint32_t)__half_as_ushort(h[3]) << 16));
      *reinterpret_cast<uint2*>(p.lo + o) = make_uint2((uint32_t)__half_as_ushort(l[0]) | ((uint32_t)__half_as_ushort(l[1]) << 16),
                                                       (uint32_t)__half_as_ushort(l[2]) | ((uint32_t)__half_as_ushort(l[3]) << 16));
    } else {
      p.hi[o] = h[0];
      p.lo[o] = l[0];
    }
  }
}

}  // namespace moe

// ------------------------------------------------------------------ C ABI
using namespace moe;

struct moe_muon_plan {
  moe_muon_config cfg;
  int device, num_sms;
  int64_t chunk;  // matrices in flight
  encode_tiled_fn encode;
};

namespace {

int64_t up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }
bool ns_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct NsLayout {
  size_t rho, part, hi[2], lo[2], a, b, da, db, total;
  int64_t m, n, ldx, lda, ldd;
};

NsLayout ns_layout(const moe_muon_plan* pl) {
  const moe_muon_config& c = pl->cfg;
  NsLayout L{};
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
  L.part = take(sizeof(double) * 3 * NS_PREP_BLOCKS * pl->chunk);
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

template <int KIND, bool A_MN, bool B_MN>
cudaError_t ns_launch(const moe_muon_plan* pl, const NsMaps& mp, const NsParams& p, cudaStream_t st) {
  cudaError_t err = cudaFuncSetAttribute(ns_gemm<KIND, A_MN, B_MN>, cudaFuncAttributeMaxDynamicSharedMemorySize, NS_SMEM);
  if (err != cudaSuccess) return err;
  const int64_t units = (int64_t)p.nb * p.n_tiles, pairs = pl->num_sms / 2;
  ns_gemm<KIND, A_MN, B_MN><<<(unsigned)(2 * (units < pairs ? units : pairs)), NS_THREADS, NS_SMEM, st>>>(mp, p);
  return cudaGetLastError();
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

  PrepParams pp{};
  pp.grs = grad_row_stride;
  pp.gms = grad_stride;
  pp.dtype = c.grad_dtype;
  pp.R = (int)c.rows;
  pp.C = (int)c.cols;
  pp.nesterov = nesterov;
  pp.ld = L.ldx;
  pp.mu = mu;
  pp.part = reinterpret_cast<double*>(ws + L.part);
  pp.rho = reinterpret_cast<float*>(ws + L.rho);
  pp.hi = half_at(L.hi[0]);
  pp.lo = half_at(L.lo[0]);
  const bool vec = c.cols % 4 == 0 && grad_row_stride % 4 == 0 && grad_stride % 4 == 0 && ns_aligned(grad, 4 * gsize) &&
                   ns_aligned(momentum, 16);
  const int64_t nvec = c.rows * c.cols / (vec ? 4 : 1);
  const int64_t nblk = up(nvec, 2048) / 2048;
  pp.nblk = (int)(nblk < NS_PREP_BLOCKS ? nblk : NS_PREP_BLOCKS);

  NsParams g{};
  g.rho = pp.rho;
  g.status = reinterpret_cast<int*>(ws);
  g.timeout_ns = (long long)c.timeout_ms * 1000000LL;
  g.scale = scale / NS_S;
  g.tall = tall;
  g.ldd = (int)L.ldd;
  g.diag_a = reinterpret_cast<float*>(ws + L.da);
  g.diag_b = reinterpret_cast<float*>(ws + L.db);
  const int64_t mt = up(L.m, NS_TILE) / NS_TILE;
  for (int64_t c0 = 0; c0 < c.count; c0 += pl->chunk) {
    const int nb = (int)(c.count - c0 < pl->chunk ? c.count - c0 : pl->chunk);
    pp.grad = static_cast<const uint8_t*>(grad) + (size_t)c0 * grad_stride * gsize;
    pp.status = c0 == 0 ? g.status : nullptr;
    pp.momentum = momentum ? momentum + (size_t)c0 * c.rows * c.cols : nullptr;
    bf16* out = static_cast<bf16*>(update) + (size_t)c0 * c.rows * c.cols;
    const dim3 pgrid((unsigned)pp.nblk, (unsigned)nb);
    if (vec) {
      ns_prep_norm<4><<<pgrid, 256, 0, st>>>(pp);
      ns_prep_first<4><<<pgrid, 256, 0, st>>>(pp);
    } else {
      ns_prep_norm<1><<<pgrid, 256, 0, st>>>(pp);
      ns_prep_first<1><<<pgrid, 256, 0, st>>>(pp);
    }
    if (cudaGetLastError() != cudaSuccess) return MOE_ERR_CUDA;
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
      g.tiles_n = (int)mt;
      g.n_tiles = (int)(mt * (mt + 1) / 2);
      const CUtensorMap& xx = tall ? xm[x] : xk[x];
      const NsMaps gram = {xx, xx, ak, ak, ak, am};
      err = tall ? ns_launch<NS_GRAM, true, true>(pl, gram, g, st) : ns_launch<NS_GRAM, false, false>(pl, gram, g, st);
      if (err != cudaSuccess) return MOE_ERR_CUDA;
      // B = b A + c A^2
      g.K = (int)L.m;
      g.ca = c.b;
      g.cb = c.c / NS_S;
      const NsMaps poly = {ak, ak, ak, ak, bk, bm};
      if (ns_launch<NS_POLY, false, false>(pl, poly, g, st) != cudaSuccess) return MOE_ERR_CUDA;
      // X <- a X + B X or a X + X B
      g.M = (int)c.rows;
      g.N = (int)c.cols;
      g.tiles_n = (int)(up(c.cols, NS_TILE) / NS_TILE);
      g.n_tiles = (int)(up(c.rows, NS_TILE) / NS_TILE) * g.tiles_n;
      g.ca = c.a;
      g.cb = 1.0f / NS_S;
      const NsMaps step = {tall ? xk[x] : bk, tall ? bk : xm[x], xk[x], xl[x], g.last ? uk : xk[x ^ 1], xl[x ^ 1]};
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
