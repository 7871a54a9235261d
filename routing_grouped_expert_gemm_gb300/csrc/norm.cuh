// Shared by the kernels of the norms around a block (norm.cu, norm_fwd.cu, norm_bwd.cu,
// norm_any_fwd.cu, norm_any_bwd.cu): parameters, packed fp32 arithmetic, rows in vectors, sums.
//
//   z = N(o),  y = a x + b g z,  h = N(y),   N(v) = (v - m) r w + c,
//   r = 1 / sqrt(mean((v - m)^2) + eps),  m = mean(v) or 0.
//
// Backward, with n = (v - m) r and u = d w for the gradient d of N's output:
//   dv = r (u - n mean(u n) - mean(u)),   dw = sum d n,   dc = sum d
// (the mean of u only where m is the row's mean), so a row needs one sum per
// norm before its gradient is known, and y's comes before o's:
//   dy += dv(dh),  dx = a dy,  dg = b dy z,  do = dv(b g dy).
//
// All of it is bound by memory: the forward reads x and o and writes y and h,
// the backward reads y, o, dy and dh and writes dx and do, each once.  Thread i of
// the threads that share a row owns the same vectors of 8 elements of every row: it
// fetches them ahead into its own part of shared memory (cp.async; no barrier, nobody
// else reads them) and meets the others only for the row's sums, one barrier each.
#pragma once
#include <cuda_fp16.h>

#include <type_traits>

#include "../../include/moe.h"
#include "common.cuh"

namespace moe {

constexpr int NORM_MAX_D = 16384;
constexpr int NORM_MAX_WARPS = 16;  // of the threads that share a row
constexpr int NORM_SUMS = 5;        // dw and dc of both norms, dg
// threads of the forward's CTA: 64 registers each suffice for two vectors a thread
constexpr int norm_fwd_threads(int nv) { return nv <= 2 ? 1024 : 512; }

// Most of a row's instructions are not its arithmetic: looking at what a call has and
// has not costs more than a hundred of them.  So the kernels have a form (`whole` 1) for
// the call between two blocks of a large batch: all rows there, both norms, no gate
// (backward: none or one per channel), as many rows in the ring as these constants say;
// one (2) where besides every thread's vectors lie in the row (D a multiple of 512); and
// one that looks (0).  16384 rows in bf16 by 0, 1 and 2, us:
//            rms forward       gradient         layer forward     gradient
//   7168     153  161  149     240  240  231    331  310  288     494  340  348
//   5952     138  122   -      218  218   -     294  270   -      460  313   -
//   2048      47   49   49      89   79   78     81   74   68     128   95   95
constexpr int NORM_FWD_STAGES = 2, NORM_BWD_STAGES = 2;

struct NormParams {
  int64_t T;
  int D, nvec;     // nvec: vectors of 8 elements in a row
  int post, pre, sdt, bdt, pdt, layer;
  int group;       // forward: threads that share a row (a CTA's are that many times its rows at a time)
  int smem_w;      // forward: the weights in shared memory
  int stages;      // rows in the ring
  int whole, places;  // places: elements of a row in the ring, 8 for every vector of every thread
  int stage_bytes; // of a row in the ring
  float inv_d, eps, w_off, x_scale, o_scale;
  const void *w1, *c1, *w2, *c2, *gate;
  int gate_rows;
  int64_t gate_ld;
  const void *x, *o, *dy, *dh;
  int64_t x_ld, o_ld, y_ld, h_ld, dy_ld, dh_ld, dx_ld, do_ld, dgate_ld;
  void *y, *h, *dx, *d_o, *dgate;
  float* stats;
  float* sums;     // backward: [gridDim.x][NORM_SUMS][D]
};

// Fast kernels: rows in whole vectors on 16-byte boundaries
cudaError_t launch_norm_fwd(const NormParams& p, unsigned grid, unsigned threads, size_t smem, cudaStream_t st);
cudaError_t launch_norm_bwd(const NormParams& p, bool gate_sum, bool pairs, unsigned grid, unsigned threads, size_t smem, cudaStream_t st);
// Any rows (norm_any_fwd.cu, norm_any_bwd.cu)
cudaError_t launch_norm_fwd_any(const NormParams& p, unsigned grid, unsigned threads, size_t smem, cudaStream_t st);
cudaError_t launch_norm_bwd_any(const NormParams& p, unsigned grid, unsigned threads, size_t smem, cudaStream_t st);

constexpr int NORM_SMEM = 200 * 1024;  // of an SM's shared memory for the rings: no launch asks for more

// The limit of shared memory belongs to the kernel, not to the launch, and another
// thread's call may set it in between: so every call sets the same.
template <typename P>
cudaError_t norm_launch(void (*kernel)(P), dim3 grid, unsigned threads, size_t smem, cudaStream_t st, const P& p) {
  if (smem > 40 * 1024) {  // 48 KB with what the kernel holds besides
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, NORM_SMEM);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t lc = {};
  lc.gridDim = grid;
  lc.blockDim = dim3(threads);
  lc.dynamicSmemBytes = smem;
  lc.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // set up while what is before it still runs
  at[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = at;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, kernel, p);
}

// Pairs of fp32 values: one instruction for both (fma.rn.f32x2 and its kin), each
// rounded as the single instruction rounds.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ F2 f2(float a) { return f2(a, a); }
__device__ __forceinline__ float2 split(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

__host__ __device__ constexpr int esize(int dt) { return dt == MOE_DTYPE_FP32 ? 4 : 2; }

// One vector of 8: 16 bytes of a 16-bit type, or two times 16 of fp32
template <int DT>
struct Raw {
  uint4 q[DT == MOE_DTYPE_FP32 ? 2 : 1];
};
template <int DT>
__device__ __forceinline__ void unpack(const Raw<DT>& r, F2 (&v)[4]) {
  if constexpr (DT == MOE_DTYPE_FP32) {
    v[0] = f2(__uint_as_float(r.q[0].x), __uint_as_float(r.q[0].y)), v[1] = f2(__uint_as_float(r.q[0].z), __uint_as_float(r.q[0].w));
    v[2] = f2(__uint_as_float(r.q[1].x), __uint_as_float(r.q[1].y)), v[3] = f2(__uint_as_float(r.q[1].z), __uint_as_float(r.q[1].w));
  } else {
    const uint32_t w[4] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == MOE_DTYPE_BF16) {
        v[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        v[i] = f2(f.x, f.y);
      }
    }
  }
}
// v rounded to the type; v holds what was rounded
template <int DT>
__device__ __forceinline__ Raw<DT> pack(F2 (&v)[4]) {
  Raw<DT> r;
  if constexpr (DT == MOE_DTYPE_FP32) {
    const float2 a = split(v[0]), b = split(v[1]), c = split(v[2]), d = split(v[3]);
    r.q[0] = make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
    r.q[1] = make_uint4(__float_as_uint(c.x), __float_as_uint(c.y), __float_as_uint(d.x), __float_as_uint(d.y));
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = split(v[i]);
      if constexpr (DT == MOE_DTYPE_BF16) {
        w[i] = pack_bf16x2(a.x, a.y);
      } else {
        const __half2 h = __floats2half2_rn(a.x, a.y);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    r.q[0] = make_uint4(w[0], w[1], w[2], w[3]);
    unpack<DT>(r, v);
  }
  return r;
}

__device__ __forceinline__ void cp_async16(char* smem, const void* g) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(smem)), "l"(g) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all but the `n` newest groups of this thread have landed (n up to 3)
constexpr int CP_ASYNC_MOST = 3;
static_assert(2 * NORM_FWD_STAGES - 1 <= CP_ASYNC_MOST && NORM_BWD_STAGES - 1 <= CP_ASYNC_MOST, "groups under way in a ring");
__device__ __forceinline__ void cp_async_wait(int n) {
  if (n <= 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
  else if (n == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
  else if (n == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
  else asm volatile("cp.async.wait_group 3;" ::: "memory");
}
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// A thread's vectors: offsets of 16 bytes a vector, and whether they lie in the row.
// In shared memory vectors of fp32 lie in two planes of 16 bytes each (no bank conflicts).
// Choosing between a value and 0 for every element would be a third of the instructions:
// ALL: all of all threads' vectors lie in the row; else the ring has places for those
// outside too, and they hold zeros.
template <int NV, bool ALL>
struct Mine {
  uint32_t off[NV], plane;
  bool in_[NV];
  __device__ __forceinline__ bool in(int j) const { return ALL || in_[j]; }
  __device__ __forceinline__ Mine(int tid, int nt, int nvec, int places) {
#pragma unroll
    for (int j = 0; j < NV; ++j) off[j] = (uint32_t)(tid + j * nt) * 16u, in_[j] = tid + j * nt < nvec;
    plane = ALL ? (uint32_t)nvec * 16u : (uint32_t)places * 2u;
  }
  // once: zeros in this thread's places outside the row, in every 16 bytes of all vectors'
  __device__ __forceinline__ void clear(char* stage, uint32_t stage_bytes) const {
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (!in(j))
        for (uint32_t at = off[j]; at < stage_bytes; at += plane) *reinterpret_cast<uint4*>(stage + at) = make_uint4(0, 0, 0, 0);
  }
  template <int DT>
  __device__ __forceinline__ void fetch(char* smem, const char* row) const {
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (in(j)) {
        if constexpr (DT == MOE_DTYPE_FP32) {
          cp_async16(smem + off[j], row + 2 * off[j]);
          cp_async16(smem + off[j] + plane, row + 2 * off[j] + 16);
        } else {
          cp_async16(smem + off[j], row + off[j]);
        }
      }
  }
  // vector j out of shared memory; 0 outside the row
  template <int DT>
  __device__ __forceinline__ void take(int j, const char* smem, F2 (&v)[4]) const {
    Raw<DT> r;
    r.q[0] = *reinterpret_cast<const uint4*>(smem + off[j]);
    if constexpr (DT == MOE_DTYPE_FP32) r.q[1] = *reinterpret_cast<const uint4*>(smem + off[j] + plane);
    unpack<DT>(r, v);
  }
  template <int DT, bool THERE>
  __device__ __forceinline__ void put(int j, char* row, F2 (&v)[4]) const {
    const Raw<DT> r = pack<DT>(v);
    if ((THERE || row) && in(j)) {
      uint4* to = reinterpret_cast<uint4*>(row + (DT == MOE_DTYPE_FP32 ? 2 * off[j] : off[j]));
      to[0] = r.q[0];
      if constexpr (DT == MOE_DTYPE_FP32) to[1] = r.q[1];
    }
  }
  // vector j in global memory, of a type known now (parameters, a gate's rows)
  __device__ __forceinline__ void global(int j, const void* row, int dt, float none, F2 (&v)[4]) const {
    if (!in(j)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = f2(none);
    } else if (dt == MOE_DTYPE_FP32) {
      Raw<MOE_DTYPE_FP32> r;
      const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(row) + 2 * off[j]);
      r.q[0] = q[0], r.q[1] = q[1];
      unpack<MOE_DTYPE_FP32>(r, v);
    } else if (dt == MOE_DTYPE_BF16) {
      unpack<MOE_DTYPE_BF16>(Raw<MOE_DTYPE_BF16>{{*reinterpret_cast<const uint4*>(static_cast<const char*>(row) + off[j])}}, v);
    } else {
      unpack<MOE_DTYPE_FP16>(Raw<MOE_DTYPE_FP16>{{*reinterpret_cast<const uint4*>(static_cast<const char*>(row) + off[j])}}, v);
    }
  }
  // a norm's weight with its offset, or ones; 0 outside the row, where gradients may
  // be other than 0 (a layer norm's mean)
  __device__ __forceinline__ void weight(int j, const void* w, int dt, float offset, F2 (&v)[4]) const {
    if (w) {
      global(j, w, dt, -offset, v);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = v[i] + f2(offset);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = f2(in(j) ? 1.0f : 0.0f);
    }
  }
};

// The threads that share a row: `warps` warps of the CTA, meeting at barrier `id`
struct Group {
  float* red;  // [2][2][NORM_MAX_WARPS]
  int id, warps, warp, turn;
};
// Sums of N values over the group, every thread getting the same bits.  `red`
// alternates between two buffers, so that one barrier a call is enough.
template <int N, int MAX_WARPS = NORM_MAX_WARPS>
__device__ __forceinline__ void group_sums(float (&v)[N], Group& g) {
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], m);
  if (g.warps == 1) return;
  float* r = g.red + g.turn * (2 * MAX_WARPS);
  g.turn ^= 1;
  const int lane = threadIdx.x & 31;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) r[i * MAX_WARPS + g.warp] = v[i];
  named_bar_sync(g.id, g.warps * 32);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = lane < g.warps ? r[i * MAX_WARPS + lane] : 0.0f;
  // (of at most 16 warps the upper half of the lanes would add zeros)
#pragma unroll
  for (int m = MAX_WARPS / 2; m >= 1; m >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], m);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, v[i], 0);
}
__device__ __forceinline__ float both(F2 a, F2 b) {
  const float2 s = split(a + b);
  return s.x + s.y;
}

// mean (or 0) and 1 / sqrt(mean((v - m)^2) + eps) of one row whose elements
// outside the row are 0 in v; two passes over the registers, so that a large
// mean does not cancel
template <int NV, bool LN, bool ALL>
__device__ __forceinline__ void row_stats(const Mine<NV, ALL>& mine, const F2 (&v)[NV][4], float inv_d, float eps, Group& grp,
                                          float& m, float& r) {
  float s[1];
  F2 q[2] = {f2(0.0f), f2(0.0f)};
  m = 0.0f;
  if constexpr (LN) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i & 1] = q[i & 1] + v[j][i];
    s[0] = both(q[0], q[1]);
    group_sums(s, grp);
    m = s[0] * inv_d;
    q[0] = q[1] = f2(0.0f);
  }
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (!LN || mine.in(j))
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const F2 d = LN ? v[j][i] + f2(-m) : v[j][i];
        q[i & 1] = fma2(d, d, q[i & 1]);
      }
  s[0] = both(q[0], q[1]);
  group_sums(s, grp);
  r = rsqrtf(fmaf(s[0], inv_d, eps));  // within 2 ulp
}

}  // namespace moe
