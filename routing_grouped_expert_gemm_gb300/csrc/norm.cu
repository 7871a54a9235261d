// Norms around a block and their gradients (moe_norm, moe_norm_bwd in
// include/moe.h):  z = N(o),  y = a x + b g z,  h = N(y),  where
//   N(v) = (v - m) r w + c,   r = 1 / sqrt(mean((v - m)^2) + eps),   m = mean(v) or 0.
//
// Backward, with n = (v - m) r and u = d w for the gradient d of N's output:
//   dv = r (u - n mean(u n) - mean(u)),   dw = sum d n,   dc = sum d
// (the mean of u only where m is the row's mean), so a row needs one sum per
// norm before its gradient is known, and y's comes before o's:
//   dy += dv(dh),  dx = a dy,  dg = b dy z,  do = dv(b g dy).
//
// All of it is bound by memory: the forward reads x and o and writes y and h,
// the backward reads y, o, dy and dh and writes dx and do, each once.  A CTA
// keeps to its own columns: thread i owns the same vectors of 8 elements of
// every row, so it fetches them ahead into its own part of shared memory
// (cp.async; no barrier, nobody else reads them), holds the norms' weights and
// the sums for dw and dc in registers, and meets the other threads only for the
// row's sums (one barrier each).
#include <cuda_fp16.h>

#include <new>
#include <type_traits>

#include "../../include/moe.h"
#include "common.cuh"

namespace moe {

constexpr int NORM_MAX_D = 16384;
constexpr int NORM_MAX_WARPS = 16;   // of the threads that share a row
// threads of the forward's CTA: 64 registers each suffice for two vectors a thread
constexpr int norm_fwd_threads(int nv) { return nv <= 2 ? 1024 : 512; }
constexpr int NORM_SUMS = 5;  // dw and dc of both norms, dg

struct NormParams {
  int64_t T;
  int D, nvec;     // nvec: vectors of 8 elements in a row, the last of which may be shorter
  int post, pre, sdt, bdt, pdt;
  int group;       // forward: threads that share a row (a CTA's are that many times its rows at a time)
  int smem_w;      // forward: the weights in shared memory
  int stages;      // rows in the ring (0: no ring)
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

// 8 consecutive elements, 16-byte aligned; `half` is where the last four of fp32 lie
__device__ __forceinline__ void norm_load8(const void* p, int dt, F2* v, size_t half = 16) {
  if (dt == MOE_DTYPE_FP32) {
    const float4 a = *static_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(static_cast<const char*>(p) + half);
    v[0] = f2(a.x, a.y), v[1] = f2(a.z, a.w), v[2] = f2(b.x, b.y), v[3] = f2(b.z, b.w);
    return;
  }
  const uint4 q = *static_cast<const uint4*>(p);
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  if (dt == MOE_DTYPE_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[i] = f2(f.x, f.y);
    }
  }
}
// 8 elements rounded to dt, stored (16-byte aligned) unless p is null; v holds what was rounded
__device__ __forceinline__ void norm_store8(void* p, int dt, F2* v) {
  if (dt == MOE_DTYPE_FP32) {
    if (p) {
      const float2 a = split(v[0]), b = split(v[1]), c = split(v[2]), d = split(v[3]);
      static_cast<float4*>(p)[0] = make_float4(a.x, a.y, b.x, b.y);
      static_cast<float4*>(p)[1] = make_float4(c.x, c.y, d.x, d.y);
    }
    return;
  }
  uint32_t w[4];
  if (dt == MOE_DTYPE_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = split(v[i]);
      w[i] = pack_bf16x2(a.x, a.y);
      v[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = split(v[i]);
      const __half2 h = __floats2half2_rn(a.x, a.y);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
      const float2 f = __half22float2(h);
      v[i] = f2(f.x, f.y);
    }
  }
  if (p) *static_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void cp_async16(void* smem, const void* g) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(smem)), "l"(g) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all but the `n` newest groups of this thread have landed (n up to 5)
__device__ __forceinline__ void cp_async_wait(int n) {
  if (n <= 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
  else if (n == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
  else if (n == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
  else if (n == 3) asm volatile("cp.async.wait_group 3;" ::: "memory");
  else if (n == 4) asm volatile("cp.async.wait_group 4;" ::: "memory");
  else asm volatile("cp.async.wait_group 5;" ::: "memory");
}
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The threads that share a row: `warps` warps of the CTA, meeting at barrier `id`
struct Group {
  float* red;  // [2][2][NORM_MAX_WARPS]
  int id, warps, warp, turn;
};
// Sums of N values over the group, every thread getting the same bits.  `red`
// alternates between two buffers, so that one barrier a call is enough.
template <int N>
__device__ __forceinline__ void group_sums(float (&v)[N], Group& g) {
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], m);
  if (g.warps == 1) return;
  float* r = g.red + g.turn * (2 * NORM_MAX_WARPS);
  g.turn ^= 1;
  const int lane = threadIdx.x & 31;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) r[i * NORM_MAX_WARPS + g.warp] = v[i];
  named_bar_sync(g.id, g.warps * 32);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = lane < g.warps ? r[i * NORM_MAX_WARPS + lane] : 0.0f;
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], m);
}

__device__ __forceinline__ int esize(int dt) { return dt == MOE_DTYPE_FP32 ? 4 : 2; }
__device__ __forceinline__ const void* row_at(const void* p, int64_t r, int64_t ld, int dt) {
  return p ? static_cast<const char*>(p) + r * ld * esize(dt) : nullptr;
}
__device__ __forceinline__ void* row_at(void* p, int64_t r, int64_t ld, int dt) {
  return p ? static_cast<char*>(p) + r * ld * esize(dt) : nullptr;
}

// The same one element at a time, for calls with rows or parameters off 16-byte
// boundaries or rows that do not end on one: elements at .. at + 7 that lie in the
// row (`none` past its end).  Calls of their own, so that they cost the kernels
// no registers: 1003 x 2053 in fp16 UNALIGNEDCOST.
struct V8 {
  float f[8];
};
__device__ __noinline__ V8 norm_load_any(const void* row, int dt, int at, int D, float none) {
  V8 v;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v.f[i] = none;
    if (at + i < D) {
      if (dt == MOE_DTYPE_FP32) {
        v.f[i] = static_cast<const float*>(row)[at + i];
      } else {
        const uint16_t h = static_cast<const uint16_t*>(row)[at + i];
        v.f[i] = dt == MOE_DTYPE_BF16 ? __uint_as_float((uint32_t)h << 16) : __half2float(__ushort_as_half(h));
      }
    }
  }
  return v;
}
__device__ __noinline__ void norm_store_any(void* row, int dt, int at, int D, V8 v) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (at + i < D) {
      if (dt == MOE_DTYPE_FP32) static_cast<float*>(row)[at + i] = v.f[i];
      else if (dt == MOE_DTYPE_BF16) static_cast<bf16*>(row)[at + i] = __float2bfloat16_rn(v.f[i]);
      else static_cast<__half*>(row)[at + i] = __float2half_rn(v.f[i]);
    }
}

// The elements of a row that a thread owns, as pairs: vectors tid + j NT of 8.
// vec: all of them whole and on 16-byte boundaries.
template <int NV, bool vec>
struct Own {
  static constexpr int N = NV * 4;  // pairs
  int nt, tid, D, nvec;
  __device__ __forceinline__ bool vec_in(int j) const { return tid + j * nt < nvec; }
  // element e (0 or 1) of pair i lies in the row
  __device__ __forceinline__ bool in(int i, int e) const { return (tid + i / 4 * nt) * 8 + 2 * (i % 4) + e < D; }

  // vector j of a parameter or a row; `none` where there is no element.  `ring`: in shared
  // memory, where vectors of fp32 lie in two planes of 16 bytes each (no bank conflicts)
  __device__ __forceinline__ void load(int j, const void* row, int dt, float none, F2* v, bool ring = false) const {
    if (vec_in(j)) {
      if (ring) {
        norm_load8(static_cast<const char*>(row) + (tid + j * nt) * 16, dt, v, (size_t)nvec * 16);
      } else if (vec) {
        norm_load8(static_cast<const char*>(row) + (size_t)(tid + j * nt) * 8 * esize(dt), dt, v);
      } else {
        const V8 w = norm_load_any(row, dt, (tid + j * nt) * 8, D, none);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = f2(w.f[2 * i], w.f[2 * i + 1]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = f2(none);
    }
  }
  __device__ __forceinline__ void load(const void* row, int dt, float none, F2 (&v)[N], bool ring = false) const {
#pragma unroll
    for (int j = 0; j < NV; ++j) load(j, row, dt, none, v + 4 * j, ring);
  }
  // round to dt, store unless row is null; v holds the rounded values
  __device__ __forceinline__ void store(int j, void* row, int dt, F2* v) const {
    const bool out = row && vec_in(j);
    norm_store8(out && vec ? static_cast<char*>(row) + (size_t)(tid + j * nt) * 8 * esize(dt) : nullptr, dt, v);
    if (out && !vec) {
      V8 w;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 a = split(v[i]);
        w.f[2 * i] = a.x, w.f[2 * i + 1] = a.y;
      }
      norm_store_any(row, dt, (tid + j * nt) * 8, D, w);
    }
  }
  __device__ __forceinline__ void store(void* row, int dt, F2 (&v)[N]) const {
#pragma unroll
    for (int j = 0; j < NV; ++j) store(j, row, dt, v + 4 * j);
  }
  // a norm's weight with its offset, or ones; 0 outside the row, where gradients
  // may be other than 0 (a layer norm's mean)
  __device__ __forceinline__ void weight(int j, const void* w, int dt, float offset, F2* v) const {
    if (w) {
      load(j, w, dt, -offset, v);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = v[i] + f2(offset);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = f2(in(4 * j + i, 0) ? 1.0f : 0.0f, in(4 * j + i, 1) ? 1.0f : 0.0f);
    }
  }
  __device__ __forceinline__ void weight(const void* w, int dt, float offset, F2 (&v)[N]) const {
#pragma unroll
    for (int j = 0; j < NV; ++j) weight(j, w, dt, offset, v + 4 * j);
  }
};

// Rows of up to four tensors, fetched ahead by the thread that owns them:
// slot (stage, tensor) of the ring holds a row's vectors in their own order.
template <int NV>
struct Ring {
  char* base;
  int stage_bytes, off[4];
  __device__ __forceinline__ void fetch(const Own<NV, true>& own, int stage, int t, const void* row, int dt) const {
    char* s = base + stage * stage_bytes + off[t];
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (own.vec_in(j)) {
        const uint32_t i = own.tid + j * own.nt;
        const char* g = static_cast<const char*>(row) + i * 8 * esize(dt);
        cp_async16(s + i * 16, g);
        if (dt == MOE_DTYPE_FP32) cp_async16(s + (own.nvec + i) * 16, g + 16);
      }
  }
  __device__ __forceinline__ const void* row(int stage, int t) const { return base + stage * stage_bytes + off[t]; }
};

// mean (or 0) and 1 / sqrt(mean((v - m)^2) + eps) of one row whose elements
// outside the row are 0 in v; two passes over the registers, so that a large
// mean does not cancel
template <int NV, bool LN, bool VEC>
__device__ __forceinline__ void row_stats(const Own<NV, VEC>& own, const F2 (&v)[NV * 4], float inv_d, float eps,
                                          Group& grp, float& m, float& r) {
  float s[1];
  F2 q[2] = {f2(0.0f), f2(0.0f)};
  m = 0.0f;
  if constexpr (LN) {
#pragma unroll
    for (int i = 0; i < NV * 4; ++i) q[i & 1] = q[i & 1] + v[i];
    const float2 a = split(q[0] + q[1]);
    s[0] = a.x + a.y;
    group_sums(s, grp);
    m = s[0] * inv_d;
    q[0] = q[1] = f2(0.0f);
#pragma unroll
    for (int i = 0; i < NV * 4; ++i) {
      float2 d = split(v[i] + f2(-m));
      d.x = own.in(i, 0) ? d.x : 0.0f, d.y = own.in(i, 1) ? d.y : 0.0f;
      q[i & 1] = fma2(f2(d.x, d.y), f2(d.x, d.y), q[i & 1]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV * 4; ++i) q[i & 1] = fma2(v[i], v[i], q[i & 1]);
  }
  const float2 a = split(q[0] + q[1]);
  s[0] = a.x + a.y;
  group_sums(s, grp);
  r = rsqrtf(fmaf(s[0], inv_d, eps));  // within 2 ulp
}

// vector j of (v - m) r w + c in place
template <int NV, bool LN, bool VEC>
__device__ __forceinline__ void apply_norm(const Own<NV, VEC>& own, const NormParams& p, int j, F2* v, float m, float r,
                                           const void* w, const void* smem_w, const void* c) {
  F2 t[4];
  if (smem_w) own.load(j, smem_w, MOE_DTYPE_FP32, 0.0f, t, true);
  else own.weight(j, w, p.pdt, p.w_off, t);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = (LN ? v[i] + f2(-m) : v[i]) * f2(r) * t[i];
  if (LN && c) {
    own.load(j, c, p.pdt, 0.0f, t);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = v[i] + t[i];
  }
}

// DT: the rows' type where it is known at compile time (stream and branch alike,
// bf16 or fp16: what the instructions of a row are counted for), else -1 and the
// types are looked at for every vector.
template <int NV, bool LN, int DT, bool VEC>
__global__ void __launch_bounds__(norm_fwd_threads(NV)) norm_fwd_kernel(const NormParams p) {
  constexpr int N = NV * 4;
  const int sdt = DT < 0 ? p.sdt : DT, bdt = DT < 0 ? p.bdt : DT;
  extern __shared__ __align__(16) char smem[];
  __shared__ float red[16 * 2 * 2 * NORM_MAX_WARPS];  // of groups of two warps and more
  const int g = threadIdx.x / p.group, groups = blockDim.x / p.group;
  const Own<NV, VEC> own{p.group, (int)threadIdx.x - g * p.group, p.D, p.nvec};
  Group grp{red + (g & 15) * (2 * 2 * NORM_MAX_WARPS), g, p.group >> 5, own.tid >> 5, 0};
  grid_dependency_wait();
  const Ring<NV> ring{smem + g * p.stages * p.stage_bytes, p.stage_bytes,
                      {0, p.x ? p.D * esize(sdt) : 0, (p.x ? p.D * esize(sdt) : 0) + (p.o ? p.D * esize(bdt) : 0), 0}};
  const int64_t step = (int64_t)groups * gridDim.x;
  int64_t row = (int64_t)g * gridDim.x + blockIdx.x;
  auto fetch_o = [&](int64_t r, int stage) {
    if constexpr (VEC) {
      if (p.stages && p.o && r < p.T) ring.fetch(own, stage, 1, row_at(p.o, r, p.o_ld, bdt), bdt);
      cp_async_commit();
    }
  };
  auto fetch_x = [&](int64_t r, int stage) {
    if constexpr (VEC) {
      if (p.stages && r < p.T) {
        if (p.x) ring.fetch(own, stage, 0, row_at(p.x, r, p.x_ld, sdt), sdt);
        if (p.gate_rows) ring.fetch(own, stage, 2, row_at(p.gate, r, p.gate_ld, bdt), bdt);
      }
      cp_async_commit();
    }
  };
  for (int s = 0; s < p.stages; ++s) {
    fetch_o(row + s * step, s);
    fetch_x(row + s * step, s);
  }
  // the norms' weights as fp32, once per CTA, where it has enough rows
  float *sw1 = nullptr, *sw2 = nullptr;
  if (VEC && p.smem_w) {
    float* w = reinterpret_cast<float*>(smem + groups * p.stages * p.stage_bytes);
    #pragma unroll 1
    for (int k = 0; k < 2; ++k) {
      if (!(k ? p.pre : p.post)) continue;
      const void* from = k ? p.w2 : p.w1;
      for (int i = threadIdx.x; i < p.nvec; i += blockDim.x) {
        F2 v[4] = {f2(1.0f), f2(1.0f), f2(1.0f), f2(1.0f)};
        if (from) {
          norm_load8(static_cast<const char*>(from) + (size_t)i * 8 * esize(p.pdt), p.pdt, v);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = v[e] + f2(p.w_off);
        }
        const float2 a = split(v[0]), b = split(v[1]), c = split(v[2]), d = split(v[3]);
        reinterpret_cast<float4*>(w)[i] = make_float4(a.x, a.y, b.x, b.y);
        reinterpret_cast<float4*>(w)[p.nvec + i] = make_float4(c.x, c.y, d.x, d.y);
      }
      (k ? sw2 : sw1) = w;
      w += p.D;
    }
    __syncthreads();
  }
  int stage = 0;
  const int64_t ahead = step * p.stages;
  // vector j of a row of tensor t
  auto take = [&](int j, int t, const void* global, int dt, F2* v) {
    if constexpr (VEC) {
      if (p.stages) {
        own.load(j, ring.row(stage, t), dt, 0.0f, v, true);
        return;
      }
    }
    own.load(j, global, dt, 0.0f, v);
  };
  for (; row < p.T; row += step) {
    float4 st = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    F2 v[N];
    if (VEC) cp_async_wait(2 * p.stages - 1);  // o
    const void* o = row_at(p.o, row, p.o_ld, bdt);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (p.o) {
        take(j, 1, o, bdt, v + 4 * j);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 * j + i] = f2(0.0f);
      }
    }
    if (p.post) {
      row_stats<NV, LN, VEC>(own, v, p.inv_d, p.eps, grp, st.x, st.y);
      fetch_o(row + ahead, stage);  // the sums have used every element of o
    }
    if (VEC) cp_async_wait(2 * p.stages - (p.post ? 1 : 2));  // x and the gate
    const void *x = row_at(p.x, row, p.x_ld, sdt), *gate = p.gate_rows ? row_at(p.gate, row, p.gate_ld, bdt) : p.gate;
    void* y = row_at(p.y, row, p.y_ld, sdt);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      F2 t[4], *w = v + 4 * j;
      if (p.post) apply_norm<NV, LN, VEC>(own, p, j, w, st.x, st.y, p.w1, sw1, p.c1);
      if (p.gate) {
        if (p.gate_rows) take(j, 2, gate, bdt, t);
        else own.load(j, gate, p.pdt, 0.0f, t);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = w[i] * t[i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = w[i] * f2(p.o_scale);
      if (p.x) {
        take(j, 0, x, sdt, t);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = fma2(f2(p.x_scale), t[i], w[i]);
      }
      own.store(j, y, sdt, w);
    }
    if (p.pre) row_stats<NV, LN, VEC>(own, v, p.inv_d, p.eps, grp, st.z, st.w);
    if (!p.post) fetch_o(row + ahead, stage);
    fetch_x(row + ahead, stage);
    if (p.pre) {
      void* h = row_at(p.h, row, p.h_ld, bdt);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        apply_norm<NV, LN, VEC>(own, p, j, v + 4 * j, st.z, st.w, p.w2, sw2, p.c2);
        own.store(j, h, bdt, v + 4 * j);
      }
    }
    if (p.stats && own.tid == 0) {
      float* s = p.stats + 4 * row;
      s[0] = st.x, s[1] = st.y, s[2] = st.z, s[3] = st.w;
    }
    stage = stage + 1 >= p.stages ? 0 : stage + 1;
  }
}

// Backward of one norm, first half: from the gradient d of its output and the
// normalised input n, the sums for dw and dc, u = d w in d, and the row's sums.
template <int NV, bool LN, bool KEEP>
__device__ __forceinline__ void norm_back_sums(F2 (&d)[NV * 4], const F2 (&n)[NV * 4], const F2 (&kept)[KEEP ? NV * 4 : 1],
                                               const F2 (&now)[KEEP ? 1 : NV * 4], F2 (&aw)[NV * 4],
                                               F2 (&ac)[LN ? NV * 4 : 1], float inv_d, Group& grp, float& c, float& m) {
  F2 q[2] = {f2(0.0f), f2(0.0f)}, e = f2(0.0f);
#pragma unroll
  for (int i = 0; i < NV * 4; ++i) {
    aw[i] = fma2(d[i], n[i], aw[i]);
    if constexpr (LN) ac[i] = ac[i] + d[i];
    d[i] = d[i] * (KEEP ? kept[KEEP ? i : 0] : now[KEEP ? 0 : i]);
    q[i & 1] = fma2(d[i], n[i], q[i & 1]);
    if constexpr (LN) e = e + d[i];
  }
  const float2 a = split(q[0] + q[1]), b = split(e);
  if constexpr (LN) {
    float s[2] = {a.x + a.y, b.x + b.y};
    group_sums(s, grp);
    c = s[0] * inv_d, m = s[1] * inv_d;
  } else {
    float s[1] = {a.x + a.y};
    group_sums(s, grp);
    c = s[0] * inv_d, m = 0.0f;
  }
}

// Sums over the rows are kept per thread for its own columns and leave the CTA
// once, at the end (norm_sums_kernel adds the CTAs in order).
template <int NV, bool LN, bool GATE, int DT, bool VEC>
__global__ void __launch_bounds__(512) norm_bwd_kernel(const NormParams p) {
  constexpr int N = NV * 4;
  const int sdt = DT < 0 ? p.sdt : DT, bdt = DT < 0 ? p.bdt : DT;
  constexpr bool KEEP = NV <= 2;
  extern __shared__ __align__(16) char smem[];
  __shared__ float red[2 * 2 * NORM_MAX_WARPS];
  const Own<NV, VEC> own{(int)blockDim.x, (int)threadIdx.x, p.D, p.nvec};
  Group grp{red, 1, (int)blockDim.x >> 5, (int)threadIdx.x >> 5, 0};
  grid_dependency_wait();
  Ring<NV> ring{smem, p.stage_bytes, {0, 0, 0, 0}};
  // order in the ring: y, dh, dy, o; the gate's rows are read when they are needed
  ring.off[1] = p.pre ? p.D * esize(sdt) : 0;
  ring.off[2] = ring.off[1] + (p.pre ? p.D * esize(bdt) : 0);
  ring.off[3] = ring.off[2] + (p.dy ? p.D * esize(sdt) : 0);
  auto fetch = [&](int64_t row, int stage) {
    if constexpr (VEC) {
      if (p.stages && row < p.T) {
        if (p.pre) ring.fetch(own, stage, 0, row_at(p.y, row, p.y_ld, sdt), sdt);
        if (p.pre) ring.fetch(own, stage, 1, row_at(p.dh, row, p.dh_ld, bdt), bdt);
        if (p.dy) ring.fetch(own, stage, 2, row_at(p.dy, row, p.dy_ld, sdt), sdt);
        if (p.o) ring.fetch(own, stage, 3, row_at(p.o, row, p.o_ld, bdt), bdt);
      }
      cp_async_commit();
    }
  };
  int64_t row = blockIdx.x;
  for (int s = 0; s + 1 < p.stages; ++s) fetch(row + (int64_t)s * gridDim.x, s);
  F2 w1[KEEP ? N : 1], w2[KEEP ? N : 1];
  if constexpr (KEEP) {
    if (p.post) own.weight(p.w1, p.pdt, p.w_off, w1);
    if (p.pre) own.weight(p.w2, p.pdt, p.w_off, w2);
  }
  F2 aw1[N], aw2[N], ac1[LN ? N : 1], ac2[LN ? N : 1], ag[GATE ? N : 1];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    aw1[i] = aw2[i] = f2(0.0f);
    if constexpr (LN) ac1[i] = ac2[i] = f2(0.0f);
    if constexpr (GATE) ag[i] = f2(0.0f);
  }
  int stage = 0;
  auto take = [&](int t, const void* global, int dt, float none, F2 (&v)[N]) {
    if constexpr (VEC) {
      if (p.stages) {
        own.load(ring.row(stage, t), dt, none, v, true);
        return;
      }
    }
    own.load(global, dt, none, v);
  };
  for (; row < p.T; row += gridDim.x) {
    if (VEC && p.stages) {
      int next = stage + p.stages - 1;
      next = next >= p.stages ? next - p.stages : next;
      fetch(row + (int64_t)(p.stages - 1) * gridDim.x, next);
      cp_async_wait(p.stages - 1);
    }
    float4 st = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (p.stats) {
      const float* sp = p.stats + 4 * row;
      st = make_float4(sp[0], sp[1], sp[2], sp[3]);
    }
    F2 d[N], n[N], now[KEEP ? 1 : N];
    float c, m;
    if (p.pre) {
      F2 u[N];
      take(0, row_at((const void*)p.y, row, p.y_ld, sdt), sdt, st.z, n);
      take(1, row_at(p.dh, row, p.dh_ld, bdt), bdt, 0.0f, u);
#pragma unroll
      for (int i = 0; i < N; ++i) n[i] = (LN ? n[i] + f2(-st.z) : n[i]) * f2(st.w);
      if constexpr (!KEEP) own.weight(p.w2, p.pdt, p.w_off, now);
      norm_back_sums<NV, LN, KEEP>(u, n, w2, now, aw2, ac2, p.inv_d, grp, c, m);
#pragma unroll
      for (int i = 0; i < N; ++i) u[i] = fma2(n[i], f2(-c), LN ? u[i] + f2(-m) : u[i]);
      if (p.dy) {
        take(2, row_at(p.dy, row, p.dy_ld, sdt), sdt, 0.0f, d);
#pragma unroll
        for (int i = 0; i < N; ++i) d[i] = fma2(f2(st.w), u[i], d[i]);
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) d[i] = f2(st.w) * u[i];
      }
    } else {
      take(2, row_at(p.dy, row, p.dy_ld, sdt), sdt, 0.0f, d);
    }
    if (p.dx) {
#pragma unroll
      for (int i = 0; i < N; ++i) n[i] = f2(p.x_scale) * d[i];
      own.store(row_at(p.dx, row, p.dx_ld, sdt), sdt, n);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] = d[i] * f2(p.o_scale);
    if (p.o) {
      take(3, row_at(p.o, row, p.o_ld, bdt), bdt, p.post ? st.x : 0.0f, n);
      if (p.post)
#pragma unroll
        for (int i = 0; i < N; ++i) n[i] = (LN ? n[i] + f2(-st.x) : n[i]) * f2(st.y);
    }
    if constexpr (!KEEP) {
      if (p.post) own.weight(p.w1, p.pdt, p.w_off, now);
    }
    if (p.gate) {
      F2 g[N];
      if (GATE || p.dgate) {  // z again, from the normalised output
        F2 z[N];
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] = p.post ? n[i] * (KEEP ? w1[KEEP ? i : 0] : now[KEEP ? 0 : i]) : n[i];
        if (LN && p.post && p.c1) {
          own.load(p.c1, p.pdt, 0.0f, g);
#pragma unroll
          for (int i = 0; i < N; ++i) z[i] = z[i] + g[i];
        }
        if constexpr (GATE) {
#pragma unroll
          for (int i = 0; i < N; ++i) ag[i] = fma2(d[i], z[i], ag[i]);
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i) z[i] = z[i] * d[i];
          own.store(row_at(p.dgate, row, p.dgate_ld, bdt), bdt, z);
        }
      }
      if (p.gate_rows) own.load(row_at(p.gate, row, p.gate_ld, bdt), bdt, 0.0f, g);
      else own.load(p.gate, p.pdt, 0.0f, g);
#pragma unroll
      for (int i = 0; i < N; ++i) d[i] = d[i] * g[i];
    }
    if (p.post) {
      norm_back_sums<NV, LN, KEEP>(d, n, w1, now, aw1, ac1, p.inv_d, grp, c, m);
#pragma unroll
      for (int i = 0; i < N; ++i) d[i] = f2(st.y) * fma2(n[i], f2(-c), LN ? d[i] + f2(-m) : d[i]);
    }
    if (p.d_o) own.store(row_at(p.d_o, row, p.do_ld, bdt), bdt, d);
    stage = stage + 1 >= p.stages ? 0 : stage + 1;
  }
  if (!p.sums) return;
  auto leave = [&](int which, F2 (&a)[N]) {
    own.store(p.sums + ((size_t)blockIdx.x * NORM_SUMS + which) * p.D, MOE_DTYPE_FP32, a);
  };
  leave(0, aw1);
  leave(2, aw2);
  if constexpr (LN) {
    leave(1, ac1);
    leave(3, ac2);
  }
  if constexpr (GATE) leave(4, ag);
}

struct NormSums {
  const float* part;
  float* out[NORM_SUMS];
  int ctas, D;
};
// One CTA per 32 columns of one sum: 32 warps' worth of CTAs' partial sums in
// parallel (warp w those of CTAs w, w + 8, ...), then the 8 in order.
__global__ void __launch_bounds__(256) norm_sums_kernel(const NormSums p) {
  __shared__ float part[8][32];
  grid_dependency_wait();
  float* out = p.out[blockIdx.y];
  if (!out) return;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (col < p.D)
    for (int c = w; c < p.ctas; c += 8) s += p.part[((size_t)c * NORM_SUMS + blockIdx.y) * p.D + col];
  part[w][lane] = s;
  __syncthreads();
  if (w == 0 && col < p.D) {
    float t = part[0][lane];
#pragma unroll
    for (int i = 1; i < 8; ++i) t += part[i][lane];
    out[col] = t;
  }
}

}  // namespace moe

// ------------------------------------------------------------------ C ABI
using namespace moe;

struct moe_norm_plan {
  moe_norm_config cfg;
  int device, num_sms;
};

namespace {

size_t norm_size(int d) { return d == MOE_DTYPE_FP32 ? 4 : 2; }
bool norm_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Vectors of 8 that a thread owns, by the row's width, and the threads that share
// a row.  Forward: as few threads as hold the row in registers, since what a
// thread does besides its elements (sums, addresses, barriers) costs as much as
// 16 of them: 16384 x 7168 with 1 / 2 / 8 vectors a thread: FWDCOST.
// Backward: the sums for its columns are in registers too, so 2 (4 past 8192).
int norm_nv(int64_t D) { return D <= 8192 ? 2 : 4; }
int norm_threads(int64_t D) {
  const int64_t per = 8 * norm_nv(D);
  return (int)(((D + per - 1) / per + 31) / 32 * 32);
}
// The backward's CTAs (resident by threads and registers; rows are handed out evenly)
int64_t norm_grid(const moe_norm_plan* pl, int64_t T) {
  int64_t per_sm = 512 / norm_threads(pl->cfg.D);
  per_sm = per_sm < 1 ? 1 : per_sm > 16 ? 16 : per_sm;
  const int64_t most = per_sm * pl->num_sms;
  return T < most ? T : most;
}
constexpr int NORM_SMEM = 200 * 1024;  // of an SM's shared memory for the rings

// The rows' type where it has kernels of its own
template <typename F>
cudaError_t norm_by_type(const moe_norm_config& c, F&& f) {
  if (c.stream_dtype == MOE_DTYPE_BF16) return f(std::integral_constant<int, MOE_DTYPE_BF16>{});
  if (c.stream_dtype == MOE_DTYPE_FP16) return f(std::integral_constant<int, MOE_DTYPE_FP16>{});
  return f(std::integral_constant<int, -1>{});
}

template <typename P>
cudaError_t norm_launch(void (*kernel)(P), dim3 grid, unsigned threads, size_t smem, cudaStream_t st, const P& p) {
  if (smem > 40 * 1024) {  // 48 KB with what the kernel holds besides
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
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

// A row tensor of a call: elements aligned, strides in range
bool norm_rows_ok(const void* p, int64_t& ld, int64_t D, int dt, int64_t T) {
  if (ld == 0) ld = D;
  if (!p) return true;
  return ld >= D && ld <= (int64_t)1 << 40 && norm_aligned(p, norm_size(dt)) && T <= ((int64_t)1 << 60) / ld;
}
bool norm_rows_vec(const void* p, int64_t ld, int dt) {
  return !p || (norm_aligned(p, 16) && ld * (int64_t)norm_size(dt) % 16 == 0);
}

int norm_params(const moe_norm_plan* pl, const moe_norm_params* q, int64_t T, NormParams& p, bool& vec) {
  const moe_norm_config& c = pl->cfg;
  p.T = T;
  p.D = (int)c.D;
  p.nvec = (int)((c.D + 7) / 8);
  p.post = c.post;
  p.pre = c.pre;
  p.sdt = c.stream_dtype;
  p.bdt = c.branch_dtype;
  p.pdt = c.param_dtype;
  p.inv_d = 1.0f / (float)c.D;
  p.eps = c.eps;
  p.w_off = c.weight_offset;
  p.x_scale = c.x_scale;
  p.o_scale = c.o_scale;
  vec = c.D % 8 == 0;
  if (!q) return MOE_OK;
  p.w1 = c.post ? q->post_weight : nullptr;
  p.c1 = c.post ? q->post_bias : nullptr;
  p.w2 = c.pre ? q->pre_weight : nullptr;
  p.c2 = c.pre ? q->pre_bias : nullptr;
  if (c.kind != MOE_NORM_LAYER && (q->post_bias || q->pre_bias)) return MOE_ERR_INVALID_ARG;
  p.gate = q->gate;
  p.gate_rows = q->gate && q->gate_stride != 0;
  p.gate_ld = q->gate_stride;
  const size_t ps = norm_size(c.param_dtype);
  for (const void* v : {p.w1, p.c1, p.w2, p.c2, p.gate_rows ? nullptr : p.gate}) {
    if (!norm_aligned(v, ps)) return MOE_ERR_INVALID_ARG;
    vec = vec && norm_aligned(v, 16);
  }
  if (p.gate_rows) {
    if (!norm_rows_ok(p.gate, p.gate_ld, c.D, c.branch_dtype, T)) return MOE_ERR_INVALID_ARG;
    vec = vec && norm_rows_vec(p.gate, p.gate_ld, c.branch_dtype);
  }
  return MOE_OK;
}

// Rows of the ring that fit with `per_sm` CTAs on an SM, up to four
void norm_ring(const moe_norm_plan* pl, NormParams& p, int64_t grid, size_t row_bytes, size_t& smem) {
  const int64_t per_sm = (grid + pl->num_sms - 1) / pl->num_sms;
  const int64_t fit = NORM_SMEM / (per_sm * (int64_t)row_bytes);
  p.stages = (int)(fit < 1 ? 0 : fit > 4 ? 4 : fit);  // 0: rows too long for it, loaded when they are needed
  const int64_t rows = (p.T + grid - 1) / grid;  // of a CTA
  if (p.stages > rows) p.stages = (int)rows;
  p.stage_bytes = (int)row_bytes;
  smem = (size_t)p.stages * row_bytes;
}

bool norm_on_device(const moe_norm_plan* pl) {
  int cur = -1;
  return cudaGetDevice(&cur) == cudaSuccess && cur == pl->device;
}
bool finite(float v) { return v - v == 0.0f; }

}  // namespace

extern "C" {

int moe_norm_plan_create(const moe_norm_config* cfg, moe_norm_plan** out) {
  if (!cfg || !out) return MOE_ERR_INVALID_ARG;
  *out = nullptr;
  const moe_norm_config& c = *cfg;
  if (c.kind != MOE_NORM_RMS && c.kind != MOE_NORM_LAYER) return MOE_ERR_INVALID_ARG;
  if ((c.post | c.pre) & ~1) return MOE_ERR_INVALID_ARG;
  for (int d : {c.stream_dtype, c.branch_dtype, c.param_dtype})
    if (d < MOE_DTYPE_FP32 || d > MOE_DTYPE_FP16) return MOE_ERR_INVALID_ARG;
  if (c.stream_dtype != MOE_DTYPE_FP32 && c.branch_dtype != c.stream_dtype) return MOE_ERR_INVALID_ARG;
  if (!(c.eps > 0.0f) || !finite(c.eps) || !finite(c.weight_offset) || !finite(c.x_scale) || !finite(c.o_scale))
    return MOE_ERR_INVALID_ARG;
  if (c.D < 1 || c.D > NORM_MAX_D) return MOE_ERR_UNSUPPORTED_SHAPE;
  int dev = 0, sms = 0, major = 0, minor = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
    return MOE_ERR_CUDA;
  if (major != 10 || minor != 3) return MOE_ERR_UNSUPPORTED_DEVICE;
  moe_norm_plan* pl = new (std::nothrow) moe_norm_plan;
  if (!pl) return MOE_ERR_INVALID_ARG;
  pl->cfg = c;
  pl->device = dev;
  pl->num_sms = sms;
  *out = pl;
  return MOE_OK;
}

int moe_norm_plan_destroy(moe_norm_plan* plan) {
  delete plan;
  return MOE_OK;
}

int moe_norm(const moe_norm_plan* pl, int64_t T, const moe_norm_params* params, const void* x, int64_t x_stride,
             const void* o, int64_t o_stride, void* y, int64_t y_stride, void* h, int64_t h_stride, float* stats,
             moe_stream_t stream) {
  if (!pl || T < 0) return MOE_ERR_INVALID_ARG;
  const moe_norm_config& c = pl->cfg;
  NormParams p{};
  bool vec = false;
  const int rc = norm_params(pl, params, T, p, vec);
  if (rc != MOE_OK) return rc;
  if (!norm_rows_ok(x, x_stride, c.D, c.stream_dtype, T) || !norm_rows_ok(y, y_stride, c.D, c.stream_dtype, T) ||
      !norm_rows_ok(o, o_stride, c.D, c.branch_dtype, T) || !norm_rows_ok(h, h_stride, c.D, c.branch_dtype, T) ||
      !norm_aligned(stats, 4))
    return MOE_ERR_INVALID_ARG;
  if (T > 0) {
    if ((!x && !o) || (!o && (c.post || p.gate)) || (c.pre ? !h : (!y || h))) return MOE_ERR_INVALID_ARG;
  }
  if (!norm_on_device(pl)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  vec = vec && norm_rows_vec(x, x_stride, c.stream_dtype) && norm_rows_vec(y, y_stride, c.stream_dtype) &&
        norm_rows_vec(o, o_stride, c.branch_dtype) && norm_rows_vec(h, h_stride, c.branch_dtype);
  p.x = x, p.x_ld = x_stride;
  p.o = o, p.o_ld = o_stride;
  p.y = y, p.y_ld = y_stride;
  p.h = h, p.h_ld = h_stride;
  p.stats = stats;
  // rows at a time on a CTA: 16 warps' worth, fewer where the rows' ring or the
  // batch do not ask for them
  p.group = norm_threads(c.D);
  const int64_t row_bytes = c.D * ((x ? norm_size(c.stream_dtype) : 0) + (o ? norm_size(c.branch_dtype) : 0) +
                                   (p.gate_rows ? norm_size(c.branch_dtype) : 0));
  const int64_t w_bytes = c.D * 4 * (c.post + c.pre);
  int64_t rows = norm_fwd_threads(norm_nv(c.D)) / p.group, need = (T + pl->num_sms - 1) / pl->num_sms;
  rows = rows < need ? rows : need;
  p.smem_w = vec && need >= 2 * rows;
  while (rows > 1 && rows * row_bytes + p.smem_w * w_bytes > NORM_SMEM) --rows;
  if (rows * row_bytes + p.smem_w * w_bytes > NORM_SMEM) p.smem_w = 0;
  if (vec) {  // rows ahead that fit, up to three; none where one row does not
    int64_t fit = (NORM_SMEM - p.smem_w * w_bytes) / (rows * row_bytes);
    const int64_t use = (need + rows - 1) / rows;
    fit = fit < use ? fit : use;
    p.stages = (int)(fit < 3 ? fit : 3);
  }
  p.stage_bytes = p.stages ? (int)row_bytes : 0;
  const size_t smem = rows * p.stages * p.stage_bytes + p.smem_w * w_bytes;
  const int64_t ctas = (T + rows - 1) / rows, grid = ctas < pl->num_sms ? ctas : pl->num_sms;
  const unsigned nt = (unsigned)(rows * p.group);
  auto by_kind = [&](auto nv) {
    return norm_by_type(c, [&](auto dt) {
      constexpr int NV = decltype(nv)::value, DT = decltype(dt)::value;
      auto kernel = c.kind == MOE_NORM_LAYER ? (vec ? norm_fwd_kernel<NV, true, DT, true> : norm_fwd_kernel<NV, true, DT, false>)
                                             : (vec ? norm_fwd_kernel<NV, false, DT, true> : norm_fwd_kernel<NV, false, DT, false>);
      return norm_launch(kernel, dim3((unsigned)grid), nt, smem, (cudaStream_t)stream, p);
    });
  };
  const int nv = norm_nv(c.D);
  const cudaError_t err = nv == 2 ? by_kind(std::integral_constant<int, 2>{}) : by_kind(std::integral_constant<int, 4>{});
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

size_t moe_norm_workspace_bytes(const moe_norm_plan* plan, int64_t T) {
  if (!plan || T < 0) return 0;
  if (T == 0) return 256;
  return ((size_t)norm_grid(plan, T) * NORM_SUMS * plan->cfg.D * 4 + 255) / 256 * 256;
}

int moe_norm_bwd(const moe_norm_plan* pl, int64_t T, const moe_norm_params* params, const float* stats, const void* o,
                 int64_t o_stride, const void* y, int64_t y_stride, const void* dy, int64_t dy_stride, const void* dh,
                 int64_t dh_stride, void* dx, int64_t dx_stride, void* d_o, int64_t d_o_stride,
                 const moe_norm_grads* grads, void* workspace, size_t workspace_bytes, moe_stream_t stream_) {
  if (!pl || T < 0) return MOE_ERR_INVALID_ARG;
  const moe_norm_config& c = pl->cfg;
  cudaStream_t stream = (cudaStream_t)stream_;
  NormParams p{};
  bool vec = false;
  const int rc = norm_params(pl, params, T, p, vec);
  if (rc != MOE_OK) return rc;
  const int sd = c.stream_dtype, bd = c.branch_dtype;
  if (!norm_rows_ok(o, o_stride, c.D, bd, T) || !norm_rows_ok(y, y_stride, c.D, sd, T) ||
      !norm_rows_ok(dy, dy_stride, c.D, sd, T) || !norm_rows_ok(dh, dh_stride, c.D, bd, T) ||
      !norm_rows_ok(dx, dx_stride, c.D, sd, T) || !norm_rows_ok(d_o, d_o_stride, c.D, bd, T) || !norm_aligned(stats, 4))
    return MOE_ERR_INVALID_ARG;
  NormSums s{};
  bool gate_sum = false;
  int64_t dgate_ld = c.D;
  if (grads) {
    if ((!c.post && (grads->post_weight || grads->post_bias)) || (!c.pre && (grads->pre_weight || grads->pre_bias)) ||
        (c.kind != MOE_NORM_LAYER && (grads->post_bias || grads->pre_bias)) || (grads->gate && !p.gate))
      return MOE_ERR_INVALID_ARG;
    s.out[0] = grads->post_weight, s.out[1] = grads->post_bias;
    s.out[2] = grads->pre_weight, s.out[3] = grads->pre_bias;
    if (grads->gate && !p.gate_rows) s.out[4] = static_cast<float*>(grads->gate), gate_sum = true;
    for (const float* v : s.out)
      if (!norm_aligned(v, 4)) return MOE_ERR_INVALID_ARG;
    if (p.gate_rows) {
      dgate_ld = grads->gate_stride;
      if (!norm_rows_ok(grads->gate, dgate_ld, c.D, bd, T)) return MOE_ERR_INVALID_ARG;
      p.dgate = grads->gate, p.dgate_ld = dgate_ld;
    }
  }
  const bool sums = s.out[0] || s.out[1] || s.out[2] || s.out[3] || s.out[4];
  if (T > 0) {
    if (c.pre ? (!y || !dh) : !dy) return MOE_ERR_INVALID_ARG;
    if ((c.post || gate_sum || p.dgate) && !o) return MOE_ERR_INVALID_ARG;
    if ((c.post || c.pre) && !stats) return MOE_ERR_INVALID_ARG;
    if (sums) {
      if (!workspace || !norm_aligned(workspace, 256)) return MOE_ERR_INVALID_ARG;
      if (workspace_bytes < moe_norm_workspace_bytes(pl, T)) return MOE_ERR_WORKSPACE_TOO_SMALL;
    }
  }
  if (!norm_on_device(pl)) return MOE_ERR_INVALID_ARG;
  if (T == 0) {
    for (float* v : s.out)
      if (v && cudaMemsetAsync(v, 0, 4 * (size_t)c.D, stream) != cudaSuccess) return MOE_ERR_CUDA;
    return MOE_OK;
  }
  const bool use_o = c.post || gate_sum || p.dgate;
  vec = vec && (!use_o || norm_rows_vec(o, o_stride, bd)) && (!c.pre || (norm_rows_vec(y, y_stride, sd) && norm_rows_vec(dh, dh_stride, bd))) &&
        norm_rows_vec(dy, dy_stride, sd) && norm_rows_vec(dx, dx_stride, sd) && norm_rows_vec(d_o, d_o_stride, bd) &&
        norm_rows_vec(p.dgate, p.dgate_ld, bd);
  p.o = use_o ? o : nullptr, p.o_ld = o_stride;
  p.y = const_cast<void*>(y), p.y_ld = y_stride;
  p.dy = dy, p.dy_ld = dy_stride;
  p.dh = dh, p.dh_ld = dh_stride;
  p.dx = dx, p.dx_ld = dx_stride;
  p.d_o = d_o, p.do_ld = d_o_stride;
  p.stats = const_cast<float*>(stats);
  p.sums = sums ? static_cast<float*>(workspace) : nullptr;
  const int64_t grid = norm_grid(pl, T);
  size_t smem = 0;
  if (vec)
    norm_ring(pl, p, grid, (size_t)c.D * ((c.pre ? norm_size(sd) + norm_size(bd) : 0) + (dy ? norm_size(sd) : 0) +
                                          (use_o ? norm_size(bd) : 0)), smem);
  const unsigned nt = (unsigned)norm_threads(c.D);
  auto go = [&](auto nv, auto dt, auto v) {
    constexpr int NV = decltype(nv)::value, DT = decltype(dt)::value;
    constexpr bool V = decltype(v)::value;
    auto kernel = c.kind == MOE_NORM_LAYER
                      ? (gate_sum ? norm_bwd_kernel<NV, true, true, DT, V> : norm_bwd_kernel<NV, true, false, DT, V>)
                      : (gate_sum ? norm_bwd_kernel<NV, false, true, DT, V> : norm_bwd_kernel<NV, false, false, DT, V>);
    return norm_launch(kernel, dim3((unsigned)grid), nt, smem, stream, p);
  };
  constexpr std::integral_constant<int, 2> two{};
  constexpr std::integral_constant<int, 4> four{};
  constexpr std::integral_constant<int, -1> any{};
  const cudaError_t err = norm_nv(c.D) == 4 ? (vec ? go(four, any, std::true_type{}) : go(four, any, std::false_type{}))
                          : vec             ? norm_by_type(c, [&](auto dt) { return go(two, dt, std::true_type{}); })
                                            : go(two, any, std::false_type{});
  if (err != cudaSuccess) return MOE_ERR_CUDA;
  if (sums) {
    s.part = p.sums;
    s.ctas = (int)grid;
    s.D = (int)c.D;
    if (norm_launch(norm_sums_kernel, dim3((unsigned)((c.D + 31) / 32), NORM_SUMS), 256, 0, stream, s) != cudaSuccess)
      return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

}  // extern "C"
