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
constexpr int NORM_MAX_WARPS = 32;
constexpr int NORM_SUMS = 5;  // dw and dc of both norms, dg

struct NormParams {
  int64_t T;
  int D, nvec;     // nvec: vectors of 8 elements in a row
  int post, pre, sdt, bdt, pdt;
  int stages;      // rows in the ring (0: no ring)
  int stage_bytes; // of one row group in the ring
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

// 8 consecutive elements, 16-byte aligned (shared or global memory)
__device__ __forceinline__ void norm_load8(const void* p, int dt, float* v) {
  if (dt == MOE_DTYPE_FP32) {
    const float4 a = static_cast<const float4*>(p)[0], b = static_cast<const float4*>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    return;
  }
  const uint4 q = *static_cast<const uint4*>(p);
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  if (dt == MOE_DTYPE_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
  }
}
// 8 elements rounded to dt and stored (16-byte aligned); v holds what was stored
template <bool kStore = true>
__device__ __forceinline__ void norm_store8(void* p, int dt, float* v) {
  if (dt == MOE_DTYPE_FP32) {
    if (kStore) {
      static_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
      static_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
    return;
  }
  uint32_t w[4];
  if (dt == MOE_DTYPE_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
      v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
      const float2 f = __half22float2(h);
      v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
  }
  if (kStore) *static_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void cp_async16(void* smem, const void* g) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(smem)), "l"(g) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all but the `n` newest groups of this thread have landed (n up to 3)
__device__ __forceinline__ void cp_async_wait(int n) {
  if (n <= 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
  else if (n == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
  else if (n == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
  else asm volatile("cp.async.wait_group 3;" ::: "memory");
}
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Sums of N values over the CTA, every thread getting the same bits.  `red`
// alternates between two buffers, so that one barrier a call is enough.
template <int N>
__device__ __forceinline__ void cta_sums(float (&v)[N], float* red, int& turn) {
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], m);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return;
  float* r = red + (turn & 1) * (4 * NORM_MAX_WARPS);
  ++turn;
  if (lane_id() == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) r[i * NORM_MAX_WARPS + (threadIdx.x >> 5)] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float s = 0.0f;
    for (int w = 0; w < warps; ++w) s += r[i * NORM_MAX_WARPS + w];
    v[i] = s;
  }
}

// The elements of a row that a thread owns: with VEC vectors tid + j NT of 8,
// else single elements tid + j NT.
template <int NV, bool VEC>
struct Own {
  int nt, tid, D, nvec;
  __device__ __forceinline__ bool vec_in(int j) const { return tid + j * nt < nvec; }
  __device__ __forceinline__ int at(int j) const { return (tid + j * nt) * 8; }        // first element of vector j
  __device__ __forceinline__ int one(int i) const { return tid + i * nt; }             // element i (not VEC)
  __device__ __forceinline__ bool one_in(int i) const { return tid + i * nt < D; }
  __device__ __forceinline__ bool in(int i) const { return VEC ? vec_in(i / 8) : one_in(i); }

  // from a parameter or a row in global memory; `none` where there is no element
  __device__ __forceinline__ void load(const void* row, int dt, float none, float (&v)[NV * 8]) const {
    if constexpr (VEC) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (vec_in(j)) {
          norm_load8(static_cast<const char*>(row) + (size_t)at(j) * (dt == MOE_DTYPE_FP32 ? 4 : 2), dt, v + 8 * j);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[8 * j + i] = none;
        }
      }
    } else {
      if (dt == MOE_DTYPE_FP32) {
#pragma unroll
        for (int i = 0; i < NV * 8; ++i) v[i] = one_in(i) ? static_cast<const float*>(row)[one(i)] : none;
      } else if (dt == MOE_DTYPE_BF16) {
#pragma unroll
        for (int i = 0; i < NV * 8; ++i) v[i] = one_in(i) ? __bfloat162float(static_cast<const bf16*>(row)[one(i)]) : none;
      } else {
#pragma unroll
        for (int i = 0; i < NV * 8; ++i) v[i] = one_in(i) ? __half2float(static_cast<const __half*>(row)[one(i)]) : none;
      }
    }
  }
  // round to dt, store unless row is null; v holds the rounded values
  __device__ __forceinline__ void store(void* row, int dt, float (&v)[NV * 8]) const {
    if constexpr (VEC) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (row && vec_in(j)) norm_store8(static_cast<char*>(row) + (size_t)at(j) * (dt == MOE_DTYPE_FP32 ? 4 : 2), dt, v + 8 * j);
        else norm_store8<false>(nullptr, dt, v + 8 * j);
      }
    } else {
      if (dt == MOE_DTYPE_FP32) {
#pragma unroll
        for (int i = 0; i < NV * 8; ++i)
          if (row && one_in(i)) static_cast<float*>(row)[one(i)] = v[i];
      } else if (dt == MOE_DTYPE_BF16) {
#pragma unroll
        for (int i = 0; i < NV * 8; ++i) {
          const bf16 w = __float2bfloat16_rn(v[i]);
          if (row && one_in(i)) static_cast<bf16*>(row)[one(i)] = w;
          v[i] = __bfloat162float(w);
        }
      } else {
#pragma unroll
        for (int i = 0; i < NV * 8; ++i) {
          const __half w = __float2half_rn(v[i]);
          if (row && one_in(i)) static_cast<__half*>(row)[one(i)] = w;
          v[i] = __half2float(w);
        }
      }
    }
  }
};

__device__ __forceinline__ size_t esize(int dt) { return dt == MOE_DTYPE_FP32 ? 4 : 2; }
__device__ __forceinline__ const void* row_at(const void* p, int64_t r, int64_t ld, int dt) {
  return static_cast<const char*>(p) + r * ld * (int64_t)esize(dt);
}
__device__ __forceinline__ void* row_at(void* p, int64_t r, int64_t ld, int dt) {
  return static_cast<char*>(p) + r * ld * (int64_t)esize(dt);
}

// Rows of up to four tensors, fetched ahead by the thread that owns them:
// slot (stage, tensor) of the ring holds a row's vectors in their own order.
template <int NV>
struct Ring {
  char* base;
  int stage_bytes, off[4];
  __device__ __forceinline__ void fetch(const Own<NV, true>& own, int stage, int t, const void* row, int dt) const {
    const int vb = 8 * (int)esize(dt);
    char* s = base + stage * stage_bytes + off[t];
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (own.vec_in(j)) {
        const size_t b = (size_t)(own.tid + j * own.nt) * vb;
        cp_async16(s + b, static_cast<const char*>(row) + b);
        if (dt == MOE_DTYPE_FP32) cp_async16(s + b + 16, static_cast<const char*>(row) + b + 16);
      }
  }
  __device__ __forceinline__ const void* row(int stage, int t) const { return base + stage * stage_bytes + off[t]; }
};

// mean (or 0) and 1 / sqrt(mean((v - m)^2) + eps) of one row whose elements
// outside the row are 0 in v; two passes over the registers, so that a large
// mean does not cancel
template <int NV, bool LN, bool VEC>
__device__ __forceinline__ void row_stats(const Own<NV, VEC>& own, const float (&v)[NV * 8], float inv_d, float eps,
                                          float* red, int& turn, float& m, float& r) {
  float s[1] = {0.0f};
  m = 0.0f;
  if constexpr (LN) {
#pragma unroll
    for (int i = 0; i < NV * 8; ++i) s[0] += v[i];
    cta_sums(s, red, turn);
    m = s[0] * inv_d;
    s[0] = 0.0f;
#pragma unroll
    for (int i = 0; i < NV * 8; ++i) {
      const float d = own.in(i) ? v[i] - m : 0.0f;
      s[0] = fmaf(d, d, s[0]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV * 8; ++i) s[0] = fmaf(v[i], v[i], s[0]);
  }
  cta_sums(s, red, turn);
  r = 1.0f / sqrtf(fmaf(s[0], inv_d, eps));
}

template <int NV, bool LN, bool VEC>
__global__ void __launch_bounds__(NV == 4 ? 512 : NV == 2 ? 512 : 256) norm_fwd_kernel(const NormParams p) {
  extern __shared__ __align__(16) char smem[];
  __shared__ float red[2 * 4 * NORM_MAX_WARPS];
  const Own<NV, VEC> own{(int)blockDim.x, (int)threadIdx.x, p.D, p.nvec};
  int turn = 0;
  grid_dependency_wait();
  Ring<NV> ring{smem, p.stage_bytes, {0, 0, 0, 0}};
  ring.off[1] = p.x ? p.D * (int)esize(p.sdt) : 0;
  ring.off[2] = ring.off[1] + (p.o ? p.D * (int)esize(p.bdt) : 0);
  auto fetch = [&](int64_t row, int stage) {
    if constexpr (VEC) {
      if (p.stages && row < p.T) {
        if (p.x) ring.fetch(own, stage, 0, row_at(p.x, row, p.x_ld, p.sdt), p.sdt);
        if (p.o) ring.fetch(own, stage, 1, row_at(p.o, row, p.o_ld, p.bdt), p.bdt);
        if (p.gate_rows) ring.fetch(own, stage, 2, row_at(p.gate, row, p.gate_ld, p.bdt), p.bdt);
      }
      cp_async_commit();
    }
  };
  int64_t row = blockIdx.x;
  for (int s = 0; s + 1 < p.stages; ++s) fetch(row + (int64_t)s * gridDim.x, s);
  // the norms' weights, once per CTA: with the offset, or ones; 0 outside the row, where gradients may
  // be other than 0 (a layer norm's mean)
  constexpr bool KEEP = NV <= 2;
  float w1[KEEP ? NV * 8 : 1], w2[KEEP ? NV * 8 : 1];
  auto weight = [&](const void* w, float (&v)[NV * 8]) {
    if (w) own.load(w, p.pdt, 0.0f, v);
#pragma unroll
    for (int i = 0; i < NV * 8; ++i) v[i] = !own.in(i) ? 0.0f : w ? v[i] + p.w_off : 1.0f;
  };
  if constexpr (KEEP) {
    if (p.post) weight(p.w1, w1);
    if (p.pre) weight(p.w2, w2);
  }
  int stage = 0;
  auto take = [&](int t, const void* global, int dt, float none, float (&v)[NV * 8]) {
    if constexpr (VEC) {
      if (p.stages) {
        own.load(ring.row(stage, t), dt, none, v);
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
    float v[NV * 8], t[NV * 8];
    if (p.o) {
      take(1, row_at(p.o, row, p.o_ld, p.bdt), p.bdt, 0.0f, v);
      if (p.post) {
        row_stats<NV, LN, VEC>(own, v, p.inv_d, p.eps, red, turn, st.x, st.y);
        if constexpr (!KEEP) {
          weight(p.w1, t);
#pragma unroll
          for (int i = 0; i < NV * 8; ++i) v[i] = (v[i] - st.x) * st.y * t[i];
        } else {
#pragma unroll
          for (int i = 0; i < NV * 8; ++i) v[i] = (v[i] - st.x) * st.y * w1[i];
        }
        if (LN && p.c1) {
          own.load(p.c1, p.pdt, 0.0f, t);
#pragma unroll
          for (int i = 0; i < NV * 8; ++i) v[i] += t[i];
        }
      }
      if (p.gate) {
        if (p.gate_rows) take(2, row_at(p.gate, row, p.gate_ld, p.bdt), p.bdt, 0.0f, t);
        else own.load(p.gate, p.pdt, 0.0f, t);
#pragma unroll
        for (int i = 0; i < NV * 8; ++i) v[i] *= t[i];
      }
#pragma unroll
      for (int i = 0; i < NV * 8; ++i) v[i] *= p.o_scale;
    } else {
#pragma unroll
      for (int i = 0; i < NV * 8; ++i) v[i] = 0.0f;
    }
    if (p.x) {
      take(0, row_at(p.x, row, p.x_ld, p.sdt), p.sdt, 0.0f, t);
#pragma unroll
      for (int i = 0; i < NV * 8; ++i) v[i] = fmaf(p.x_scale, t[i], v[i]);
    }
    // elements outside the row: 0 for the sums that follow (a layer norm's bias and mean moved them)
#pragma unroll
    for (int i = 0; i < NV * 8; ++i)
      if (!own.in(i)) v[i] = 0.0f;
    own.store(p.y ? row_at(p.y, row, p.y_ld, p.sdt) : nullptr, p.sdt, v);
    if (p.pre) {
      row_stats<NV, LN, VEC>(own, v, p.inv_d, p.eps, red, turn, st.z, st.w);
      if constexpr (!KEEP) {
        weight(p.w2, t);
#pragma unroll
        for (int i = 0; i < NV * 8; ++i) v[i] = (v[i] - st.z) * st.w * t[i];
      } else {
#pragma unroll
        for (int i = 0; i < NV * 8; ++i) v[i] = (v[i] - st.z) * st.w * w2[i];
      }
      if (LN && p.c2) {
        own.load(p.c2, p.pdt, 0.0f, t);
#pragma unroll
        for (int i = 0; i < NV * 8; ++i) v[i] += t[i];
      }
      own.store(row_at(p.h, row, p.h_ld, p.bdt), p.bdt, v);
    }
    if (p.stats && threadIdx.x == 0) {
      float* s = p.stats + 4 * row;
      s[0] = st.x, s[1] = st.y, s[2] = st.z, s[3] = st.w;
    }
    stage = stage + 1 >= p.stages ? 0 : stage + 1;
  }
}

// Sums over the rows are kept per thread for its own columns and leave the CTA
// once, at the end (norm_sums_kernel adds the CTAs in order).
template <int NV, bool LN, bool VEC, bool GATE>
__global__ void __launch_bounds__(NV == 1 ? 256 : 512) norm_bwd_kernel(const NormParams p) {
  extern __shared__ __align__(16) char smem[];
  __shared__ float red[2 * 4 * NORM_MAX_WARPS];
  const Own<NV, VEC> own{(int)blockDim.x, (int)threadIdx.x, p.D, p.nvec};
  int turn = 0;
  grid_dependency_wait();
  Ring<NV> ring{smem, p.stage_bytes, {0, 0, 0, 0}};
  const bool need_gate_rows = p.gate_rows;
  // order in the ring: y, dh, dy, o; the gate's rows are read when they are needed
  ring.off[1] = p.pre ? p.D * (int)esize(p.sdt) : 0;
  ring.off[2] = ring.off[1] + (p.pre ? p.D * (int)esize(p.bdt) : 0);
  ring.off[3] = ring.off[2] + (p.dy ? p.D * (int)esize(p.sdt) : 0);
  auto fetch = [&](int64_t row, int stage) {
    if constexpr (VEC) {
      if (p.stages && row < p.T) {
        if (p.pre) ring.fetch(own, stage, 0, row_at(p.y, row, p.y_ld, p.sdt), p.sdt);
        if (p.pre) ring.fetch(own, stage, 1, row_at(p.dh, row, p.dh_ld, p.bdt), p.bdt);
        if (p.dy) ring.fetch(own, stage, 2, row_at(p.dy, row, p.dy_ld, p.sdt), p.sdt);
        if (p.o) ring.fetch(own, stage, 3, row_at(p.o, row, p.o_ld, p.bdt), p.bdt);
      }
      cp_async_commit();
    }
  };
  int64_t row = blockIdx.x;
  for (int s = 0; s + 1 < p.stages; ++s) fetch(row + (int64_t)s * gridDim.x, s);
  constexpr bool KEEP = NV <= 2;
  float w1[KEEP ? NV * 8 : 1], w2[KEEP ? NV * 8 : 1];
  auto weight = [&](const void* w, float (&v)[NV * 8]) {
    if (w) own.load(w, p.pdt, 0.0f, v);
#pragma unroll
    for (int i = 0; i < NV * 8; ++i) v[i] = !own.in(i) ? 0.0f : w ? v[i] + p.w_off : 1.0f;
  };
  if constexpr (KEEP) {
    if (p.post) weight(p.w1, w1);
    if (p.pre) weight(p.w2, w2);
  }
  float aw1[NV * 8], aw2[NV * 8], ac1[LN ? NV * 8 : 1], ac2[LN ? NV * 8 : 1], ag[GATE ? NV * 8 : 1];
#pragma unroll
  for (int i = 0; i < NV * 8; ++i) {
    aw1[i] = aw2[i] = 0.0f;
    if constexpr (LN) ac1[i] = ac2[i] = 0.0f;
    if constexpr (GATE) ag[i] = 0.0f;
  }
  int stage = 0;
  auto take = [&](int t, const void* global, int dt, float none, float (&v)[NV * 8]) {
    if constexpr (VEC) {
      if (p.stages) {
        own.load(ring.row(stage, t), dt, none, v);
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
    const float* sp = p.stats + 4 * row;
    const float4 st = make_float4(sp[0], sp[1], sp[2], sp[3]);
    float d[NV * 8], n[NV * 8], t[NV * 8];
    if (p.dy) {
      take(2, row_at(p.dy, row, p.dy_ld, p.sdt), p.sdt, 0.0f, d);
    } else {
#pragma unroll
      for (int i = 0; i < NV * 8; ++i) d[i] = 0.0f;
    }
    if (p.pre) {
      float u[NV * 8], s[2] = {0.0f, 0.0f};
      take(0, row_at(p.y, row, p.y_ld, p.sdt), p.sdt, st.z, n);
      take(1, row_at(p.dh, row, p.dh_ld, p.bdt), p.bdt, 0.0f, u);
      if constexpr (!KEEP) weight(p.w2, t);
#pragma unroll
      for (int i = 0; i < NV * 8; ++i) {
        n[i] = (n[i] - st.z) * st.w;
        aw2[i] = fmaf(u[i], n[i], aw2[i]);
        if constexpr (LN) ac2[i] += u[i];
        u[i] *= KEEP ? w2[KEEP ? i : 0] : t[i];
        s[0] = fmaf(u[i], n[i], s[0]);
        if constexpr (LN) s[1] += u[i];
      }
      if constexpr (LN) {
        cta_sums(s, red, turn);
      } else {
        float s1[1] = {s[0]};
        cta_sums(s1, red, turn);
        s[0] = s1[0];
      }
      const float c = s[0] * p.inv_d, m = LN ? s[1] * p.inv_d : 0.0f;
#pragma unroll
      for (int i = 0; i < NV * 8; ++i) d[i] = fmaf(st.w, LN ? fmaf(-n[i], c, u[i]) - m : fmaf(-n[i], c, u[i]), d[i]);
    }
    if (p.dx) {
#pragma unroll
      for (int i = 0; i < NV * 8; ++i) t[i] = p.x_scale * d[i];
      own.store(row_at(p.dx, row, p.dx_ld, p.sdt), p.sdt, t);
    }
#pragma unroll
    for (int i = 0; i < NV * 8; ++i) d[i] *= p.o_scale;
    if (p.o) {
      take(3, row_at(p.o, row, p.o_ld, p.bdt), p.bdt, p.post ? st.x : 0.0f, n);
      if (p.post)
#pragma unroll
        for (int i = 0; i < NV * 8; ++i) n[i] = (n[i] - st.x) * st.y;
    }
    if constexpr (!KEEP) {
      if (p.post) weight(p.w1, t);
    }
    if (p.gate) {
      float g[NV * 8];
      if (p.o && (GATE || p.dgate)) {  // z from the normalised output
        float z[NV * 8];
#pragma unroll
        for (int i = 0; i < NV * 8; ++i) z[i] = p.post ? n[i] * (KEEP ? w1[KEEP ? i : 0] : t[i]) : n[i];
        if (LN && p.post && p.c1) {
          own.load(p.c1, p.pdt, 0.0f, g);
#pragma unroll
          for (int i = 0; i < NV * 8; ++i) z[i] += g[i];
        }
        if constexpr (GATE) {
#pragma unroll
          for (int i = 0; i < NV * 8; ++i) ag[i] = fmaf(d[i], z[i], ag[i]);
        } else {
#pragma unroll
          for (int i = 0; i < NV * 8; ++i) z[i] *= d[i];
          own.store(row_at(p.dgate, row, p.dgate_ld, p.bdt), p.bdt, z);
        }
      }
      if (need_gate_rows) own.load(row_at(p.gate, row, p.gate_ld, p.bdt), p.bdt, 0.0f, g);
      else own.load(p.gate, p.pdt, 0.0f, g);
#pragma unroll
      for (int i = 0; i < NV * 8; ++i) d[i] *= g[i];
    }
    if (p.post) {
      float s[2] = {0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < NV * 8; ++i) {
        aw1[i] = fmaf(d[i], n[i], aw1[i]);
        if constexpr (LN) ac1[i] += d[i];
        d[i] *= KEEP ? w1[KEEP ? i : 0] : t[i];
        s[0] = fmaf(d[i], n[i], s[0]);
        if constexpr (LN) s[1] += d[i];
      }
      if constexpr (LN) {
        cta_sums(s, red, turn);
      } else {
        float s1[1] = {s[0]};
        cta_sums(s1, red, turn);
        s[0] = s1[0];
      }
      const float c = s[0] * p.inv_d, m = LN ? s[1] * p.inv_d : 0.0f;
#pragma unroll
      for (int i = 0; i < NV * 8; ++i) d[i] = st.y * (LN ? fmaf(-n[i], c, d[i]) - m : fmaf(-n[i], c, d[i]));
    }
    if (p.d_o) own.store(row_at(p.d_o, row, p.do_ld, p.bdt), p.bdt, d);
    stage = stage + 1 >= p.stages ? 0 : stage + 1;
  }
  if (!p.sums) return;
  auto leave = [&](int which, float (&a)[NV * 8]) {
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

// Vectors of 8 per thread by the row's width, and the threads of a CTA
int norm_nv(int64_t D) { return D <= 2048 ? 1 : D <= 8192 ? 2 : 4; }
int norm_threads(int64_t D) {
  const int64_t per = 8 * norm_nv(D);
  return (int)(((D + per - 1) / per + 31) / 32 * 32);
}
// CTAs that stay resident (by threads and registers; rows are handed out evenly)
int64_t norm_grid(const moe_norm_plan* pl, int64_t T) {
  const int nt = norm_threads(pl->cfg.D);
  const int64_t per_sm = nt >= 384 ? 1 : nt >= 256 ? 2 : nt >= 160 ? 3 : nt >= 96 ? 5 : 8;
  const int64_t most = per_sm * pl->num_sms;
  return T < most ? T : most;
}
constexpr int NORM_SMEM = 200 * 1024;  // of an SM's shared memory for the rings

template <typename F>
cudaError_t norm_by_width(int64_t D, F&& f) {
  switch (norm_nv(D)) {
    case 1: return f(std::integral_constant<int, 1>{});
    case 2: return f(std::integral_constant<int, 2>{});
    default: return f(std::integral_constant<int, 4>{});
  }
}

template <typename P>
cudaError_t norm_launch(void (*kernel)(P), dim3 grid, unsigned threads, size_t smem, cudaStream_t st, const P& p) {
  if (smem > 48 * 1024) {
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
  p.nvec = (int)(c.D / 8);
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
  const int64_t grid = norm_grid(pl, T);
  size_t smem = 0;
  if (vec)
    norm_ring(pl, p, grid, (size_t)c.D * ((x ? norm_size(c.stream_dtype) : 0) + (o ? norm_size(c.branch_dtype) : 0) +
                                          (p.gate_rows ? norm_size(c.branch_dtype) : 0)), smem);
  const cudaError_t err = norm_by_width(c.D, [&](auto nv) {
    constexpr int NV = decltype(nv)::value;
    auto go = [&](auto ln, auto v) {
      return norm_launch(norm_fwd_kernel<NV, decltype(ln)::value, decltype(v)::value>, dim3((unsigned)grid),
                         (unsigned)norm_threads(c.D), smem, (cudaStream_t)stream, p);
    };
    if (c.kind == MOE_NORM_LAYER) return vec ? go(std::true_type{}, std::true_type{}) : go(std::true_type{}, std::false_type{});
    return vec ? go(std::false_type{}, std::true_type{}) : go(std::false_type{}, std::false_type{});
  });
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
  const cudaError_t err = norm_by_width(c.D, [&](auto nv) {
    constexpr int NV = decltype(nv)::value;
    auto go = [&](auto ln, auto v, auto g) {
      return norm_launch(norm_bwd_kernel<NV, decltype(ln)::value, decltype(v)::value, decltype(g)::value>,
                         dim3((unsigned)grid), (unsigned)norm_threads(c.D), smem, stream, p);
    };
    auto by_gate = [&](auto ln, auto v) { return gate_sum ? go(ln, v, std::true_type{}) : go(ln, v, std::false_type{}); };
    if (c.kind == MOE_NORM_LAYER)
      return vec ? by_gate(std::true_type{}, std::true_type{}) : by_gate(std::true_type{}, std::false_type{});
    return vec ? by_gate(std::false_type{}, std::true_type{}) : by_gate(std::false_type{}, std::false_type{});
  });
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
