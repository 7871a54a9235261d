// Norms around a block and their gradients for rows that are not whole vectors on
// 16-byte boundaries, or do not fit the other kernels' shared memory (norm.cuh has the
// formulas).  1003 x 2053 in fp16 with a gate per row: ANYTIME.
//
// A CTA a row; thread i takes elements i, i + NT, ... one by one, so that whatever the
// alignment a warp's accesses lie together.  A row is read once, all its tensors at
// once, and waits in shared memory as fp32 between the passes over it.
#include "norm.cuh"

namespace moe {

template <int DT>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if constexpr (DT == MOE_DTYPE_FP32) return static_cast<const float*>(p)[i];
  if constexpr (DT == MOE_DTYPE_BF16) return __bfloat162float(static_cast<const bf16*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}
// rounds to the type, stores unless p is null, returns what was rounded
template <int DT>
__device__ __forceinline__ float store1(void* p, int64_t i, float v) {
  if constexpr (DT == MOE_DTYPE_FP32) {
    if (p) static_cast<float*>(p)[i] = v;
    return v;
  } else if constexpr (DT == MOE_DTYPE_BF16) {
    const bf16 w = __float2bfloat16_rn(v);
    if (p) static_cast<bf16*>(p)[i] = w;
    return __bfloat162float(w);
  } else {
    const __half w = __float2half_rn(v);
    if (p) static_cast<__half*>(p)[i] = w;
    return __half2float(w);
  }
}

// mean and 1 / sqrt(variance + eps) of the row in shared memory
__device__ __forceinline__ void any_stats(const NormParams& p, const float* v, float first /* this thread's sum */, Group& grp, float& m, float& r) {
  float s[1] = {first};
  m = 0.0f;
  if (p.layer) {
    group_sums(s, grp);
    m = s[0] * p.inv_d;
  }
  s[0] = 0.0f;
#pragma unroll 4
  for (int e = threadIdx.x; e < p.D; e += blockDim.x) s[0] = fmaf(v[e] - m, v[e] - m, s[0]);
  group_sums(s, grp);
  r = rsqrtf(fmaf(s[0], p.inv_d, p.eps));
}

template <int S, int B, int P>
__global__ void __launch_bounds__(512) norm_fwd_any_kernel(const NormParams p) {
  extern __shared__ __align__(16) float any_smem[];  // o (then y), x, gate of the row
  __shared__ float red[2 * 2 * NORM_MAX_WARPS];
  float *const v = any_smem, *const xr = v + p.D, *const gr = xr + p.D;
  Group grp{red, 0, (int)blockDim.x >> 5, (int)threadIdx.x >> 5, 0};
  grid_dependency_wait();
#pragma unroll 1
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    float m[2] = {0.0f, 0.0f}, r[2] = {0.0f, 0.0f}, s = 0.0f;
#pragma unroll 4
    for (int e = threadIdx.x; e < p.D; e += blockDim.x) {
      const float o = p.o ? load1<B>(p.o, t * p.o_ld + e) : 0.0f;
      if (p.x) xr[e] = load1<S>(p.x, t * p.x_ld + e);
      if (p.gate) gr[e] = p.gate_rows ? load1<B>(p.gate, t * p.gate_ld + e) : load1<P>(p.gate, e);
      v[e] = o;
      s += o;
    }
    if (p.post) any_stats(p, v, s, grp, m[0], r[0]);
    s = 0.0f;
#pragma unroll 4
    for (int e = threadIdx.x; e < p.D; e += blockDim.x) {
      float z = v[e];
      if (p.post) {
        z = (z - m[0]) * r[0] * (p.w1 ? load1<P>(p.w1, e) + p.w_off : 1.0f);
        if (p.c1) z += load1<P>(p.c1, e);
      }
      if (p.gate) z *= gr[e];
      z *= p.o_scale;
      if (p.x) z = fmaf(p.x_scale, xr[e], z);
      s += v[e] = store1<S>(p.y, t * p.y_ld + e, z);
    }
    if (p.pre) {
      any_stats(p, v, s, grp, m[1], r[1]);
#pragma unroll 4
      for (int e = threadIdx.x; e < p.D; e += blockDim.x) {
        float z = (v[e] - m[1]) * r[1] * (p.w2 ? load1<P>(p.w2, e) + p.w_off : 1.0f);
        if (p.c2) z += load1<P>(p.c2, e);
        store1<B>(p.h, t * p.h_ld + e, z);
      }
    }
    if (p.stats && threadIdx.x == 0) {
      float* st = p.stats + 4 * t;
      st[0] = m[0], st[1] = r[0], st[2] = m[1], st[3] = r[1];
    }
  }
}

// Short rows (p.stages) are fetched whole before anything else; of long ones only the
// gradient and the normalised input wait in shared memory.  The sums over the rows are
// kept by the element's own thread: in shared memory where they fit beside the row
// (p.smem_w), else in the CTA's part of the workspace.
template <int S, int B, int P>
__global__ void __launch_bounds__(512) norm_bwd_any_kernel(const NormParams p) {
  extern __shared__ __align__(16) float any_smem[];  // gradient, normalised input, dy, o, gate of the row; sums
  __shared__ float red[2 * 2 * NORM_MAX_WARPS];
  float *const row_d = any_smem, *const row_n = row_d + p.D, *const row_y = row_n + p.D, *const row_o = row_y + p.D,
        *const row_g = row_o + p.D;
  Group grp{red, 0, (int)blockDim.x >> 5, (int)threadIdx.x >> 5, 0};
  grid_dependency_wait();
  float* const out = p.sums ? p.sums + (size_t)blockIdx.x * NORM_SUMS * p.D : nullptr;
  float* const sums = out && p.smem_w ? any_smem + 5 * p.D : out;
  auto add = [&](int which, int e, float v, bool first) {
    float* at = sums + which * p.D + e;
    *at = first ? v : *at + v;
  };
#pragma unroll 1
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    const bool first = t == blockIdx.x;
    float st[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (p.stats)
      for (int i = 0; i < 4; ++i) st[i] = p.stats[4 * t + i];
    // the whole row on its way at once
    if (p.stages) {
#pragma unroll 4
      for (int e = threadIdx.x; e < p.D; e += blockDim.x) {
        if (p.pre) row_d[e] = load1<B>(p.dh, t * p.dh_ld + e), row_n[e] = load1<S>(p.y, t * p.y_ld + e);
        if (p.dy) row_y[e] = load1<S>(p.dy, t * p.dy_ld + e);
        if (p.o) row_o[e] = load1<B>(p.o, t * p.o_ld + e);
        if (p.gate) row_g[e] = p.gate_rows ? load1<B>(p.gate, t * p.gate_ld + e) : load1<P>(p.gate, e);
      }
    }
    float s[2] = {0.0f, 0.0f};
    if (p.pre) {
#pragma unroll 4
      for (int e = threadIdx.x; e < p.D; e += blockDim.x) {
        const float d = p.stages ? row_d[e] : load1<B>(p.dh, t * p.dh_ld + e);
        const float n = ((p.stages ? row_n[e] : load1<S>(p.y, t * p.y_ld + e)) - st[2]) * st[3];
        const float u = d * (p.w2 ? load1<P>(p.w2, e) + p.w_off : 1.0f);
        if (sums) {
          add(2, e, d * n, first);
          if (p.layer) add(3, e, d, first);
        }
        s[0] = fmaf(u, n, s[0]), s[1] += u;
        row_d[e] = u, row_n[e] = n;
      }
      group_sums(s, grp);
    }
    const float c2 = s[0] * p.inv_d, m2 = p.layer ? s[1] * p.inv_d : 0.0f;
    s[0] = s[1] = 0.0f;
#pragma unroll 4
    for (int e = threadIdx.x; e < p.D; e += blockDim.x) {
      float d = !p.dy ? 0.0f : p.stages ? row_y[e] : load1<S>(p.dy, t * p.dy_ld + e);
      if (p.pre) d = fmaf(st[3], row_d[e] - row_n[e] * c2 - m2, d);
      if (p.dx) store1<S>(p.dx, t * p.dx_ld + e, p.x_scale * d);
      d *= p.o_scale;
      float n = !p.o ? 0.0f : p.stages ? row_o[e] : load1<B>(p.o, t * p.o_ld + e);
      if (p.post) n = (n - st[0]) * st[1];
      const float w = p.post && p.w1 ? load1<P>(p.w1, e) + p.w_off : 1.0f;
      if (p.gate) {
        const float z = n * w + (p.post && p.c1 ? load1<P>(p.c1, e) : 0.0f);
        if (p.gate_sum && sums) add(4, e, d * z, first);
        if (p.dgate) store1<B>(p.dgate, t * p.dgate_ld + e, d * z);
        d *= p.stages ? row_g[e] : p.gate_rows ? load1<B>(p.gate, t * p.gate_ld + e) : load1<P>(p.gate, e);
      }
      if (p.post) {
        if (sums) {
          add(0, e, d * n, first);
          if (p.layer) add(1, e, d, first);
        }
        d *= w;
        s[0] = fmaf(d, n, s[0]), s[1] += d;
        row_d[e] = d, row_n[e] = n;
      } else if (p.d_o) {
        store1<B>(p.d_o, t * p.do_ld + e, d);
      }
    }
    if (p.post) {
      group_sums(s, grp);
      const float c1 = s[0] * p.inv_d, m1 = p.layer ? s[1] * p.inv_d : 0.0f;
      if (p.d_o)
#pragma unroll 4
        for (int e = threadIdx.x; e < p.D; e += blockDim.x) store1<B>(p.d_o, t * p.do_ld + e, st[1] * (row_d[e] - row_n[e] * c1 - m1));
    }
  }
  if (out && p.smem_w)
#pragma unroll 1
    for (int k = 0; k < NORM_SUMS; ++k) {
      if (k == 4 ? !p.gate_sum : (k & 1 && !p.layer) || !(k < 2 ? p.post : p.pre)) continue;
#pragma unroll 4
      for (int e = threadIdx.x; e < p.D; e += blockDim.x) out[(size_t)k * p.D + e] = sums[k * p.D + e];
    }
}

namespace {

// the kernel of a call's types
template <typename F>
cudaError_t any_by_type(const NormParams& p, F&& f) {
  constexpr std::integral_constant<int, MOE_DTYPE_FP32> f32{};
  constexpr std::integral_constant<int, MOE_DTYPE_BF16> b16{};
  constexpr std::integral_constant<int, MOE_DTYPE_FP16> f16{};
  auto by_param = [&](auto s, auto b) { return p.pdt == MOE_DTYPE_FP32 ? f(s, b, f32) : p.pdt == MOE_DTYPE_BF16 ? f(s, b, b16) : f(s, b, f16); };
  if (p.sdt == MOE_DTYPE_BF16) return by_param(b16, b16);
  if (p.sdt == MOE_DTYPE_FP16) return by_param(f16, f16);
  return p.bdt == MOE_DTYPE_FP32 ? by_param(f32, f32) : p.bdt == MOE_DTYPE_BF16 ? by_param(f32, b16) : by_param(f32, f16);
}

}  // namespace

cudaError_t launch_norm_fwd_any(const NormParams& p, unsigned grid, unsigned threads, cudaStream_t st) {
  return any_by_type(p, [&](auto s, auto b, auto q) {
    return norm_launch(norm_fwd_any_kernel<decltype(s)::value, decltype(b)::value, decltype(q)::value>, dim3(grid), threads,
                       (size_t)p.D * 12, st, p);
  });
}
cudaError_t launch_norm_bwd_any(const NormParams& p, unsigned grid, unsigned threads, cudaStream_t st) {
  return any_by_type(p, [&](auto s, auto b, auto q) {
    return norm_launch(norm_bwd_any_kernel<decltype(s)::value, decltype(b)::value, decltype(q)::value>, dim3(grid), threads,
                       (size_t)p.D * 4 * (p.smem_w ? 5 + NORM_SUMS : p.stages ? 5 : 2), st, p);
  });
}

}  // namespace moe
