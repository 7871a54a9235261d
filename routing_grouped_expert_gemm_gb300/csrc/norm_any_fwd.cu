// Forward of the norms around a block for rows off vectors (norm_any.cuh).
// 1003 x 2053 layer norms in fp16 with a gate per row: 17.3 us (22 with
// the row in shared memory between the passes).  An element's own instructions bound it
// (2000 x 2056 layer norms take 25.8 us, in vectors 15), hence the elements of a thread in
// arrays that are read without a branch between them.
#include "norm_any.cuh"

namespace moe {

template <int NE, bool LN>
__device__ __forceinline__ void any_stats(const NormParams& p, const float (&v)[NE], Group& grp, float& m, float& r) {
  float s[1] = {0.0f};
  m = 0.0f;
  if constexpr (LN) {
#pragma unroll
    for (int j = 0; j < NE; ++j) s[0] += v[j];
    group_sums<1, ANY_MAX_WARPS>(s, grp);
    m = p.layer ? s[0] * p.inv_d : 0.0f;
    s[0] = 0.0f;
  }
#pragma unroll
  for (int j = 0; j < NE; ++j)
    if (!LN || threadIdx.x + j * blockDim.x < p.D) s[0] = fmaf(v[j] - m, v[j] - m, s[0]);
  group_sums<1, ANY_MAX_WARPS>(s, grp);
  r = rsqrtf(fmaf(s[0], p.inv_d, p.eps));
}

template <int MODE, int NE, bool LN, int S, int B>
__global__ void __launch_bounds__(1024) norm_fwd_any_kernel(const NormParams p) {
  extern __shared__ __align__(16) char smem[];
  __shared__ float red[2 * 2 * ANY_MAX_WARPS];
  const int tid = threadIdx.x, nt = blockDim.x;
  Group grp{red, 0, nt >> 5, tid >> 5, 0};
  uint32_t end = 0;
  const AnyRows ro(p.o, p.o_ld, p.D, B, end), rx(p.x, p.x_ld, p.D, S, end), rg(p.gate_rows ? p.gate : nullptr, p.gate_ld, p.D, B, end);
  auto fetch = [&](char* stage, int64_t t) { ro.fetch(stage, t), rx.fetch(stage, t), rg.fetch(stage, t); };
  grid_dependency_wait();
  if (MODE != ANY_NONE) any_first(p, smem, fetch);
  char* room = smem + p.stages * p.stage_bytes;
  const AnyParam<MODE> w1(p, p.w1, p.w_off, p.post, room), w2(p, p.w2, p.w_off, p.pre, room), c1(p, p.c1, 0.0f, false, room),
      c2(p, p.c2, 0.0f, false, room), gate(p, p.gate_rows ? nullptr : p.gate, 0.0f, false, room);
  any_rows<MODE>(p, smem, fetch, [&](const char* stage, int64_t t) {
    float v[NE], a[NE], m[2] = {0.0f, 0.0f}, r[2] = {0.0f, 0.0f};
    // (v - m) r w + c
    auto apply = [&](float m, float r, const AnyParam<MODE>& w, const AnyParam<MODE>& c, bool biased) {
      w.mine(p.D, a);
#pragma unroll
      for (int j = 0; j < NE; ++j) v[j] = (v[j] - m) * r * a[j];
      if (LN && biased) {
        c.mine(p.D, a);
#pragma unroll
        for (int j = 0; j < NE; ++j) v[j] += a[j];
      }
    };
    if (p.o) {
      load_mine<B>(ro.row<MODE>(stage, t), p.D, v);
    } else {
#pragma unroll
      for (int j = 0; j < NE; ++j) v[j] = 0.0f;
    }
    if (p.post) {
      any_stats<NE, LN>(p, v, grp, m[0], r[0]);
      apply(m[0], r[0], w1, c1, p.c1);
    }
    if (p.gate) {
      if (p.gate_rows) load_mine<B>(rg.row<MODE>(stage, t), p.D, a);
      else gate.mine(p.D, a);
#pragma unroll
      for (int j = 0; j < NE; ++j) v[j] *= a[j];
    }
#pragma unroll
    for (int j = 0; j < NE; ++j) v[j] *= p.o_scale;
    if (p.x) {
      load_mine<S>(rx.row<MODE>(stage, t), p.D, a);
#pragma unroll
      for (int j = 0; j < NE; ++j) v[j] = fmaf(p.x_scale, a[j], v[j]);
    }
    char* const y = p.y ? static_cast<char*>(p.y) + t * p.y_ld * esize(S) : nullptr;
#pragma unroll
    for (int j = 0; j < NE; ++j) v[j] = store1<S>(tid + j * nt < p.D ? y : nullptr, tid + j * nt, v[j]);
    if (p.pre) {
      any_stats<NE, LN>(p, v, grp, m[1], r[1]);
      apply(m[1], r[1], w2, c2, p.c2);
      char* const h = static_cast<char*>(p.h) + t * p.h_ld * esize(B);
#pragma unroll
      for (int j = 0; j < NE; ++j) store1<B>(tid + j * nt < p.D ? h : nullptr, tid + j * nt, v[j]);
    }
    if (p.stats && tid == 0) {
      float* st = p.stats + 4 * t;
      st[0] = m[0], st[1] = r[0], st[2] = m[1], st[3] = r[1];
    }
  });
}

cudaError_t launch_norm_fwd_any(const NormParams& p, unsigned grid, unsigned threads, size_t smem, cudaStream_t st) {
  return any_by_type(p, [&](auto s, auto b) {
    constexpr int S = decltype(s)::value, B = decltype(b)::value;
    auto kernel = !p.stages   ? norm_fwd_any_kernel<ANY_NONE, any_wide(ANY_NONE), true, S, B>
                  : !p.smem_w ? norm_fwd_any_kernel<ANY_ROWS, any_wide(ANY_ROWS), true, S, B>
                  : p.layer   ? norm_fwd_any_kernel<ANY_ALL, ANY_FWD, true, S, B>
                              : norm_fwd_any_kernel<ANY_ALL, ANY_FWD, false, S, B>;
    return norm_launch(kernel, dim3(grid), threads, smem, st, p);
  });
}

}  // namespace moe
