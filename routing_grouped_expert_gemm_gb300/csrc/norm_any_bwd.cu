// Backward of the norms around a block for rows off vectors (norm_any.cuh).
// 777 x 1001 layer norms in fp32: 20.2 us (28.9 with the row's elements and
// sums in shared memory), 20850 x 1455 in fp16 205 us (458).
#include "norm_any.cuh"

namespace moe {

template <int MODE, int NE, bool LN, bool GATE, int S, int B>
__global__ void __launch_bounds__(1024) norm_bwd_any_kernel(const NormParams p) {
  extern __shared__ __align__(16) char smem[];
  __shared__ float red[2 * 2 * ANY_MAX_WARPS];
  const int tid = threadIdx.x, nt = blockDim.x;
  Group grp{red, 0, nt >> 5, tid >> 5, 0};
  uint32_t end = 0;
  const AnyRows ry(p.pre ? p.y : nullptr, p.y_ld, p.D, S, end), rh(p.pre ? p.dh : nullptr, p.dh_ld, p.D, B, end),
      rd(p.dy, p.dy_ld, p.D, S, end), ro(p.o, p.o_ld, p.D, B, end),
      rg(GATE && p.gate_rows ? p.gate : nullptr, p.gate_ld, p.D, B, end),
      rs(p.stats, 4, 4, MOE_DTYPE_FP32, end);  // (the row's statistics with it)
  auto fetch = [&](char* stage, int64_t t) {
    ry.fetch(stage, t), rh.fetch(stage, t), rd.fetch(stage, t), ro.fetch(stage, t), rs.fetch(stage, t);
    if (GATE) rg.fetch(stage, t);
  };
  grid_dependency_wait();
  if (MODE != ANY_NONE) any_first(p, smem, fetch);
  char* room = smem + p.stages * p.stage_bytes;
  const AnyParam<MODE> w1(p, p.w1, p.w_off, p.post, room), w2(p, p.w2, p.w_off, p.pre, room),
      c1(p, GATE && p.gate ? p.c1 : nullptr, 0.0f, false, room),
      gate(p, GATE && !p.gate_rows ? p.gate : nullptr, 0.0f, false, room);
  // the sums: dw and dc of both norms, dg
  float aw1[NE], aw2[NE], ac1[LN ? NE : 1], ac2[LN ? NE : 1], ag[GATE ? NE : 1];
#pragma unroll
  for (int j = 0; j < NE; ++j) {
    aw1[j] = aw2[j] = 0.0f;
    if constexpr (LN) ac1[j] = ac2[j] = 0.0f;
    if constexpr (GATE) ag[j] = 0.0f;
  }
  any_rows<MODE>(p, smem, fetch, [&](const char* stage, int64_t t) {
    float st[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (p.stats) {
      const float* from = reinterpret_cast<const float*>(rs.row<MODE>(stage, t));
#pragma unroll
      for (int i = 0; i < 4; ++i) st[i] = from[i];
    }
    // outside the row gradients and weights are 0, and so is all that enters the sums
    float v[NE], d[NE], n[NE], w[NE], s[LN ? 2 : 1] = {0.0f};
    if (p.dy) {
      load_mine<S>(rd.row<MODE>(stage, t), p.D, v);
    } else {
#pragma unroll
      for (int j = 0; j < NE; ++j) v[j] = 0.0f;
    }
    if (p.pre) {
      load_mine<S>(ry.row<MODE>(stage, t), p.D, n);
      load_mine<B>(rh.row<MODE>(stage, t), p.D, d);
      w2.mine(p.D, w);
#pragma unroll
      for (int j = 0; j < NE; ++j) {
        n[j] = (n[j] - st[2]) * st[3];
        aw2[j] = fmaf(d[j], n[j], aw2[j]);
        if constexpr (LN) ac2[j] += d[j];
        d[j] *= w[j];
        s[0] = fmaf(d[j], n[j], s[0]);
        if constexpr (LN) s[1] += d[j];
      }
      group_sums<LN ? 2 : 1, ANY_MAX_WARPS>(s, grp);
      const float q = s[0] * p.inv_d, m = LN && p.layer ? s[LN ? 1 : 0] * p.inv_d : 0.0f;
#pragma unroll
      for (int j = 0; j < NE; ++j) v[j] = fmaf(st[3], d[j] - n[j] * q - m, v[j]);
    }
    if (p.dx) {
      char* const dx = static_cast<char*>(p.dx) + t * p.dx_ld * esize(S);
#pragma unroll
      for (int j = 0; j < NE; ++j) store1<S>(tid + j * nt < p.D ? dx : nullptr, tid + j * nt, p.x_scale * v[j]);
    }
    if (p.o) load_mine<B>(ro.row<MODE>(stage, t), p.D, n);
    if (p.post) w1.mine(p.D, w);
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      v[j] *= p.o_scale;
      if (!p.o) n[j] = 0.0f;
      if (p.post) n[j] = (n[j] - st[0]) * st[1];
      else w[j] = 1.0f;
    }
    if constexpr (GATE) {
      if (p.post && p.c1) c1.mine(p.D, d);
      char* const dg = p.dgate ? static_cast<char*>(p.dgate) + t * p.dgate_ld * esize(B) : nullptr;
#pragma unroll
      for (int j = 0; j < NE; ++j) {
        const float a = v[j] * (p.post && p.c1 ? fmaf(n[j], w[j], d[j]) : n[j] * w[j]);
        ag[j] += a;
        store1<B>(tid + j * nt < p.D ? dg : nullptr, tid + j * nt, a);
      }
      if (p.gate) {
        if (p.gate_rows) load_mine<B>(rg.row<MODE>(stage, t), p.D, d);
        else gate.mine(p.D, d);
#pragma unroll
        for (int j = 0; j < NE; ++j) v[j] *= d[j];
      }
    }
    if (p.post) {
#pragma unroll
      for (float& a : s) a = 0.0f;
#pragma unroll
      for (int j = 0; j < NE; ++j) {
        aw1[j] = fmaf(v[j], n[j], aw1[j]);
        if constexpr (LN) ac1[j] += v[j];
        v[j] *= w[j];
        s[0] = fmaf(v[j], n[j], s[0]);
        if constexpr (LN) s[1] += v[j];
      }
      group_sums<LN ? 2 : 1, ANY_MAX_WARPS>(s, grp);
      const float q = s[0] * p.inv_d, m = LN && p.layer ? s[LN ? 1 : 0] * p.inv_d : 0.0f;
#pragma unroll
      for (int j = 0; j < NE; ++j) v[j] = st[1] * (v[j] - n[j] * q - m);
    }
    if (p.d_o) {
      char* const d_o = static_cast<char*>(p.d_o) + t * p.do_ld * esize(B);
#pragma unroll
      for (int j = 0; j < NE; ++j) store1<B>(tid + j * nt < p.D ? d_o : nullptr, tid + j * nt, v[j]);
    }
  });
  if (!p.sums) return;
  float* const out = p.sums + (size_t)blockIdx.x * NORM_SUMS * p.D;
#pragma unroll
  for (int j = 0; j < NE; ++j)
    if (const int e = tid + j * nt; e < p.D) {
      out[e] = aw1[j];
      out[2 * p.D + e] = aw2[j];
      if constexpr (LN) out[p.D + e] = ac1[j], out[3 * p.D + e] = ac2[j];
      if constexpr (GATE) out[4 * p.D + e] = ag[j];
    }
}

cudaError_t launch_norm_bwd_any(const NormParams& p, unsigned grid, unsigned threads, size_t smem, cudaStream_t st) {
  return any_by_type(p, [&](auto s, auto b) {
    constexpr int S = decltype(s)::value, B = decltype(b)::value;
    auto pick = [&](auto per) {
      constexpr int NE = decltype(per)::value;
      return p.gate ? (p.layer ? norm_bwd_any_kernel<ANY_ALL, NE, true, true, S, B> : norm_bwd_any_kernel<ANY_ALL, NE, false, true, S, B>)
                    : (p.layer ? norm_bwd_any_kernel<ANY_ALL, NE, true, false, S, B> : norm_bwd_any_kernel<ANY_ALL, NE, false, false, S, B>);
    };
    auto kernel = !p.stages               ? norm_bwd_any_kernel<ANY_NONE, any_wide(ANY_NONE), true, true, S, B>
                  : !p.smem_w             ? norm_bwd_any_kernel<ANY_ROWS, any_wide(ANY_ROWS), true, true, S, B>
                  : any_bwd_per(p.D) == 4 ? pick(std::integral_constant<int, 4>{})
                                          : pick(std::integral_constant<int, 8>{});
    return norm_launch(kernel, dim3(grid), threads, smem, st, p);
  });
}

}  // namespace moe
