// Forward of the norms around a block, rows in whole vectors (norm.cuh has the
// formulas).  16384 x 7168 in bf16: 147 to 149 us, 94% of the copy rate.
//
// A CTA works on several rows at a time, each in a group of threads of its own, so
// that one row's barriers are another's work; a thread takes two vectors (four past
// 8192): with one, what a thread does besides its elements (sums, barriers, addresses)
// is most of its instructions (194 us, two then took 160), with four too few warps hide
// a row's latency (221 us).  A group's rows are grid rows apart: with neighbouring rows 161
// us, where this took 149.  The weights are in shared memory as fp32 where the CTA has rows
// enough for that to pay.
#include "norm.cuh"

namespace moe {

template <int NV, bool LN, int S, int B, int W /* whole */>
__global__ void __launch_bounds__(norm_fwd_threads(NV)) norm_fwd_kernel(const NormParams p) {
  const bool has_x = W || p.x, has_o = W || p.o, post = W || p.post, pre = W || p.pre, has_y = W || p.y, smem_w = W || p.smem_w,
             gated = !W && p.gate, gate_rows = !W && p.gate_rows;
  const int stages = W ? NORM_FWD_STAGES : p.stages, stage_bytes = p.stage_bytes;
  extern __shared__ __align__(16) char smem[];
  __shared__ float red[16 * 2 * 2 * NORM_MAX_WARPS];  // of groups of two warps and more
  const int g = threadIdx.x / p.group, groups = blockDim.x / p.group, tid = threadIdx.x - g * p.group;
  const int row = W == 2 ? p.D : p.places;  // elements of a row in the ring
  const Mine<NV, W == 2> mine(tid, p.group, p.nvec, row);
  Group grp{red + (g & 15) * (2 * 2 * NORM_MAX_WARPS), g, p.group >> 5, tid >> 5, 0};
  char* const ring = smem + g * stages * stage_bytes;
  const uint32_t at_o = has_x ? row * esize(S) : 0, at_g = at_o + (has_o ? row * esize(B) : 0);
  // this group's rows, and the pointers that go along with them (`a`: to what is fetched ahead)
  const int64_t row0 = (int64_t)g * gridDim.x + blockIdx.x, step = (int64_t)groups * gridDim.x;
  const int rows = row0 < p.T ? (int)((p.T - row0 + step - 1) / step) : 0;
  const char* xa = static_cast<const char*>(p.x) + row0 * p.x_ld * esize(S);
  const char* oa = static_cast<const char*>(p.o) + row0 * p.o_ld * esize(B);
  const char* ga = static_cast<const char*>(p.gate) + (gate_rows ? row0 * p.gate_ld * esize(B) : 0);
  char* y = has_y ? static_cast<char*>(p.y) + row0 * p.y_ld * esize(S) : nullptr;
  char* h = static_cast<char*>(p.h) + row0 * p.h_ld * esize(B);
  const int64_t xs = step * p.x_ld * esize(S), os = step * p.o_ld * esize(B), gs = step * p.gate_ld * esize(B),
                ys = has_y ? step * p.y_ld * esize(S) : 0, hs = step * p.h_ld * esize(B);
  grid_dependency_wait();
  auto fetch_o = [&](bool on, char* stage) {
    if (on && has_o) {
      mine.template fetch<B>(stage + at_o, oa);
      oa += os;
    }
    cp_async_commit();
  };
  auto fetch_x = [&](bool on, char* stage) {
    if (on) {
      if (has_x) {
        mine.template fetch<S>(stage, xa);
        xa += xs;
      }
      if (gate_rows) {
        mine.template fetch<B>(stage + at_g, ga);
        ga += gs;
      }
    }
    cp_async_commit();
  };
  if constexpr (W != 2)
    for (int s = 0; s < stages; ++s) mine.clear(ring + s * stage_bytes, stage_bytes);
  for (int s = 0; s < stages; ++s) {
    fetch_o(s < rows, ring + s * stage_bytes);
    fetch_x(s < rows, ring + s * stage_bytes);
  }
  // the norms' weights as fp32, once per CTA
  char *sw1 = nullptr, *sw2 = nullptr;
  if (smem_w) {
    sw1 = sw2 = smem + groups * stages * stage_bytes;
    if (post) sw2 += row * 4;
    const int vecs = W == 2 ? p.nvec : row / 8;
#pragma unroll 1
    for (int i = threadIdx.x; i < 2 * vecs; i += blockDim.x) {
      const bool second = i >= vecs;
      const int v = second ? i - vecs : i;
      if (!(second ? pre : post)) continue;
      const Mine<1, W == 2> one(v, 0, p.nvec, row);
      F2 w[4];
      one.weight(0, second ? p.w2 : p.w1, p.pdt, p.w_off, w);
      const Raw<MOE_DTYPE_FP32> r = pack<MOE_DTYPE_FP32>(w);
      char* to = (second ? sw2 : sw1) + one.off[0];
      *reinterpret_cast<uint4*>(to) = r.q[0];
      *reinterpret_cast<uint4*>(to + one.plane) = r.q[1];
    }
    __syncthreads();
  }
  // vector j of (v - m) r w + c in place
  auto apply = [&](int j, F2 (&v)[4], float m, float r, const char* sw, const void* w, const void* c) {
    F2 t[4];
    if (smem_w) mine.template take<MOE_DTYPE_FP32>(j, sw, t);
    else mine.weight(j, w, p.pdt, p.w_off, t);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (LN ? v[i] + f2(-m) : v[i]) * f2(r) * t[i];
    if (LN && c) {
      mine.global(j, c, p.pdt, 0.0f, t);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = v[i] + t[i];
    }
  };
  int stage = 0;
  float* stat = p.stats ? p.stats + 4 * row0 : nullptr;
#pragma unroll 1
  for (int i = 0; i < rows; ++i) {
    char* const at = ring + stage * stage_bytes;
    const bool more = i + stages < rows;
    float4 st = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    F2 v[NV][4];
    cp_async_wait(2 * stages - 1);  // o
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (has_o) {
        mine.template take<B>(j, at + at_o, v[j]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[j][e] = f2(0.0f);
      }
    }
    if (post) row_stats<NV, LN, W == 2>(mine, v, p.inv_d, p.eps, grp, st.x, st.y);
    cp_async_wait(2 * stages - 2);  // x and the gate
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      F2 t[4];
      if (post) apply(j, v[j], st.x, st.y, sw1, p.w1, p.c1);
      if (gated) {
        if (gate_rows) mine.template take<B>(j, at + at_g, t);
        else mine.global(j, p.gate, p.pdt, 0.0f, t);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[j][e] = v[j][e] * t[e];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) v[j][e] = v[j][e] * f2(p.o_scale);
      if (has_x) {
        mine.template take<S>(j, at, t);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[j][e] = fma2(f2(p.x_scale), t[e], v[j][e]);
      }
      mine.template put<S, (W > 0)>(j, y, v[j]);
    }
    if (pre) row_stats<NV, LN, W == 2>(mine, v, p.inv_d, p.eps, grp, st.z, st.w);
    if (pre) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        apply(j, v[j], st.z, st.w, sw2, p.w2, p.c2);
        mine.template put<B, true>(j, h, v[j]);
      }
    }
    fetch_o(more, at);  // (as soon as its place is free, between the row's writes, a row costs 6% more)
    fetch_x(more, at);
    if (stat) {
      if (tid == 0) stat[0] = st.x, stat[1] = st.y, stat[2] = st.z, stat[3] = st.w;
      stat += 4 * step;
    }
    y += ys, h += hs;
    stage = stage + 1 >= stages ? 0 : stage + 1;
  }
}

cudaError_t launch_norm_fwd(const NormParams& p, unsigned grid, unsigned threads, size_t smem, cudaStream_t st) {
  auto by_type = [&](auto s, auto b) {
    constexpr int S = decltype(s)::value, B = decltype(b)::value;
    auto kernel = p.whole == 2  ? (p.layer ? norm_fwd_kernel<2, true, S, B, 2> : norm_fwd_kernel<2, false, S, B, 2>)
                  : p.whole     ? (p.layer ? norm_fwd_kernel<2, true, S, B, 1> : norm_fwd_kernel<2, false, S, B, 1>)
                  : p.D <= 8192 ? (p.layer ? norm_fwd_kernel<2, true, S, B, 0> : norm_fwd_kernel<2, false, S, B, 0>)
                                : (p.layer ? norm_fwd_kernel<4, true, S, B, 0> : norm_fwd_kernel<4, false, S, B, 0>);
    return norm_launch(kernel, dim3(grid), threads, smem, st, p);
  };
  constexpr std::integral_constant<int, MOE_DTYPE_FP32> f32{};
  constexpr std::integral_constant<int, MOE_DTYPE_BF16> b16{};
  constexpr std::integral_constant<int, MOE_DTYPE_FP16> f16{};
  if (p.sdt == MOE_DTYPE_BF16) return by_type(b16, b16);
  if (p.sdt == MOE_DTYPE_FP16) return by_type(f16, f16);
  return p.bdt == MOE_DTYPE_FP32 ? by_type(f32, f32) : p.bdt == MOE_DTYPE_BF16 ? by_type(f32, b16) : by_type(f32, f16);
}

}  // namespace moe
