// Backward of the norms around a block, rows in whole vectors (norm.cuh has the
// formulas).  16384 x 7168 in bf16: 231 us, 90% of the copy rate.
//
// A CTA keeps to its own rows, a thread to its own columns: the sums over the rows (dw
// and dc of both norms, dg) stay in its registers, and leave the CTA once, at the end.  The
// norms' weights are in registers too (up to 8192 elements a row, but for pairs of rows,
// which have them in shared memory; above they are read again in every row).  128 registers
// do not hold all of it in every form.  Bytes spilled a thread: rms none, with a channel's gate
// 16 to 64; pairs none (fp32 64 to 68), with a gate 116 to 192; layer norms 88 to 252, with a
// gate 400 to 440; rows of more than 8192 elements 408 to 1704.
#include "norm.cuh"

namespace moe {

// One norm's sums over the rows, for dw and (layer norms) dc: this thread's columns
template <int NV, bool LN>
struct NormBack {
  F2 aw[NV][4], ac[LN ? NV : 1][4];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        aw[j][i] = f2(0.0f);
        if constexpr (LN) ac[j][i] = f2(0.0f);
      }
  }
};

template <int NV, bool LN, bool GATE, int S, int B, int W /* whole */>
__global__ void __launch_bounds__(512) norm_bwd_kernel(const NormParams p) {
  const bool pre = W || p.pre, post = W || p.post, has_dy = W || p.dy, has_o = W || p.o, gated = GATE || (!W && p.gate),
             gate_rows = !W && p.gate_rows, has_dx = W || p.dx, has_do = W || p.d_o, has_dgate = !W && p.dgate;
  const int stages = W ? NORM_BWD_STAGES : p.stages, stage_bytes = p.stage_bytes;
  constexpr bool KEEP = NV <= 2;  // the weights in registers
  extern __shared__ __align__(16) char smem[];
  __shared__ float red[2 * 2 * NORM_MAX_WARPS];
  const int tid = threadIdx.x;
  const int row = W == 2 ? p.D : p.places;  // elements of a row in the ring
  const Mine<NV, W == 2> mine(tid, blockDim.x, p.nvec, row);
  Group grp{red, 0, (int)blockDim.x >> 5, tid >> 5, 0};
  // order in the ring: y, dh, dy, o; the gate's rows are read when they are needed
  char* const ring = smem;
  const uint32_t at_h = pre ? row * esize(S) : 0, at_d = at_h + (pre ? row * esize(B) : 0), at_o = at_d + (has_dy ? row * esize(S) : 0);
  const int64_t row0 = blockIdx.x, step = gridDim.x;
  const int rows = (int)((p.T - row0 + step - 1) / step);
  auto at_row = [&](const void* v, int64_t ld, int size) { return v ? static_cast<const char*>(v) + row0 * ld * size : nullptr; };
  const char *ya = at_row(p.y, p.y_ld, esize(S)), *ha = at_row(p.dh, p.dh_ld, esize(B)), *da = at_row(p.dy, p.dy_ld, esize(S)),
             *oa = at_row(p.o, p.o_ld, esize(B));
  const char* gate = static_cast<const char*>(p.gate) + (gate_rows ? row0 * p.gate_ld * esize(B) : 0);
  char *dx = const_cast<char*>(at_row(p.dx, p.dx_ld, esize(S))), *d_o = const_cast<char*>(at_row(p.d_o, p.do_ld, esize(B))),
       *dgate = const_cast<char*>(at_row(p.dgate, p.dgate_ld, esize(B)));
  const int64_t y_step = step * p.y_ld * esize(S), h_step = step * p.dh_ld * esize(B), d_step = step * p.dy_ld * esize(S),
                o_step = step * p.o_ld * esize(B), dx_step = step * p.dx_ld * esize(S), do_step = step * p.do_ld * esize(B),
                dgate_step = step * p.dgate_ld * esize(B), gate_step = step * p.gate_ld * esize(B);
  const float* stat = p.stats ? p.stats + 4 * row0 : nullptr;
  grid_dependency_wait();
  auto fetch = [&](bool on, char* stage) {
    if (on) {
      if (pre) {
        mine.template fetch<S>(stage, ya);
        mine.template fetch<B>(stage + at_h, ha);
        ya += y_step, ha += h_step;
      }
      if (has_dy) {
        mine.template fetch<S>(stage + at_d, da);
        da += d_step;
      }
      if (has_o) {
        mine.template fetch<B>(stage + at_o, oa);
        oa += o_step;
      }
    }
    cp_async_commit();
  };
  if constexpr (W != 2)
    for (int s = 0; s < stages; ++s) mine.clear(ring + s * stage_bytes, stage_bytes);
  for (int s = 0; s + 1 < stages; ++s) fetch(s < rows, ring + s * stage_bytes);
  F2 w1[KEEP ? NV : 1][4], w2[KEEP ? NV : 1][4];
  if constexpr (KEEP)
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (post) mine.weight(j, p.w1, p.pdt, p.w_off, w1[j]);
      if (pre) mine.weight(j, p.w2, p.pdt, p.w_off, w2[j]);
    }
  NormBack<NV, LN> b1, b2;
  b1.clear(), b2.clear();
  F2 ag[GATE ? NV : 1][4];
  if constexpr (GATE)
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) ag[j][i] = f2(0.0f);
  // the row's means of u n and of u
  auto means = [&](F2 (&q)[2], F2 e, float& c, float& m) {
    m = 0.0f;
    if constexpr (LN) {
      const float2 b = split(e);
      float s[2] = {both(q[0], q[1]), b.x + b.y};
      group_sums(s, grp);
      c = s[0] * p.inv_d, m = s[1] * p.inv_d;
    } else {
      float s[1] = {both(q[0], q[1])};
      group_sums(s, grp);
      c = s[0] * p.inv_d;
    }
  };
  int stage = 0;
#pragma unroll 1
  for (int i = 0; i < rows; ++i) {
    char* const at = ring + stage * stage_bytes;
    {
      int next = stage + stages - 1;
      next = next >= stages ? next - stages : next;
      fetch(i + stages - 1 < rows, ring + next * stage_bytes);
    }
    float4 st = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (W || stat) {
      st = make_float4(stat[0], stat[1], stat[2], stat[3]);
      stat += 4 * step;
    }
    cp_async_wait(stages - 1);
    F2 d[NV][4], n[NV][4];
    float c, m;
    if (pre) {
      F2 u[NV][4], q[2] = {f2(0.0f), f2(0.0f)}, e = f2(0.0f);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        F2 w[4];
        mine.template take<S>(j, at, n[j]);
        mine.template take<B>(j, at + at_h, u[j]);
        if constexpr (!KEEP) mine.weight(j, p.w2, p.pdt, p.w_off, w);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          n[j][k] = (LN ? n[j][k] + f2(-st.z) : n[j][k]) * f2(st.w);
          b2.aw[j][k] = fma2(u[j][k], n[j][k], b2.aw[j][k]);
          if constexpr (LN) b2.ac[j][k] = b2.ac[j][k] + u[j][k];
          u[j][k] = u[j][k] * (KEEP ? w2[KEEP ? j : 0][k] : w[k]);
          q[k & 1] = fma2(u[j][k], n[j][k], q[k & 1]);
          if constexpr (LN) e = e + u[j][k];
        }
      }
      means(q, e, c, m);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (has_dy) {
          mine.template take<S>(j, at + at_d, d[j]);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) d[j][k] = f2(0.0f);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) d[j][k] = fma2(f2(st.w), fma2(n[j][k], f2(-c), LN ? u[j][k] + f2(-m) : u[j][k]), d[j][k]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) mine.template take<S>(j, at + at_d, d[j]);
    }
    F2 q[2] = {f2(0.0f), f2(0.0f)}, e = f2(0.0f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      F2 t[4], w[4];
      if (has_dx) {
#pragma unroll
        for (int k = 0; k < 4; ++k) t[k] = f2(p.x_scale) * d[j][k];
        mine.template put<S, true>(j, dx, t);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) d[j][k] = d[j][k] * f2(p.o_scale);
      if (has_o) {
        mine.template take<B>(j, at + at_o, n[j]);
        if (post)
#pragma unroll
          for (int k = 0; k < 4; ++k) n[j][k] = (LN ? n[j][k] + f2(-st.x) : n[j][k]) * f2(st.y);
      }
      if constexpr (!KEEP)
        if (post) mine.weight(j, p.w1, p.pdt, p.w_off, w);
      if (gated) {
        if (GATE || has_dgate) {  // z again, from the normalised output
          F2 z[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) z[k] = post ? n[j][k] * (KEEP ? w1[KEEP ? j : 0][k] : w[k]) : n[j][k];
          if (LN && post && p.c1) {
            mine.global(j, p.c1, p.pdt, 0.0f, t);
#pragma unroll
            for (int k = 0; k < 4; ++k) z[k] = z[k] + t[k];
          }
          if constexpr (GATE) {
#pragma unroll
            for (int k = 0; k < 4; ++k) ag[j][k] = fma2(d[j][k], z[k], ag[j][k]);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) z[k] = z[k] * d[j][k];
            mine.template put<B, true>(j, dgate, z);
          }
        }
        mine.global(j, gate, gate_rows ? B : p.pdt, 0.0f, t);
#pragma unroll
        for (int k = 0; k < 4; ++k) d[j][k] = d[j][k] * t[k];
      }
      if (post) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          b1.aw[j][k] = fma2(d[j][k], n[j][k], b1.aw[j][k]);
          if constexpr (LN) b1.ac[j][k] = b1.ac[j][k] + d[j][k];
          d[j][k] = d[j][k] * (KEEP ? w1[KEEP ? j : 0][k] : w[k]);
          q[k & 1] = fma2(d[j][k], n[j][k], q[k & 1]);
          if constexpr (LN) e = e + d[j][k];
        }
      }
    }
    if (post) {
      means(q, e, c, m);
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) d[j][k] = f2(st.y) * fma2(n[j][k], f2(-c), LN ? d[j][k] + f2(-m) : d[j][k]);
    }
    if (has_do) {
#pragma unroll
      for (int j = 0; j < NV; ++j) mine.template put<B, true>(j, d_o, d[j]);
      d_o += do_step;
    }
    if (has_dx) dx += dx_step;
    if (has_dgate) dgate += dgate_step;
    if (gate_rows) gate += gate_step;
    stage = stage + 1 >= stages ? 0 : stage + 1;
  }
  if (!p.sums) return;
  auto leave = [&](int which, F2 (&a)[NV][4]) {
    char* to = reinterpret_cast<char*>(p.sums + ((size_t)blockIdx.x * NORM_SUMS + which) * p.D);
#pragma unroll
    for (int j = 0; j < NV; ++j) mine.template put<MOE_DTYPE_FP32, true>(j, to, a[j]);
  };
  if (post) leave(0, b1.aw);
  if (pre) leave(2, b2.aw);
  if constexpr (LN) {
    if (post) leave(1, b1.ac);
    if (pre) leave(3, b2.ac);
  }
  if constexpr (GATE) leave(4, ag);
}

// The whole call's rms form for long rows, of which an SM has room for one CTA: two rows
// at a time, so that one's arithmetic fills the other's barriers (335 -> 291 us where it
// was taken), the weights in shared memory to make registers for them.  One place a tensor and row in the ring, filled
// again as soon as it has been read.
template <bool GATE, int S, int B, bool ALL>
__global__ void __launch_bounds__(512) norm_bwd_pairs_kernel(const NormParams p) {
  constexpr int NV = 2;
  extern __shared__ __align__(16) char smem[];
  __shared__ float red[2 * 2 * NORM_MAX_WARPS];
  const int tid = threadIdx.x;
  const int row = ALL ? p.D : p.places;
  const Mine<NV, ALL> mine(tid, blockDim.x, p.nvec, row);
  Group grp{red, 0, (int)blockDim.x >> 5, tid >> 5, 0};
  char* const ring = smem;
  const uint32_t at_h = row * esize(S), at_d = at_h + row * esize(B), at_o = at_d + row * esize(S), row_bytes = at_o + row * esize(B);
  char *const sw1 = ring + 2 * row_bytes, *const sw2 = sw1 + row * 4;
  const int64_t row0 = 2 * (int64_t)blockIdx.x, step = 2 * (int64_t)gridDim.x;
  const int pairs = (int)(((p.T + 1) / 2 - blockIdx.x + gridDim.x - 1) / gridDim.x);
  const char* in[4] = {static_cast<const char*>(p.y) + row0 * p.y_ld * esize(S), static_cast<const char*>(p.dh) + row0 * p.dh_ld * esize(B),
                       static_cast<const char*>(p.dy) + row0 * p.dy_ld * esize(S), static_cast<const char*>(p.o) + row0 * p.o_ld * esize(B)};
  const int64_t ld[4] = {p.y_ld * esize(S), p.dh_ld * esize(B), p.dy_ld * esize(S), p.o_ld * esize(B)};
  char *dx = static_cast<char*>(p.dx) + row0 * p.dx_ld * esize(S), *d_o = static_cast<char*>(p.d_o) + row0 * p.do_ld * esize(B);
  const int64_t dx_ld = p.dx_ld * esize(S), do_ld = p.do_ld * esize(B);
  const float* stat = p.stats + 4 * row0;
  grid_dependency_wait();
  // both rows of a tensor for the next pair (the batch's last may have one)
  int64_t left = p.T - row0;  // rows from this pair's first on
  auto fetch = [&](auto which, bool on, bool two) {
    constexpr int K = decltype(which)::value, DT = K == 0 || K == 2 ? S : B;
    char* const at = ring + (K == 0 ? 0 : K == 1 ? at_h : K == 2 ? at_d : at_o);
    if (on) {
      mine.template fetch<DT>(at, in[K]);
      if (two) mine.template fetch<DT>(at + row_bytes, in[K] + ld[K]);
      in[K] += (int64_t)step * ld[K];
    }
    cp_async_commit();
  };
  constexpr std::integral_constant<int, 0> k0{};
  constexpr std::integral_constant<int, 1> k1{};
  constexpr std::integral_constant<int, 2> k2{};
  constexpr std::integral_constant<int, 3> k3{};
  if constexpr (!ALL) mine.clear(ring, 2 * row_bytes);
  fetch(k0, pairs > 0, left > 1);
  fetch(k1, pairs > 0, left > 1);
  fetch(k2, pairs > 0, left > 1);
  fetch(k3, pairs > 0, left > 1);
#pragma unroll
  for (int j = 0; j < NV; ++j)
    {  // a thread's own weights into its own places
      F2 w[4];
      mine.weight(j, p.w1, p.pdt, p.w_off, w);
      Raw<MOE_DTYPE_FP32> r = pack<MOE_DTYPE_FP32>(w);
      char* to = sw1 + mine.off[j];
      *reinterpret_cast<uint4*>(to) = r.q[0], *reinterpret_cast<uint4*>(to + mine.plane) = r.q[1];
      mine.weight(j, p.w2, p.pdt, p.w_off, w);
      r = pack<MOE_DTYPE_FP32>(w);
      to += row * 4;
      *reinterpret_cast<uint4*>(to) = r.q[0], *reinterpret_cast<uint4*>(to + mine.plane) = r.q[1];
    }
  F2 a1[NV][4], a2[NV][4], ag[GATE ? NV : 1][4];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      a1[j][k] = a2[j][k] = f2(0.0f);
      if constexpr (GATE) ag[j][k] = f2(0.0f);
    }
#pragma unroll 1
  for (int i = 0; i < pairs; ++i) {
    const bool two = left > 1, more = i + 1 < pairs, more_two = left - step > 1;
    left -= step;
    float r1[2], r2[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float* st = stat + (two ? 4 * r : 0);
      r1[r] = st[1], r2[r] = st[3];
    }
    stat += 4 * step;
    F2 d[2][NV][4], n[2][NV][4];
    float s[2];
    cp_async_wait(2);  // y and dh
    {
      F2 q[2] = {f2(0.0f), f2(0.0f)};
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        F2 w[4];
        mine.template take<MOE_DTYPE_FP32>(j, sw2, w);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if (r && !two) break;
          mine.template take<S>(j, ring + r * row_bytes, n[r][j]);
          mine.template take<B>(j, ring + r * row_bytes + at_h, d[r][j]);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            n[r][j][k] = n[r][j][k] * f2(r2[r]);
            a2[j][k] = fma2(d[r][j][k], n[r][j][k], a2[j][k]);
            d[r][j][k] = d[r][j][k] * w[k];
            q[r] = fma2(d[r][j][k], n[r][j][k], q[r]);
          }
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float2 a = split(q[r]);
        s[r] = a.x + a.y;
      }
    }
    group_sums(s, grp);
    fetch(k0, more, more_two);  // (the sums have used them)
    fetch(k1, more, more_two);
    cp_async_wait(3);  // dy
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float c = s[r] * p.inv_d;
      if (r && !two) break;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        F2 t[4];
        mine.template take<S>(j, ring + r * row_bytes + at_d, t);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          d[r][j][k] = fma2(f2(r2[r]), fma2(n[r][j][k], f2(-c), d[r][j][k]), t[k]);
          t[k] = f2(p.x_scale) * d[r][j][k];
          d[r][j][k] = d[r][j][k] * f2(p.o_scale);
        }
        mine.template put<S, true>(j, dx + r * dx_ld, t);
      }
    }
    dx += step * dx_ld;
    cp_async_wait(2);  // o
    {
      F2 q[2] = {f2(0.0f), f2(0.0f)};
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        F2 w[4], g[GATE ? 4 : 1];
        mine.template take<MOE_DTYPE_FP32>(j, sw1, w);
        if constexpr (GATE) mine.global(j, p.gate, p.pdt, 0.0f, g);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if (r && !two) break;
          mine.template take<B>(j, ring + r * row_bytes + at_o, n[r][j]);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            n[r][j][k] = n[r][j][k] * f2(r1[r]);
            if constexpr (GATE) {
              ag[j][k] = fma2(d[r][j][k], n[r][j][k] * w[k], ag[j][k]);
              d[r][j][k] = d[r][j][k] * g[k];
            }
            a1[j][k] = fma2(d[r][j][k], n[r][j][k], a1[j][k]);
            d[r][j][k] = d[r][j][k] * w[k];
            q[r] = fma2(d[r][j][k], n[r][j][k], q[r]);
          }
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float2 a = split(q[r]);
        s[r] = a.x + a.y;
      }
    }
    group_sums(s, grp);
    fetch(k2, more, more_two);
    fetch(k3, more, more_two);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float c = s[r] * p.inv_d;
      if (r && !two) break;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int k = 0; k < 4; ++k) d[r][j][k] = f2(r1[r]) * fma2(n[r][j][k], f2(-c), d[r][j][k]);
        mine.template put<B, true>(j, d_o + r * do_ld, d[r][j]);
      }
    }
    d_o += step * do_ld;
  }
  if (!p.sums) return;
  auto leave = [&](int which, F2 (&a)[NV][4]) {
    char* to = reinterpret_cast<char*>(p.sums + ((size_t)blockIdx.x * NORM_SUMS + which) * p.D);
#pragma unroll
    for (int j = 0; j < NV; ++j) mine.template put<MOE_DTYPE_FP32, true>(j, to, a[j]);
  };
  leave(0, a1);
  leave(2, a2);
  if constexpr (GATE) leave(4, ag);
}

cudaError_t launch_norm_bwd(const NormParams& p, bool gate_sum, bool pairs, unsigned grid, unsigned threads, size_t smem, cudaStream_t st) {
  auto by_type = [&](auto s, auto b) {
    constexpr int S = decltype(s)::value, B = decltype(b)::value;
    auto by_form = [&](auto gate) {
      constexpr bool G = decltype(gate)::value;
      if (pairs) return p.whole == 2 ? norm_bwd_pairs_kernel<G, S, B, true> : norm_bwd_pairs_kernel<G, S, B, false>;
      if (p.D > 8192) return p.layer ? norm_bwd_kernel<4, true, G, S, B, 0> : norm_bwd_kernel<4, false, G, S, B, 0>;
      if (p.layer)
        return p.whole == 2 ? norm_bwd_kernel<2, true, G, S, B, 2>
               : p.whole    ? norm_bwd_kernel<2, true, G, S, B, 1>
                            : norm_bwd_kernel<2, true, G, S, B, 0>;
      return p.whole == 2 ? norm_bwd_kernel<2, false, G, S, B, 2>
             : p.whole    ? norm_bwd_kernel<2, false, G, S, B, 1>
                          : norm_bwd_kernel<2, false, G, S, B, 0>;
    };
    auto kernel = gate_sum ? by_form(std::true_type{}) : by_form(std::false_type{});
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
