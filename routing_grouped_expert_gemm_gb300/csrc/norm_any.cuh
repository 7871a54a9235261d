// Norms around a block for rows that are not whole vectors on 16-byte boundaries
// (norm_any_fwd.cu, norm_any_bwd.cu; norm.cuh has the formulas).
//
// Thread i of a CTA's NT owns elements i, i + NT, ... of every row: whatever the
// alignment a warp's accesses lie together, and the sums over the rows stay in the
// thread's registers.  Rows are fetched ahead in granules of 16 bytes (cp.async), so that
// the bytes under way cost no registers; element by element they leave shared memory,
// where the parameters lie as fp32 too if they fit beside two rows (ANY_ALL).  A row's
// first granule starts at most 14 bytes before it: a granule never straddles two
// allocations (they start on 256 bytes), and what lies before the row is not used.  The
// last one ends with the row.
// Where only the rows fit (ANY_ROWS) the parameters are read where they lie (8000 x 5952
// rms gradients in bf16: 439 us against 336), and rows of more than 8192 elements as well
// (ANY_NONE): two kernels for all the kinds of call.
#pragma once
#include "norm.cuh"

namespace moe {

// Elements a thread, of the forward and of the backward (which holds the sums besides),
// at 64 registers each.  The backward takes 8 where 4 would need too many threads: 8000 x
// 4001 in bf16 takes 193 us with 4, 223 with 8; layer norms in fp16 239 and 377, spilled.
constexpr int ANY_FWD = 8;
constexpr int any_bwd_per(int64_t D) { return D <= 4096 ? 4 : 8; }
constexpr int ANY_MAX_WARPS = 32, ANY_RESIDENT = 1024;  // (threads an SM)
constexpr int ANY_STAGES = 4, ANY_MAX_CTAS = 32;
static_assert(ANY_STAGES - 1 <= CP_ASYNC_MOST, "groups under way in a ring");
__host__ __device__ constexpr int any_slot(int64_t D, int dt) { return (int)((D * esize(dt) + 31) & ~15); }

__device__ __forceinline__ float load_any(const void* p, int e, int dt) {
  if (dt == MOE_DTYPE_FP32) return static_cast<const float*>(p)[e];
  if (dt == MOE_DTYPE_BF16) return __bfloat162float(static_cast<const bf16*>(p)[e]);
  return __half2float(static_cast<const __half*>(p)[e]);
}
enum { ANY_NONE, ANY_ROWS, ANY_ALL };  // what waits in shared memory
constexpr int any_wide(int mode) { return mode == ANY_NONE ? 16 : 8; }  // elements a thread of those two

template <int DT>
__device__ __forceinline__ float load1(const void* p, int e) {
  return load_any(p, e, DT);
}
// this thread's elements of a row or a vector of parameters, 0 outside it
template <int DT, int NE>
__device__ __forceinline__ void load_mine(const void* p, int D, float (&v)[NE]) {
#pragma unroll
  for (int j = 0; j < NE; ++j) {
    const int e = threadIdx.x + j * blockDim.x;
    v[j] = e < D ? load1<DT>(p, e) : 0.0f;
  }
}
// rounds to the type, stores unless p is null, returns what was rounded
template <int DT>
__device__ __forceinline__ float store1(void* p, int e, float v) {
  if constexpr (DT == MOE_DTYPE_FP32) {
    if (p) static_cast<float*>(p)[e] = v;
    return v;
  } else if constexpr (DT == MOE_DTYPE_BF16) {
    const bf16 w = __float2bfloat16_rn(v);
    if (p) static_cast<bf16*>(p)[e] = w;
    return __bfloat162float(w);
  } else {
    const __half w = __float2half_rn(v);
    if (p) static_cast<__half*>(p)[e] = w;
    return __half2float(w);
  }
}

// One tensor's rows, and where in a stage of the ring they wait
struct AnyRows {
  const char* base;  // or null
  int64_t pitch;
  uint32_t at, bytes;
  __device__ __forceinline__ AnyRows(const void* p, int64_t ld, int D, int dt, uint32_t& end)
      : base(static_cast<const char*>(p)), pitch(ld * esize(dt)), at(end), bytes((uint32_t)D * esize(dt)) {
    if (p) end += any_slot(D, dt);
  }
  __device__ __forceinline__ void fetch(char* stage, int64_t t) const {
    if (!base) return;
    const char* from = base + t * pitch;
    const uint32_t shift = (uint32_t)reinterpret_cast<uintptr_t>(from) & 15u, all = shift + bytes;
    from -= shift;
    const uint32_t to = smem_u32(stage + at);
    for (uint32_t c = threadIdx.x * 16; c < all; c += blockDim.x * 16) {
      const uint32_t n = all - c < 16u ? all - c : 16u;  // (the rest of the granule becomes zero)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + c), "l"(from + c), "r"(n) : "memory");
    }
  }
  // row t, in its stage or in global memory
  template <int MODE>
  __device__ __forceinline__ const char* row(const char* stage, int64_t t) const {
    const char* from = base + t * pitch;
    if constexpr (MODE != ANY_NONE) return stage + at + ((uint32_t)reinterpret_cast<uintptr_t>(from) & 15u);
    else return from;
  }
};

// A vector of parameters plus `off`; all ones where a norm (`weight`) has none
template <int MODE>
struct AnyParam {
  const void* p;
  int dt;
  float off;
  __device__ __forceinline__ AnyParam(const NormParams& q, const void* v, float offset, bool weight, char*& room)
      : p(v), dt(q.pdt), off(v ? offset : 1.0f) {
    if (MODE != ANY_ALL || !(v || weight)) return;
    float* sm = reinterpret_cast<float*>(room);
    room += q.D * 4;
    for (int e = threadIdx.x; e < q.D; e += blockDim.x) sm[e] = v ? load_any(v, e, dt) + off : 1.0f;
    p = sm;
  }
  template <int NE>
  __device__ __forceinline__ void mine(int D, float (&v)[NE]) const {
    if constexpr (MODE == ANY_ALL) {
      load_mine<MOE_DTYPE_FP32>(p, D, v);
      return;
    }
    if (!p) {
#pragma unroll
      for (int j = 0; j < NE; ++j) v[j] = 0.0f;
    } else if (dt == MOE_DTYPE_FP32) {
      load_mine<MOE_DTYPE_FP32>(p, D, v);
    } else if (dt == MOE_DTYPE_BF16) {
      load_mine<MOE_DTYPE_BF16>(p, D, v);
    } else {
      load_mine<MOE_DTYPE_FP16>(p, D, v);
    }
#pragma unroll
    for (int j = 0; j < NE; ++j)
      if (threadIdx.x + j * blockDim.x < D) v[j] += off;
  }
};

// The CTA's rows, one after the other: row(stage, t) on each, fetch(stage, t) ahead of it
template <typename Fetch>
__device__ __forceinline__ void any_first(const NormParams& p, char* ring, Fetch&& fetch) {
#pragma unroll 1
  for (int s = 0; s < p.stages; ++s) {
    const int64_t t = blockIdx.x + (int64_t)s * gridDim.x;
    if (t < p.T) fetch(ring + s * p.stage_bytes, t);
    cp_async_commit();
  }
}
template <int MODE, typename Fetch, typename Row>
__device__ __forceinline__ void any_rows(const NormParams& p, char* ring, Fetch&& fetch, Row&& row) {
  const int rows = (int)((p.T - blockIdx.x + gridDim.x - 1) / gridDim.x);
  int64_t t = blockIdx.x;
  char *at = ring, *old = ring;
#pragma unroll 1
  for (int i = 0; i < rows; ++i, t += gridDim.x) {
    if constexpr (MODE != ANY_NONE) {
      if (MODE == ANY_ROWS && i && p.stages == 1) {
        __syncthreads();
        fetch(ring, t);
        cp_async_commit();
      }
      cp_async_wait(p.stages - (i ? 2 : 1));
      __syncthreads();  // the row has come for everybody, and nobody is at the one before it any more
      if (i && p.stages > 1) {
        if (i - 1 + p.stages < rows) fetch(old, t + (int64_t)(p.stages - 1) * gridDim.x);
        cp_async_commit();
      }
    }
    row(at, t);
    old = at;
    at += p.stage_bytes;
    if (at == ring + p.stages * p.stage_bytes) at = ring;
  }
}

// the kernel of a call's types: f(stream type, branch type)
template <typename F>
cudaError_t any_by_type(const NormParams& p, F&& f) {
  constexpr std::integral_constant<int, MOE_DTYPE_FP32> f32{};
  constexpr std::integral_constant<int, MOE_DTYPE_BF16> b16{};
  constexpr std::integral_constant<int, MOE_DTYPE_FP16> f16{};
  if (p.sdt == MOE_DTYPE_BF16) return f(b16, b16);
  if (p.sdt == MOE_DTYPE_FP16) return f(f16, f16);
  return p.bdt == MOE_DTYPE_FP32 ? f(f32, f32) : p.bdt == MOE_DTYPE_BF16 ? f(f32, b16) : f(f32, f16);
}

}  // namespace moe
