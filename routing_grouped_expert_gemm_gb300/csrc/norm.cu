// Norms around a block and their gradients (moe_norm, moe_norm_bwd in
// include/moe.h): the C entries and the sums over the rows.  norm.cuh has the formulas.
#include <new>
#include <type_traits>

#include "norm_any.cuh"

namespace moe {

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
#pragma unroll 8
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

// Vectors of 8 that a thread owns, by the row's width, and the threads that share a row
int norm_nv(int64_t D) { return D <= 8192 ? 2 : 4; }
int norm_threads(int64_t D) {
  const int64_t per = 8 * norm_nv(D);
  return (int)(((D + per - 1) / per + 31) / 32 * 32);
}
// ... and the vectors' places in a ring, as elements
int64_t norm_places(int64_t D) { return (int64_t)norm_threads(D) * 8 * norm_nv(D); }
// The backward's CTAs: resident by threads and registers, but each leaves sums for
// every column, so not so many that those outweigh the rows (8 a CTA)
int64_t norm_grid(const moe_norm_plan* pl, int64_t T) {
  int64_t per_sm = 512 / norm_threads(pl->cfg.D);
  per_sm = per_sm < 1 ? 1 : per_sm > 16 ? 16 : per_sm;
  const int64_t enough = (T + 8 * pl->num_sms - 1) / (8 * pl->num_sms);
  per_sm = per_sm < enough ? per_sm : enough;
  const int64_t most = per_sm * pl->num_sms;
  return T < most ? T : most;
}

// Rows off vectors: threads of a CTA (`per` elements each), CTAs of the backward at most
// (each leaves sums, so eight rows a CTA where there are more than two CTAs an SM), and a
// call's threads, ring and grid
int any_threads(int64_t D, int per) { return (int)(((D + per - 1) / per + 31) / 32 * 32); }
int64_t any_bwd_grid(const moe_norm_plan* pl, int64_t T) {
  const int64_t n = T / 8 > 2 * pl->num_sms ? T / 8 : 2 * pl->num_sms, all = (int64_t)ANY_MAX_CTAS * pl->num_sms;
  const int64_t most = n < all ? n : all;
  return most < T ? most : T;
}
struct AnyCall {
  int64_t grid;
  int threads;
  size_t smem;
};
// row_bytes: of a row's tensors in the ring; params: vectors of parameters
AnyCall any_call(const moe_norm_plan* pl, NormParams& p, int per, int64_t row_bytes, int params, int64_t most) {
  const int threads = any_threads(p.D, per);
  const int64_t need = (p.T + pl->num_sms - 1) / pl->num_sms, w = params * 4 * (int64_t)p.D;
  int64_t per_sm = ANY_RESIDENT / threads;  // 0: too wide
  per_sm = per_sm < ANY_MAX_CTAS ? per_sm : ANY_MAX_CTAS;
  per_sm = per_sm < need ? per_sm : need;
  p.stage_bytes = (int)row_bytes;
  for (; per_sm >= 1; --per_sm) {
    int64_t grid = per_sm * pl->num_sms;
    grid = grid < most ? grid : most;
    const int64_t rows = (p.T + grid - 1) / grid, room = NORM_SMEM / per_sm - 1024;
    int64_t fit = room > w ? (room - w) / row_bytes : 0;
    p.smem_w = fit >= (rows < 2 ? rows : 2);
    if (!p.smem_w) {
      if (per_sm > 1) continue;
      fit = room / row_bytes;  // at least 1: 8192 elements of 20 bytes
    }
    fit = fit < rows ? fit : rows;
    p.stages = (int)(fit < ANY_STAGES ? fit : ANY_STAGES);
    return {grid, p.smem_w ? threads : any_threads(p.D, any_wide(ANY_ROWS)), (size_t)(p.stages * row_bytes + p.smem_w * w)};
  }
  p.stages = 0;
  return {pl->num_sms < most ? pl->num_sms : most, any_threads(p.D, any_wide(ANY_NONE)), 0};
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
  p.places = (int)norm_places(c.D);
  p.layer = c.kind == MOE_NORM_LAYER;
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
  // rows at a time on a CTA, fewer where the rows' ring or the batch do not ask for them
  p.group = norm_threads(c.D);
  const int64_t row_bytes = norm_places(c.D) * ((x ? norm_size(c.stream_dtype) : 0) + (o ? norm_size(c.branch_dtype) : 0) +
                                   (p.gate_rows ? norm_size(c.branch_dtype) : 0));
  const int64_t w_bytes = norm_places(c.D) * 4 * (c.post + c.pre);
  int64_t rows = norm_fwd_threads(norm_nv(c.D)) / p.group, need = (T + pl->num_sms - 1) / pl->num_sms;
  rows = rows < need ? rows : need;
  cudaError_t err;
  if (vec && row_bytes <= NORM_SMEM) {
    p.smem_w = need >= 2 * rows;
    while (rows > 1 && rows * row_bytes + p.smem_w * w_bytes > NORM_SMEM) --rows;
    if (rows * row_bytes + p.smem_w * w_bytes > NORM_SMEM) p.smem_w = 0;
    // rows ahead that fit
    int64_t fit = (NORM_SMEM - p.smem_w * w_bytes) / (rows * row_bytes);
    const int64_t use = (need + rows - 1) / rows;
    fit = fit < use ? fit : use;
    p.stages = (int)(fit < NORM_FWD_STAGES ? fit : NORM_FWD_STAGES);
    p.stage_bytes = (int)row_bytes;
    p.whole = p.stages == NORM_FWD_STAGES && c.D <= 8192 && p.smem_w && c.post && c.pre && x && o && y && !p.gate;
    if (p.whole && c.D % 512 == 0) p.whole = 2;
    const int64_t ctas = (T + rows - 1) / rows, grid = ctas < pl->num_sms ? ctas : pl->num_sms;
    err = launch_norm_fwd(p, (unsigned)grid, (unsigned)(rows * p.group), rows * p.stages * p.stage_bytes + p.smem_w * w_bytes,
                          (cudaStream_t)stream);
  } else {
    const int64_t slot = (o ? any_slot(c.D, c.branch_dtype) : 0) + (x ? any_slot(c.D, c.stream_dtype) : 0) +
                         (p.gate_rows ? any_slot(c.D, c.branch_dtype) : 0);
    const AnyCall a = any_call(pl, p, ANY_FWD, slot, c.post + c.pre + (p.c1 != nullptr) + (p.c2 != nullptr) + (p.gate && !p.gate_rows), T);
    err = launch_norm_fwd_any(p, (unsigned)a.grid, (unsigned)a.threads, a.smem, (cudaStream_t)stream);
  }
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

size_t moe_norm_workspace_bytes(const moe_norm_plan* plan, int64_t T) {
  if (!plan || T < 0) return 0;
  if (T == 0) return 256;
  const int64_t a = norm_grid(plan, T), b = any_bwd_grid(plan, T);
  return ((size_t)(a > b ? a : b) * NORM_SUMS * plan->cfg.D * 4 + 255) / 256 * 256;
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
  int64_t grid = norm_grid(pl, T);
  const int64_t row_bytes = norm_places(c.D) * ((c.pre ? norm_size(sd) + norm_size(bd) : 0) + (dy ? norm_size(sd) : 0) + (use_o ? norm_size(bd) : 0));
  cudaError_t err;
  if (vec && row_bytes <= NORM_SMEM) {
    // rows of the ring
    const int64_t per_sm = (grid + pl->num_sms - 1) / pl->num_sms, fit = NORM_SMEM / (per_sm * row_bytes), rows = (T + grid - 1) / grid;
    p.stages = (int)(fit < NORM_BWD_STAGES ? fit : NORM_BWD_STAGES);
    if (p.stages > rows) p.stages = (int)rows;
    if (p.stages < 1) p.stages = 1;
    p.stage_bytes = (int)row_bytes;
    p.whole = p.stages == NORM_BWD_STAGES && c.D <= 8192 && c.post && c.pre && dy && dx && d_o && (!p.gate || gate_sum);
    size_t smem = (size_t)p.stages * row_bytes;
    bool pairs = false;
    const size_t pair_bytes = 2 * row_bytes + 8 * norm_places(c.D);
    if (p.whole && c.kind == MOE_NORM_RMS && c.D > 4096 && T >= 4 * grid && pair_bytes <= NORM_SMEM) {
      pairs = true;  // two rows at a time, with the weights
      smem = pair_bytes;
    }
    if (p.whole && c.D % 512 == 0) p.whole = 2;
    err = launch_norm_bwd(p, gate_sum, pairs, (unsigned)grid, (unsigned)norm_threads(c.D), smem, stream);
  } else {
    const int64_t slot = (c.pre ? any_slot(c.D, sd) + any_slot(c.D, bd) : 0) + (dy ? any_slot(c.D, sd) : 0) +
                         (use_o ? any_slot(c.D, bd) : 0) + (p.gate_rows ? any_slot(c.D, bd) : 0) + (stats ? any_slot(4, MOE_DTYPE_FP32) : 0);
    const AnyCall a = any_call(pl, p, any_bwd_per(c.D), slot, c.post + c.pre + (p.gate ? (p.c1 != nullptr) + !p.gate_rows : 0), any_bwd_grid(pl, T));
    grid = a.grid;
    err = launch_norm_bwd_any(p, (unsigned)grid, (unsigned)a.threads, a.smem, stream);
  }
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
