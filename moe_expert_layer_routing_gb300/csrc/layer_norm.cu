// Layer normalisation (and its form without a mean, RMS) forward and backward, with the residual add in
// front of the forward, the skip connection's gradient added behind the backward, and the weight
// gradients' reduction over the rows.
//
//   forward   s = round(x + r),  mu = mean(s),  q = 1 / sqrt(mean((s - mu)^2) + eps),
//             y = (s - mu) q gamma + beta                              (RMS: mu = 0)
//   backward  xh = (s - mu) q,  w = dy gamma,
//             dx = q (w - mean(w) - xh mean(w xh)) + dres              (RMS: no mean(w))
//             dgamma = sum_t dy xh,  dbeta = sum_t dy
//
// The statistics are of the rounded sum s, which is what the backward reads again.  All arithmetic and all
// sums are fp32; the variance is that of the differences from the mean, never a difference of squares.
#include <cuda_runtime.h>

#include <algorithm>

#include "moebwd_internal.h"
#include "mx_device.cuh"

namespace moebwd {

struct LnFwdArgs {
  const void *x, *r, *gamma, *beta;
  void *y, *sum;
  float *mean, *rstd;
  int64_t ldx, ldr, T;
  int H, rms;
  float eps;
};

struct LnBwdArgs {
  const void *dy, *x, *gamma, *dres;
  const float *mean, *rstd;
  void* dx;
  float* part;  // [2][G][H]: dgamma's and dbeta's partial sums of G groups of rows
  int64_t lddy, ldx, ldres, T;
  int H, rms, G;
};

__device__ __forceinline__ float ln_ld(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float ln_ld(const uint16_t* p, int64_t i) { return bf16_bits_to_float(p[i]); }
__device__ __forceinline__ void ln_st(float* p, int64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void ln_st(uint16_t* p, int64_t i, float v) { p[i] = float_to_bf16_bits(v); }
// the value as the type holds it
__device__ __forceinline__ float ln_round(float v, const float*) { return v; }
__device__ __forceinline__ float ln_round(float v, const uint16_t*) {
  return bf16_bits_to_float(float_to_bf16_bits(v));
}

constexpr int kLnThreads = 256;

// Sums of a and b over the block, in a fixed order, to every thread; `red` holds 2 * 8 floats.
__device__ __forceinline__ void ln_block_sum2(float& a, float& b, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  const int w = threadIdx.x >> 5;
  __syncthreads();  // the last call's readers are through
  if ((threadIdx.x & 31) == 0) {
    red[w] = a;
    red[8 + w] = b;
  }
  __syncthreads();
  a = b = 0.f;
#pragma unroll
  for (int i = 0; i < kLnThreads / 32; ++i) {
    a += red[i];
    b += red[8 + i];
  }
}

// Any width, alignment and stride: a block walks rows, three passes over each (the second and third hit
// the caches).
template <typename X, typename W>
__global__ void __launch_bounds__(kLnThreads) ln_fwd_any_kernel(const LnFwdArgs a) {
  __shared__ float red[16];
  pdl_wait();
  pdl_trigger();
  const X *x = static_cast<const X*>(a.x), *r = static_cast<const X*>(a.r);
  const W *gamma = static_cast<const W*>(a.gamma), *beta = static_cast<const W*>(a.beta);
  X *y = static_cast<X*>(a.y), *sum = static_cast<X*>(a.sum);
  const float inv = 1.f / (float)a.H;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    auto at = [&](int i) {
      const float v = ln_ld(x, t * a.ldx + i);
      return r ? ln_round(v + ln_ld(r, t * a.ldr + i), x) : v;
    };
    float s = 0.f, q = 0.f;
    if (!a.rms)
      for (int i = threadIdx.x; i < a.H; i += kLnThreads) s += at(i);
    ln_block_sum2(s, q, red);
    const float mu = s * inv;
    s = q = 0.f;
    for (int i = threadIdx.x; i < a.H; i += kLnThreads) {
      const float d = at(i) - mu;
      s = fmaf(d, d, s);
    }
    ln_block_sum2(s, q, red);
    const float rs = 1.f / sqrtf(s * inv + a.eps);
    for (int i = threadIdx.x; i < a.H; i += kLnThreads) {
      const float v = at(i);
      if (sum) ln_st(sum, t * a.H + i, v);
      const float n = (v - mu) * rs * ln_ld(gamma, i);
      ln_st(y, t * a.H + i, beta ? n + ln_ld(beta, i) : n);
    }
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[t] = mu;
      a.rstd[t] = rs;
    }
  }
}

template <typename X, typename W>
__global__ void __launch_bounds__(kLnThreads) ln_bwd_dx_any_kernel(const LnBwdArgs a) {
  __shared__ float red[16];
  pdl_wait();
  pdl_trigger();
  const X *dy = static_cast<const X*>(a.dy), *x = static_cast<const X*>(a.x), *dres = static_cast<const X*>(a.dres);
  const W* gamma = static_cast<const W*>(a.gamma);
  X* dx = static_cast<X*>(a.dx);
  const float inv = 1.f / (float)a.H;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const float mu = a.rms ? 0.f : a.mean[t], rs = a.rstd[t];
    float c1 = 0.f, c2 = 0.f;
    for (int i = threadIdx.x; i < a.H; i += kLnThreads) {
      const float w = ln_ld(dy, t * a.lddy + i) * ln_ld(gamma, i);
      c1 = fmaf(w, (ln_ld(x, t * a.ldx + i) - mu) * rs, c1);
      c2 += w;
    }
    ln_block_sum2(c1, c2, red);
    c1 *= inv;
    c2 = a.rms ? 0.f : c2 * inv;
    for (int i = threadIdx.x; i < a.H; i += kLnThreads) {
      const float w = ln_ld(dy, t * a.lddy + i) * ln_ld(gamma, i);
      const float xh = (ln_ld(x, t * a.ldx + i) - mu) * rs;
      float d = rs * (w - c2 - xh * c1);
      if (dres) d += ln_ld(dres, t * a.ldres + i);
      ln_st(dx, t * a.H + i, d);
    }
  }
}

// Partial column sums: block (column tile of 32, row group g), eight rows at a time, a warp each.
template <typename X>
__global__ void __launch_bounds__(kLnThreads) ln_bwd_part_any_kernel(const LnBwdArgs a) {
  __shared__ float red[2][8][32];
  pdl_wait();
  pdl_trigger();
  const X *dy = static_cast<const X*>(a.dy), *x = static_cast<const X*>(a.x);
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + lane, g = blockIdx.y;
  const int64_t t0 = a.T * g / a.G, t1 = a.T * (g + 1) / a.G;
  float sg = 0.f, sb = 0.f;
  if (i < a.H)
    for (int64_t t = t0 + w; t < t1; t += 8) {
      const float d = ln_ld(dy, t * a.lddy + i);
      sg = fmaf(d, (ln_ld(x, t * a.ldx + i) - (a.rms ? 0.f : a.mean[t])) * a.rstd[t], sg);
      sb += d;
    }
  red[0][w][lane] = sg;
  red[1][w][lane] = sb;
  __syncthreads();
  if (w < 2 && i < a.H) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) v += red[w][k][lane];
    a.part[((int64_t)w * a.G + g) * a.H + i] = v;
  }
}

// dgamma and dbeta (grid.y) from the partial sums of the G row groups: thread columns of 32, the groups
// split over eight warps, all in a fixed order.
__global__ void __launch_bounds__(kLnThreads) ln_bwd_reduce_kernel(const float* part, int G, int H, float* dgamma,
                                                                   float* dbeta, int accumulate) {
  __shared__ float red[8][32];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + lane;
  float* out = blockIdx.y ? dbeta : dgamma;
  float s = 0.f;
  if (i < H && out)
    for (int g = w; g < G; g += 8) s += part[((int64_t)blockIdx.y * G + g) * H + i];
  red[w][lane] = s;
  __syncthreads();
  if (w == 0 && i < H && out) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) v += red[k][lane];
    out[i] = accumulate ? out[i] + v : v;
  }
}

// Row groups of the backward's partial sums.
static int ln_groups(int64_t T) { return (int)std::max<int64_t>(1, std::min<int64_t>(1024, (T + 31) / 32)); }

static int ln_check(const char* who, int kind, int x_dtype, int w_dtype, int64_t T, int64_t H) {
  if (kind != MOE_NORM_LAYER && kind != MOE_NORM_RMS) return fail(MOE_ERR_INVALID, "%s: bad kind", who);
  if ((x_dtype != MOE_DT_BF16 && x_dtype != MOE_DT_F32) || (w_dtype != MOE_DT_BF16 && w_dtype != MOE_DT_F32))
    return fail(MOE_ERR_INVALID, "%s: bad dtype", who);
  if (T < 0 || H <= 0) return fail(MOE_ERR_INVALID, "%s: bad sizes (need T >= 0, H >= 1)", who);
  if (H > INT32_MAX / 8) return fail(MOE_ERR_UNSUPPORTED, "%s: H too large", who);
  return MOE_OK;
}

static int ln_aligned(const char* who, const void* p, int dtype) {
  return (reinterpret_cast<uintptr_t>(p) & (dtype == MOE_DT_BF16 ? 1 : 3))
             ? fail(MOE_ERR_INVALID, "%s: a tensor is not aligned to its element", who)
             : MOE_OK;
}

}  // namespace moebwd

using namespace moebwd;

extern "C" int layer_norm_fwd(int kind, const void* x, int64_t ldx, const void* residual, int64_t ldr,
                              const void* gamma, const void* beta, int x_dtype, int w_dtype, int64_t T, int64_t H,
                              float eps, void* y, void* sum, float* mean, float* rstd, moe_stream_t stream) {
  clear_error();
  int rc = ln_check("layer_norm_fwd", kind, x_dtype, w_dtype, T, H);
  if (rc) return rc;
  if (!(eps >= 0.f)) return fail(MOE_ERR_INVALID, "layer_norm_fwd: eps must be >= 0");
  if (T == 0) return MOE_OK;
  if (!x || !gamma || !y || !rstd) return fail(MOE_ERR_INVALID, "layer_norm_fwd: null pointer");
  if (kind == MOE_NORM_LAYER && !mean) return fail(MOE_ERR_INVALID, "layer_norm_fwd: mean needed");
  if (residual && !sum) return fail(MOE_ERR_INVALID, "layer_norm_fwd: a residual needs the sum output");
  if (ldx < H || (residual && ldr < H)) return fail(MOE_ERR_INVALID, "layer_norm_fwd: row stride below H");
  for (const void* p : {x, residual, static_cast<const void*>(y), static_cast<const void*>(sum)})
    if ((rc = ln_aligned("layer_norm_fwd", p, x_dtype))) return rc;
  for (const void* p : {gamma, beta})
    if ((rc = ln_aligned("layer_norm_fwd", p, w_dtype))) return rc;
  LnFwdArgs a{x, residual, gamma, beta, y, sum, kind == MOE_NORM_LAYER ? mean : nullptr, rstd, ldx, ldr, T, (int)H,
              kind == MOE_NORM_RMS, eps};
  const int grid = (int)std::min<int64_t>(T, 65536);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  auto kern = x_dtype == MOE_DT_BF16
                  ? (w_dtype == MOE_DT_BF16 ? ln_fwd_any_kernel<uint16_t, uint16_t> : ln_fwd_any_kernel<uint16_t, float>)
                  : (w_dtype == MOE_DT_BF16 ? ln_fwd_any_kernel<float, uint16_t> : ln_fwd_any_kernel<float, float>);
  return launch_pdl(kern, dim3(grid), dim3(kLnThreads), 0, st, "layer_norm_fwd", a);
}

extern "C" size_t layer_norm_bwd_workspace_size(int64_t T, int64_t H) {
  if (T <= 0 || H <= 0 || H > INT32_MAX / 8) return 0;
  return sizeof(float) * 2 * (size_t)ln_groups(T) * (size_t)H;
}

extern "C" int layer_norm_bwd(int kind, const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* gamma,
                              const float* mean, const float* rstd, const void* dres, int64_t ldres, int x_dtype,
                              int w_dtype, int64_t T, int64_t H, void* dx, float* dgamma, float* dbeta, int accumulate,
                              void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  clear_error();
  int rc = ln_check("layer_norm_bwd", kind, x_dtype, w_dtype, T, H);
  if (rc) return rc;
  if (accumulate != 0 && accumulate != 1) return fail(MOE_ERR_INVALID, "layer_norm_bwd: accumulate must be 0 or 1");
  if (!dgamma) return fail(MOE_ERR_INVALID, "layer_norm_bwd: null pointer");
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0) {  // sums over no rows
    if (accumulate) return MOE_OK;
    rc = cuda_check(cudaMemsetAsync(dgamma, 0, sizeof(float) * (size_t)H, st), "memset dgamma");
    if (!rc && dbeta) rc = cuda_check(cudaMemsetAsync(dbeta, 0, sizeof(float) * (size_t)H, st), "memset dbeta");
    return rc;
  }
  if (!dy || !x || !gamma || !rstd || !dx || !workspace) return fail(MOE_ERR_INVALID, "layer_norm_bwd: null pointer");
  if (kind == MOE_NORM_LAYER && !mean) return fail(MOE_ERR_INVALID, "layer_norm_bwd: mean needed");
  if (lddy < H || ldx < H || (dres && ldres < H)) return fail(MOE_ERR_INVALID, "layer_norm_bwd: row stride below H");
  for (const void* p : {dy, x, dres, static_cast<const void*>(dx)})
    if ((rc = ln_aligned("layer_norm_bwd", p, x_dtype))) return rc;
  if ((rc = ln_aligned("layer_norm_bwd", gamma, w_dtype))) return rc;
  if (reinterpret_cast<uintptr_t>(workspace) & 255)
    return fail(MOE_ERR_INVALID, "layer_norm_bwd: workspace must be 256-byte aligned");
  const size_t need = layer_norm_bwd_workspace_size(T, H);
  if (workspace_bytes < need)
    return fail(MOE_ERR_INVALID, "layer_norm_bwd: workspace too small (%zu < %zu)", workspace_bytes, need);
  LnBwdArgs a{dy, x, gamma, dres, mean, rstd, dx, static_cast<float*>(workspace), lddy, ldx, ldres, T, (int)H,
              kind == MOE_NORM_RMS, ln_groups(T)};
  const int grid = (int)std::min<int64_t>(T, 65536);
  auto kern = x_dtype == MOE_DT_BF16 ? (w_dtype == MOE_DT_BF16 ? ln_bwd_dx_any_kernel<uint16_t, uint16_t>
                                                               : ln_bwd_dx_any_kernel<uint16_t, float>)
                                     : (w_dtype == MOE_DT_BF16 ? ln_bwd_dx_any_kernel<float, uint16_t>
                                                               : ln_bwd_dx_any_kernel<float, float>);
  const int tiles = (int)((H + 31) / 32);
  auto part = x_dtype == MOE_DT_BF16 ? ln_bwd_part_any_kernel<uint16_t> : ln_bwd_part_any_kernel<float>;
  if ((rc = launch_pdl(kern, dim3(grid), dim3(kLnThreads), 0, st, "layer_norm_bwd dx", a))) return rc;
  if ((rc = launch_pdl(part, dim3(tiles, a.G), dim3(kLnThreads), 0, st, "layer_norm_bwd partial sums", a))) return rc;
  return launch_pdl(ln_bwd_reduce_kernel, dim3(tiles, dbeta ? 2 : 1), dim3(kLnThreads), 0, st,
                    "layer_norm_bwd weight gradients", static_cast<const float*>(a.part), a.G, (int)H, dgamma, dbeta,
                    accumulate);
}
