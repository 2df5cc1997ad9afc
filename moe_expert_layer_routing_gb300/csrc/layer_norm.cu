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
// sums are fp32; the variance is that of the differences from the mean, never a difference of squares.  y and dx
// are rounded once; dgamma and dbeta stay fp32 and every sum has a fixed order.
//
// Bound by HBM: 65536 x 4096 bf16 with residual / skip gradient moves 2.15 GB each way, 317 us at the measured copy
// rate of 6.78 TB/s.  Measured: forward 344 us (6.3 TB/s: equal reads and writes), backward with the weight gradients
// 311 us (6.9 TB/s).  Three passes over each row with the caches' help had taken 747 and 1376 us, and rows above 8192
// columns still go that way: 16384 x 16384 bf16 without residual or skip gradient 453 us (2.4 TB/s) and 1125 us (1.4
// TB/s), bound by single-element accesses and the repeated reads.  Few rows are bound by latency: 2.7 us (forward) and
// 5 us (backward, two kernels) for 1 to 64 rows.  Rows that are not whole 16-byte pieces are bound by the shared-memory
// and store instructions of their single elements: fp32 32768 x 1111 at 3.7 to 4.0 TB/s, 16384 x 3001 at 5.4, bf16
// (2-byte elements) 32768 x 3001 at 3.6 to 3.8 TB/s with residual and skip gradient, 2.1 and 3.1 TB/s without.
#include <cuda_runtime.h>

#include <algorithm>
#include <initializer_list>

#include "moebwd_internal.h"
#include "mx_device.cuh"
#include "ptx.cuh"

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

// Rows above kLnMaxH columns: a block walks rows, three passes over each (the second and third hit the caches).
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

// dgamma and dbeta (grid.y) from the partial sums of the G row groups: a block takes 32 columns, its 32 warps every
// 32nd group, all in a fixed order.
constexpr int kLnReduceThreads = 1024;
__global__ void __launch_bounds__(kLnReduceThreads) ln_bwd_reduce_kernel(const float* part, int G, int H, float* dgamma,
                                                                         float* dbeta, int accumulate) {
  __shared__ float red[32][33];
  pdl_wait();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + lane;
  float* out = blockIdx.y ? dbeta : dgamma;
  float s = 0.f;
  if (i < H)
    for (int g = w; g < G; g += 32) s += part[((int64_t)blockIdx.y * G + g) * H + i];
  red[w][lane] = s;
  __syncthreads();
  if (w == 0 && i < H) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) v += red[k][lane];
    out[i] = accumulate ? out[i] + v : v;
  }
}

// ------------------------------------------------------------------------------------------
// Rows in registers
// ------------------------------------------------------------------------------------------
// A row belongs to a group of GT = 32 WPR threads (one to all eight warps of the block) and passes once: a
// thread holds CPT of its columns.  Blocks are persistent; rows come through a ring in shared memory by 16-byte
// asynchronous copies, so the rows in flight cost no registers.
//   vectors   rows and strides are multiples of 16 bytes: a thread holds NV vectors VEC wide (v GT + li of the
//             row) and copies what it alone reads, so the ring needs no barrier
//   shifted   rows of any width on an aligned base: the 16-byte pieces a row touches are copied as they lie (the
//             first begins in the row before it, the last is cut at the row's end), thread li reads the single
//             elements v GT + li behind a barrier
//   direct    an unaligned base: single elements from global memory
enum LnMode { kLnDirect = 0, kLnVector = 1, kLnShifted = 2 };

template <typename X, int CPT, int WPR, int MODE>
struct LnTile {
  static constexpr int VEC = MODE == kLnVector ? 16 / (int)sizeof(X) : 1;
  static constexpr int NV = CPT / VEC;
  static constexpr int GT = 32 * WPR;
  static constexpr int GROUPS = kLnThreads / GT;
  __device__ static int col(int v, int li) { return (v * GT + li) * VEC; }
  // (told apart at compile time for a whole block: the division costs the row kernels registers they spill)
  __device__ static int group() { return WPR == 8 ? 0 : threadIdx.x / GT; }
  __device__ static int li() { return WPR == 8 ? threadIdx.x : threadIdx.x % GT; }
  __device__ static void sync() {  // the group
    if constexpr (WPR == 1)
      __syncwarp();
    else if constexpr (WPR == 8)
      __syncthreads();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group()), "n"(GT) : "memory");
  }
};

// Bytes of a row's slot in the shifted ring.
__host__ __device__ constexpr int ln_row_bytes(int H, int es) { return ((H * es + 15) / 16 + 1) * 16; }

// One tensor's rows in the ring: tensor `which` of TENSORS.
template <typename X, int CPT, int WPR, int MODE, int TENSORS>
struct LnStream {
  using L = LnTile<X, CPT, WPR, MODE>;
  const X* p;
  int64_t ld;
  int H, which;
  char* ring;
  __device__ char* slot(int stage) const {  // shifted
    return ring + ((stage * TENSORS + which) * L::GROUPS + L::group()) * ln_row_bytes(H, sizeof(X));
  }
  __device__ uint4* slot(int stage, int v) const {  // vectors
    return reinterpret_cast<uint4*>(ring) + ((stage * TENSORS + which) * L::NV + v) * kLnThreads + threadIdx.x;
  }
  __device__ int shift(int64_t t) const { return (int)(reinterpret_cast<uintptr_t>(p + t * ld) & 15); }
  // copies of row t (nothing for a null tensor)
  __device__ void fetch(int64_t t, int stage) const {
    if (!p) return;
    const int li = L::li();
    if constexpr (MODE == kLnVector) {
#pragma unroll
      for (int v = 0; v < L::NV; ++v)
        if (L::col(v, li) < H) cp_async_16(smem_u32(slot(stage, v)), p + t * ld + L::col(v, li));
    } else if constexpr (MODE == kLnShifted) {
      const char* row = reinterpret_cast<const char*>(p + t * ld);
      const int d = shift(t), end = d + H * (int)sizeof(X);
      char* dst = slot(stage);
      for (int c = 16 * li; c < end; c += 16 * L::GT) cp_async_16_zfill(smem_u32(dst + c), row - d + c, min(16, end - c));
    }
  }
  // columns col(v, li) .. of row t, which the group's copies have brought (c < H)
  __device__ void read(int64_t t, int stage, int v, int c, float (&f)[L::VEC]) const;
};

__device__ __forceinline__ void ln_unpack(const uint4& w, float (&f)[4]) {
  f[0] = __uint_as_float(w.x);
  f[1] = __uint_as_float(w.y);
  f[2] = __uint_as_float(w.z);
  f[3] = __uint_as_float(w.w);
}
__device__ __forceinline__ void ln_unpack(const uint4& w, float (&f)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 ln_pack(const float (&f)[4]) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
__device__ __forceinline__ uint4 ln_pack(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// VEC weights from column c on, in fp32 (16-byte loads when VEC > 1).  Ordinary loads here and for mean and rstd: a
// kernel starts while the one before it on the stream still runs, and the read-only path (__ldg) is only for memory
// that nothing writes during the whole of a kernel.
template <int VEC>
__device__ __forceinline__ void ln_weights(const void* p, int bf16, int c, float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    f[0] = bf16 ? bf16_bits_to_float(static_cast<const uint16_t*>(p)[c]) : static_cast<const float*>(p)[c];
  } else if (!bf16) {
#pragma unroll
    for (int i = 0; i < VEC; i += 4) {
      const float4 w = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + c + i);
      f[i] = w.x;
      f[i + 1] = w.y;
      f[i + 2] = w.z;
      f[i + 3] = w.w;
    }
  } else if constexpr (VEC == 8) {
    ln_unpack(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + c), f);
  } else {
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + c);
    f[0] = __uint_as_float(w.x << 16);
    f[1] = __uint_as_float(w.x & 0xffff0000u);
    f[2] = __uint_as_float(w.y << 16);
    f[3] = __uint_as_float(w.y & 0xffff0000u);
  }
}

// VEC consecutive fp32 values (16-byte stores when VEC > 1)
template <int VEC>
__device__ __forceinline__ void ln_store(float* p, const float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    p[0] = f[0];
  } else {
#pragma unroll
    for (int i = 0; i < VEC; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
  }
}

__device__ __forceinline__ float ln_warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <typename X, int CPT, int WPR, int MODE, int TENSORS>
__device__ __forceinline__ void LnStream<X, CPT, WPR, MODE, TENSORS>::read(int64_t t, int stage, int v, int c,
                                                                           float (&f)[L::VEC]) const {
  if constexpr (MODE == kLnVector)
    ln_unpack(*slot(stage, v), f);
  else if constexpr (MODE == kLnShifted)
    f[0] = ln_ld(reinterpret_cast<const X*>(slot(stage) + shift(t)), c);
  else
    f[0] = ln_ld(p, t * ld + c);
}

// Resident blocks (registers) and rows of the ring, as many as 192 KB an SM hold.
__host__ __device__ constexpr int ln_fwd_blocks(int cpt, int es) { return cpt == 8 ? 4 : cpt <= 16 ? 3 : es == 2 ? 2 : 1; }
__host__ __device__ constexpr int ln_bwd_blocks(int cpt) { return cpt == 32 ? 1 : 2; }
__host__ __device__ constexpr int ln_stages(int blocks, int tensors, int cpt, int es) {
  return 196608 / (blocks * tensors * kLnThreads * cpt * es) > 6 ? 6 : 196608 / (blocks * tensors * kLnThreads * cpt * es);
}

// Forward.  Four rows of the ring and weights in registers: 350 us at 65536 x 4096 (three rows and the weights re-read
// from L1 for every row: 397 us).  The statistics of a row: each warp takes the mean and the squared differences of its own columns (two
// shuffle sums), the warps' pairs (n, mean, M2) are combined exactly: M2 = sum M2_w + n_w (mean_w - mean)^2.  So a
// row costs one barrier and no difference of squares.
template <typename X, int CPT, int WPR, int MODE>
__global__ void __launch_bounds__(kLnThreads, ln_fwd_blocks(CPT, sizeof(X))) ln_fwd_kernel(const LnFwdArgs a, int w_bf16) {
  using L = LnTile<X, CPT, WPR, MODE>;
  constexpr int VEC = L::VEC, NV = L::NV, S = ln_stages(ln_fwd_blocks(CPT, sizeof(X)), 2, CPT, sizeof(X));
  extern __shared__ uint4 ring[];
  __shared__ float wn[8], wmean[2][8], wm2[2][8];
  const LnStream<X, CPT, WPR, MODE, 2> x{static_cast<const X*>(a.x), a.ldx, a.H, 0, reinterpret_cast<char*>(ring)};
  const LnStream<X, CPT, WPR, MODE, 2> r{static_cast<const X*>(a.r), a.ldr, a.H, 1, reinterpret_cast<char*>(ring)};
  X *y = static_cast<X*>(a.y), *sum = static_cast<X*>(a.sum);
  const int li = L::li(), w = threadIdx.x >> 5, w0 = L::group() * WPR;
  const int64_t step = (int64_t)gridDim.x * L::GROUPS;
  const float inv = 1.f / (float)a.H;
  float n_w = 0.f;  // columns of this warp
#pragma unroll
  for (int v = 0; v < NV; ++v) n_w += L::col(v, li) < a.H ? (float)VEC : 0.f;
  n_w = ln_warp_sum(n_w);
  if (WPR > 1) {
    if ((threadIdx.x & 31) == 0) wn[w] = n_w;
    __syncthreads();
  }
  pdl_wait();
  pdl_trigger();
  float gamma[NV][VEC], beta[NV][VEC];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = L::col(v, li);
#pragma unroll
    for (int i = 0; i < VEC; ++i) gamma[v][i] = beta[v][i] = 0.f;
    if (c < a.H) {
      ln_weights<VEC>(a.gamma, w_bf16, c, gamma[v]);
      if (a.beta) ln_weights<VEC>(a.beta, w_bf16, c, beta[v]);
    }
  }
  auto fetch = [&](int64_t t, int stage) {
    if constexpr (MODE != kLnDirect) {
      if (t < a.T) {
        x.fetch(t, stage);
        r.fetch(t, stage);
      }
      cp_async_commit();
    }
  };
  int64_t t = (int64_t)blockIdx.x * L::GROUPS + L::group();
#pragma unroll
  for (int s = 0; s < S - 1; ++s) fetch(t + s * step, s);
  int stage = 0, par = 0;
  // a group leaves when its rows are through
  for (; t < a.T; t += step) {
    float f[NV][VEC];
    if constexpr (MODE == kLnShifted && WPR == 1) __syncwarp();  // the slot filled next was read by the whole group
    fetch(t + (S - 1) * step, stage == 0 ? S - 1 : stage - 1);  // the slot read last time round
    if constexpr (MODE != kLnDirect) cp_async_wait<S - 1>();
    if constexpr (MODE == kLnShifted) L::sync();
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = L::col(v, li);
#pragma unroll
      for (int i = 0; i < VEC; ++i) f[v][i] = 0.f;
      if (c < a.H) {
        x.read(t, stage, v, c, f[v]);
        if (r.p) {
          float q[VEC];
          r.read(t, stage, v, c, q);
#pragma unroll
          for (int i = 0; i < VEC; ++i) f[v][i] = ln_round(f[v][i] + q[i], x.p);
        }
        if (sum) {
          if constexpr (MODE == kLnVector)
            *reinterpret_cast<uint4*>(sum + t * a.H + c) = ln_pack(f[v]);
          else
            ln_st(sum, t * a.H + c, f[v][0]);
        }
      }
    }
    float mu = 0.f, m2 = 0.f;
    if (!a.rms) {
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < VEC; ++i) mu += f[v][i];
      mu = n_w > 0.f ? ln_warp_sum(mu) / n_w : 0.f;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (L::col(v, li) < a.H)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float d = f[v][i] - mu;
          m2 = fmaf(d, d, m2);
        }
    m2 = ln_warp_sum(m2);
    if constexpr (WPR > 1) {
      if ((threadIdx.x & 31) == 0) {
        wmean[par][w] = mu;
        wm2[par][w] = m2;
      }
      L::sync();  // the buffers alternate: the next row's writes meet no reader of this one
      mu = m2 = 0.f;
      if (!a.rms) {
#pragma unroll
        for (int k = 0; k < WPR; ++k) mu = fmaf(wn[w0 + k], wmean[par][w0 + k], mu);
        mu *= inv;
      }
#pragma unroll
      for (int k = 0; k < WPR; ++k) {
        const float d = wmean[par][w0 + k] - mu;
        m2 += a.rms ? wm2[par][w0 + k] : fmaf(wn[w0 + k] * d, d, wm2[par][w0 + k]);
      }
      par ^= 1;
    }
    const float rs = 1.f / sqrtf(m2 * inv + a.eps);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = L::col(v, li);
      if (c < a.H) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[v][i] = fmaf((f[v][i] - mu) * rs, gamma[v][i], beta[v][i]);
        if constexpr (MODE == kLnVector)
          *reinterpret_cast<uint4*>(y + t * a.H + c) = ln_pack(f[v]);
        else
          ln_st(y, t * a.H + c, f[v][0]);
      }
    }
    if (li == 0) {
      if (a.mean) a.mean[t] = mu;
      a.rstd[t] = rs;
    }
    stage = stage + 1 == S ? 0 : stage + 1;
  }
}

// Backward: dx and, in the thread's registers over all rows of its group, dgamma and dbeta of its columns; a
// block leaves one partial row of each.  With vectors a thread refills a slot as soon as it has read it (dy and x
// before the row's sums, the skip gradient at the row's end): S rows in flight (refilled at the start of the next row,
// S - 1 in flight: 394 instead of 316 us at 65536 x 4096; in the forward the same change cost 3%).
template <typename X, int CPT, int WPR, int MODE>
__global__ void __launch_bounds__(kLnThreads, ln_bwd_blocks(CPT)) ln_bwd_kernel(const LnBwdArgs a, int w_bf16) {
  using L = LnTile<X, CPT, WPR, MODE>;
  constexpr int VEC = L::VEC, NV = L::NV, GT = L::GT, S = ln_stages(ln_bwd_blocks(CPT), 3, CPT, sizeof(X));
  extern __shared__ uint4 ring[];
  __shared__ float r1[2][8], r2[2][8];
  const LnStream<X, CPT, WPR, MODE, 3> dy{static_cast<const X*>(a.dy), a.lddy, a.H, 0, reinterpret_cast<char*>(ring)};
  const LnStream<X, CPT, WPR, MODE, 3> x{static_cast<const X*>(a.x), a.ldx, a.H, 1, reinterpret_cast<char*>(ring)};
  const LnStream<X, CPT, WPR, MODE, 3> dres{static_cast<const X*>(a.dres), a.ldres, a.H, 2, reinterpret_cast<char*>(ring)};
  X* dx = static_cast<X*>(a.dx);
  const int li = L::li(), w = threadIdx.x >> 5, w0 = L::group() * WPR;
  const int64_t step = (int64_t)gridDim.x * L::GROUPS;
  const float inv = 1.f / (float)a.H;
  pdl_wait();
  pdl_trigger();
  float gamma[NV][VEC], ag[NV][VEC], ab[NV][VEC];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) gamma[v][i] = ag[v][i] = ab[v][i] = 0.f;
    if (L::col(v, li) < a.H) ln_weights<VEC>(a.gamma, w_bf16, L::col(v, li), gamma[v]);
  }
  int64_t t = (int64_t)blockIdx.x * L::GROUPS + L::group();
  // a row's copies are one group: with vectors S of them ahead, shifted S - 1
  constexpr int AHEAD = MODE == kLnVector ? S : S - 1;
  auto fetch = [&](int64_t t, int stage) {
    if (t < a.T) {
      dy.fetch(t, stage);
      x.fetch(t, stage);
    }
  };
  auto fetch_skip = [&](int64_t t, int stage) {
    if (t < a.T) dres.fetch(t, stage);
    cp_async_commit();
  };
  if constexpr (MODE != kLnDirect) {
#pragma unroll
    for (int s = 0; s < AHEAD; ++s) {
      fetch(t + s * step, s);
      fetch_skip(t + s * step, s);
    }
  }
  int stage = 0, par = 0;
  float mu_next = 0.f, rs_next = 0.f;  // a row ahead, like the ring
  auto stats = [&](int64_t t) {
    if (t < a.T) {
      mu_next = a.rms ? 0.f : a.mean[t];
      rs_next = a.rstd[t];
    }
  };
  stats(t);
  for (; t < a.T; t += step) {
    const float mu = mu_next, rs = rs_next;
    stats(t + step);
    if constexpr (MODE != kLnDirect) cp_async_wait<AHEAD - 1>();
    if constexpr (MODE == kLnShifted) L::sync();
    float wd[NV][VEC], xh[NV][VEC], c1 = 0.f, c2 = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = L::col(v, li);
#pragma unroll
      for (int i = 0; i < VEC; ++i) wd[v][i] = xh[v][i] = 0.f;
      if (c < a.H) {
        dy.read(t, stage, v, c, wd[v]);
        x.read(t, stage, v, c, xh[v]);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float d = wd[v][i];
          xh[v][i] = (xh[v][i] - mu) * rs;
          ag[v][i] = fmaf(d, xh[v][i], ag[v][i]);
          ab[v][i] += d;
          wd[v][i] = d * gamma[v][i];
          c1 = fmaf(wd[v][i], xh[v][i], c1);
          c2 += wd[v][i];
        }
      }
    }
    if constexpr (MODE == kLnVector) fetch(t + S * step, stage);  // the slots just read
    c1 = ln_warp_sum(c1);
    c2 = ln_warp_sum(c2);
    if constexpr (WPR > 1) {
      if ((threadIdx.x & 31) == 0) {
        r1[par][w] = c1;
        r2[par][w] = c2;
      }
      L::sync();
      c1 = c2 = 0.f;
#pragma unroll
      for (int k = 0; k < WPR; ++k) {
        c1 += r1[par][w0 + k];
        c2 += r2[par][w0 + k];
      }
      par ^= 1;
    }
    if constexpr (MODE == kLnShifted) {  // the group is through with the row before this one
      if constexpr (WPR == 1) __syncwarp();
      const int before = stage == 0 ? S - 1 : stage - 1;
      fetch(t + (S - 1) * step, before);
      fetch_skip(t + (S - 1) * step, before);
    }
    c1 *= inv;
    c2 = a.rms ? 0.f : c2 * inv;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = L::col(v, li);
      if (c < a.H) {
        float d[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) d[i] = rs * (wd[v][i] - c2 - xh[v][i] * c1);
        if (dres.p) {
          float q[VEC];
          dres.read(t, stage, v, c, q);
#pragma unroll
          for (int i = 0; i < VEC; ++i) d[i] += q[i];
        }
        if constexpr (MODE == kLnVector)
          *reinterpret_cast<uint4*>(dx + t * a.H + c) = ln_pack(d);
        else
          ln_st(dx, t * a.H + c, d[0]);
      }
    }
    if constexpr (MODE == kLnVector) fetch_skip(t + S * step, stage);
    stage = stage + 1 == S ? 0 : stage + 1;
  }
  // the block's partial rows: several groups' sums first, in order, through shared memory
  float* sm = reinterpret_cast<float*>(ring);
  if constexpr (WPR < 8) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if constexpr (MODE != kLnDirect) cp_async_wait<0>();
      __syncthreads();
#pragma unroll
      for (int v = 0; v < NV; ++v) ln_store<VEC>(sm + L::group() * (GT * CPT) + L::col(v, li), half ? ab[v] : ag[v]);
      __syncthreads();
      for (int c = threadIdx.x; c < a.H; c += kLnThreads) {
        float q = 0.f;
#pragma unroll
        for (int k = 0; k < L::GROUPS; ++k) q += sm[k * (GT * CPT) + c];
        a.part[((int64_t)half * a.G + blockIdx.x) * a.H + c] = q;
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = L::col(v, li);
      if (c < a.H) {
        ln_store<VEC>(a.part + (int64_t)blockIdx.x * a.H + c, ag[v]);
        ln_store<VEC>(a.part + ((int64_t)a.G + blockIdx.x) * a.H + c, ab[v]);
      }
    }
  }
}

// Variants by width: 16 columns a thread and one, two, four or eight warps a row (8 columns up to 256, 32 above
// 4096): narrower groups hold several rows of a block in flight, wider threads pay a row's sums over more columns.
typedef void (*LnFwdKernel)(const LnFwdArgs, int);
typedef void (*LnBwdKernel)(const LnBwdArgs, int);
constexpr int kLnMaxH = 8192;

#define LN_PICK(KERN, X, MODE)                                                                                     \
  (H <= 256 ? KERN<X, 8, 1, MODE> : H <= 512 ? KERN<X, 16, 1, MODE> : H <= 1024 ? KERN<X, 16, 2, MODE>             \
   : H <= 2048 ? KERN<X, 16, 4, MODE> : H <= 4096 ? KERN<X, 16, 8, MODE> : KERN<X, 32, 8, MODE>)

// Shifted rows pay per element: 12 columns a thread where they reach (32768 x 3001 bf16: backward 267 -> 217 us,
// forward 235 -> 209 us; 65536 x 333: 62 -> 54 and 51 -> 44 us).
static bool ln_twelve(int64_t H, int mode) {
  return mode == kLnShifted && ((H > 256 && H <= 384) || (H > 512 && H <= 768) || (H > 1024 && H <= 1536) || (H > 2048 && H <= 3072));
}
#define LN_PICK_SHIFTED(KERN, X)                                                                                   \
  (!ln_twelve(H, kLnShifted) ? LN_PICK(KERN, X, kLnShifted) : H <= 384 ? KERN<X, 12, 1, kLnShifted>                \
   : H <= 768 ? KERN<X, 12, 2, kLnShifted> : H <= 1536 ? KERN<X, 12, 4, kLnShifted> : KERN<X, 12, 8, kLnShifted>)

static int ln_cpt(int64_t H, int mode) { return ln_twelve(H, mode) ? 12 : H <= 256 ? 8 : H <= 4096 ? 16 : 32; }
static int ln_rows_per_block(int64_t H) { return H <= 512 ? 8 : H <= 1024 ? 4 : H <= 2048 ? 2 : 1; }

// Bytes of the ring.
static size_t ln_ring(int mode, int stages, int tensors, int64_t H, int es) {
  if (mode == kLnDirect) return 0;
  if (mode == kLnVector) return (size_t)stages * tensors * kLnThreads * ln_cpt(H, mode) * es;
  return (size_t)stages * tensors * ln_rows_per_block(H) * ln_row_bytes((int)H, es);
}

// A kernel instance by mode and width.
template <typename X>
static LnFwdKernel ln_fwd_pick(int mode, int64_t H) {
  return mode == kLnVector    ? LN_PICK(ln_fwd_kernel, X, kLnVector)
         : mode == kLnShifted ? LN_PICK_SHIFTED(ln_fwd_kernel, X)
                              : LN_PICK(ln_fwd_kernel, X, kLnDirect);
}
template <typename X>
static LnBwdKernel ln_bwd_pick(int mode, int64_t H) {
  return mode == kLnVector    ? LN_PICK(ln_bwd_kernel, X, kLnVector)
         : mode == kLnShifted ? LN_PICK_SHIFTED(ln_bwd_kernel, X)
                              : LN_PICK(ln_bwd_kernel, X, kLnDirect);
}

// Row groups of the backward's partial sums.
static int ln_groups(int64_t T, int64_t H) {
  if (H > kLnMaxH) return (int)std::max<int64_t>(1, std::min<int64_t>(304, (T + 31) / 32));
  // A partial row costs about what a pass over a row does: a pass a block up to 64 blocks, two up to 256, four up to
  // what stays resident on 152 SMs (512 x 4096: 9.7 us at 256 blocks, 11.2 at 128, 10.4 at 304; 1024 x 4096: 12.4 us
  // at 256, 13.2 at 304).
  const int rows = ln_rows_per_block(H);
  const int64_t fit = (T + rows - 1) / rows;
  const int64_t most = 152 * ln_bwd_blocks(ln_cpt(H, kLnVector));  // (the same in every mode)
  return (int)std::min(most, std::max({std::min<int64_t>(fit, 64), std::min<int64_t>((fit + 1) / 2, 256), (fit + 3) / 4}));
}

// How rows are read: see LnMode.  `in`: the row tensors read, `rest`: the other tensors that vectors would touch.
static int ln_mode(int64_t H, int es, std::initializer_list<const void*> in, std::initializer_list<const void*> rest,
                   std::initializer_list<int64_t> strides) {
  const int vec = 16 / es;
  for (const void* p : in)
    if (reinterpret_cast<uintptr_t>(p) & 15) return kLnDirect;
  if (H % vec) return kLnShifted;
  for (const void* p : rest)
    if (reinterpret_cast<uintptr_t>(p) & 15) return kLnShifted;
  for (int64_t ld : strides)
    if (ld % vec) return kLnShifted;
  return kLnVector;
}

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
  for (const float* p : {mean, rstd})
    if ((rc = ln_aligned("layer_norm_fwd", p, MOE_DT_F32))) return rc;
  LnFwdArgs a{x, residual, gamma, beta, y, sum, kind == MOE_NORM_LAYER ? mean : nullptr, rstd, ldx, ldr, T, (int)H,
              kind == MOE_NORM_RMS, eps};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool b16 = x_dtype == MOE_DT_BF16;
  if (H <= kLnMaxH) {
    const int es = b16 ? 2 : 4, mode = ln_mode(H, es, {x, residual}, {y, sum, gamma, beta}, {ldx, ldr});
    const LnFwdKernel k = b16 ? ln_fwd_pick<uint16_t>(mode, H) : ln_fwd_pick<float>(mode, H);
    const int cpt = ln_cpt(H, mode), blocks = ln_fwd_blocks(cpt, es);
    const size_t smem = ln_ring(mode, ln_stages(blocks, 2, cpt, es), 2, H, es);
    const int rows = ln_rows_per_block(H);
    const int64_t grid = std::min<int64_t>((T + rows - 1) / rows, 152 * blocks);
    return launch_pdl(k, dim3((unsigned)grid), dim3(kLnThreads), smem, st, "layer_norm_fwd", a,
                      (int)(w_dtype == MOE_DT_BF16));
  }
  const int grid = (int)std::min<int64_t>(T, 65536);
  auto kern = x_dtype == MOE_DT_BF16
                  ? (w_dtype == MOE_DT_BF16 ? ln_fwd_any_kernel<uint16_t, uint16_t> : ln_fwd_any_kernel<uint16_t, float>)
                  : (w_dtype == MOE_DT_BF16 ? ln_fwd_any_kernel<float, uint16_t> : ln_fwd_any_kernel<float, float>);
  return launch_pdl(kern, dim3(grid), dim3(kLnThreads), 0, st, "layer_norm_fwd", a);
}

extern "C" size_t layer_norm_bwd_workspace_size(int64_t T, int64_t H) {
  if (T <= 0 || H <= 0 || H > INT32_MAX / 8) return 0;
  return sizeof(float) * 2 * (size_t)ln_groups(T, H) * (size_t)H;
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
  for (const float* p : {mean, rstd, static_cast<const float*>(dgamma), static_cast<const float*>(dbeta)})
    if ((rc = ln_aligned("layer_norm_bwd", p, MOE_DT_F32))) return rc;
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
              kind == MOE_NORM_RMS, ln_groups(T, H)};
  const int tiles = (int)((H + 31) / 32);
  auto weights = [&]() {
    return launch_pdl(ln_bwd_reduce_kernel, dim3(tiles, dbeta ? 2 : 1), dim3(kLnReduceThreads), 0, st,
                      "layer_norm_bwd weight gradients", static_cast<const float*>(a.part), a.G, (int)H, dgamma, dbeta,
                      accumulate);
  };
  if (H <= kLnMaxH) {
    const bool b16 = x_dtype == MOE_DT_BF16;
    const int es = b16 ? 2 : 4, mode = ln_mode(H, es, {dy, x, dres}, {dx, gamma}, {lddy, ldx, ldres});
    const LnBwdKernel k = b16 ? ln_bwd_pick<uint16_t>(mode, H) : ln_bwd_pick<float>(mode, H);
    const int cpt = ln_cpt(H, mode);
    const size_t sums = ln_rows_per_block(H) > 1 ? sizeof(float) * kLnThreads * cpt : 0;
    const size_t smem = std::max(ln_ring(mode, ln_stages(ln_bwd_blocks(cpt), 3, cpt, es), 3, H, es), sums);
    if ((rc = launch_pdl(k, dim3(a.G), dim3(kLnThreads), smem, st, "layer_norm_bwd", a, (int)(w_dtype == MOE_DT_BF16))))
      return rc;
    return weights();
  }
  const int grid = (int)std::min<int64_t>(T, 65536);
  auto kern = x_dtype == MOE_DT_BF16 ? (w_dtype == MOE_DT_BF16 ? ln_bwd_dx_any_kernel<uint16_t, uint16_t>
                                                               : ln_bwd_dx_any_kernel<uint16_t, float>)
                                     : (w_dtype == MOE_DT_BF16 ? ln_bwd_dx_any_kernel<float, uint16_t>
                                                               : ln_bwd_dx_any_kernel<float, float>);
  auto part = x_dtype == MOE_DT_BF16 ? ln_bwd_part_any_kernel<uint16_t> : ln_bwd_part_any_kernel<float>;
  if ((rc = launch_pdl(kern, dim3(grid), dim3(kLnThreads), 0, st, "layer_norm_bwd dx", a))) return rc;
  if ((rc = launch_pdl(part, dim3(tiles, a.G), dim3(kLnThreads), 0, st, "layer_norm_bwd partial sums", a))) return rc;
  return weights();
}
