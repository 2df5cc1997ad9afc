// Dropout from a counter-based generator, with the residual add of the branch it stands in, and its gradient:
//
//   y = residual + keep(t, j) x / (1 - p),    dx = keep(t, j) dy / (1 - p)
//
// keep(t, j) is word j % 4 of Philox4x32-10 (J. K. Salmon, M. A. Moraes, R. O. Dror, D. E. Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", SC'11) on the counter (j / 4, t, offset low, offset high) under the key (seed low, seed high), compared
// with round(p 2^32).  The mask is a function of (seed, offset, row, column) alone, not of strides, types, launch or
// device, so nothing is stored: the backward computes it again.
//
// Bound: HBM.  Per 16 bytes of a tensor one or two generator calls (ten rounds of two 32 x 32 -> 64 bit products and two
// three-way exclusive ors) run beside the copies.  A warp takes ITERS x 32 16-byte pieces of a row, all their loads issued
// before the first generator call.  Rows that are not whole 16-byte pieces (odd widths) are still moved in aligned pieces:
// such a piece straddles two generator groups, and a lane takes the other's keep bits from its neighbour.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "moebwd_internal.h"
#include "mx_device.cuh"

namespace moebwd {
namespace {

struct DropArgs {
  const void *x, *r;
  void* y;
  int64_t ldx, ldr, T;
  int H, segs, iters;  // segments of a row, 32-piece steps of a segment
  uint32_t thr;
  float scale;
  uint64_t offset;
  const int64_t* offset_dev;
  uint32_t key[20];  // the rounds' keys
};

// The four words of counter (c0, c1, c2, c3); key(i): word i of the rounds' keys.  Read from the constant bank they save the
// kernel of odd rows two additions a round (fp32 16411 x 1111: 31.7 -> 28.5 us); the kernel of whole rows, which has eight
// calls under way, then takes more registers and loses warps (65536 x 4096 bf16: 267 -> 290 us), and adds them up.
template <typename Key>
__device__ __forceinline__ uint4 philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, Key key) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t p0 = (uint64_t)0xD2511F53u * c0, p1 = (uint64_t)0xCD9E8D57u * c2;
    c0 = (uint32_t)(p1 >> 32) ^ c1 ^ key(2 * i);
    c2 = (uint32_t)(p0 >> 32) ^ c3 ^ key(2 * i + 1);
    c1 = (uint32_t)p1;
    c3 = (uint32_t)p0;
  }
  return make_uint4(c0, c1, c2, c3);
}
__device__ __forceinline__ uint32_t keep_bits(const uint4& w, uint32_t thr) {
  return (uint32_t)(w.x >= thr) | (uint32_t)(w.y >= thr) << 1 | (uint32_t)(w.z >= thr) << 2 | (uint32_t)(w.w >= thr) << 3;
}

__device__ __forceinline__ float dr_ld(const float* p) { return *p; }
__device__ __forceinline__ float dr_ld(const uint16_t* p) { return bf16_bits_to_float(*p); }
__device__ __forceinline__ void dr_st(float* p, float v) { *p = v; }
__device__ __forceinline__ void dr_st(uint16_t* p, float v) { *p = float_to_bf16_bits(v); }

template <typename E>
__device__ __forceinline__ void unpack16(const uint4& v, float (&f)[16 / sizeof(E)]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(E) == 4) {
      f[i] = __uint_as_float(w[i]);
    } else {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}
template <typename E>
__device__ __forceinline__ uint4 pack16(const float (&f)[16 / sizeof(E)]) {
  if constexpr (sizeof(E) == 4)
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  else
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// E: float or uint16_t (bf16).  SAME: every row of x (and r) lies at its y row's offset within 16 bytes, so that all move in
// aligned pieces; else their elements are loaded one by one.  A warp walks `iters` steps of 32 pieces, four at a time.
template <typename E, bool RES, bool SAME>
__global__ void __launch_bounds__(256) dropout_kernel(const DropArgs a) {
  constexpr int N = 16 / sizeof(E), B = 4;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const uint64_t off = a.offset + (a.offset_dev ? (uint64_t)*a.offset_dev : 0);
  const uint32_t o0 = (uint32_t)off, o1 = (uint32_t)(off >> 32);
  const int64_t units = a.T * a.segs;
  // product and sum in one rounding, as in the kernel of whole rows: a row gives the same bits wherever it lies
  const auto value = [&](float v, float s) { return RES ? fmaf(v, a.scale, s) : v * a.scale; };
  for (int64_t unit = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); unit < units; unit += (int64_t)gridDim.x * 8) {
    const int64_t t = unit / a.segs;
    const int seg = (int)(unit - t * a.segs);
    E* y = static_cast<E*>(a.y) + t * a.H;
    const E* x = static_cast<const E*>(a.x) + t * a.ldx;
    const E* r = RES ? static_cast<const E*>(a.r) + t * a.ldr : nullptr;
    // columns in front of the first aligned piece of y
    const int shift = (int)((N - (reinterpret_cast<uintptr_t>(y) / sizeof(E)) % N) % N);
    const int first = seg * 32 * a.iters + lane;  // this lane's first piece: columns shift + N first ..
    // keep bits of columns N k .. N k + N - 1
    auto bits = [&](int k) {
      uint32_t m = 0;
#pragma unroll
      for (int g = 0; g < N / 4; ++g)
        m |= keep_bits(philox((uint32_t)(k * (N / 4) + g), (uint32_t)t, o0, o1, [&](int i) { return a.key[i]; }), a.thr) << (4 * g);
      return m;
    };
    uint32_t m = bits(first);
    if (seg == 0 && shift) {  // the row's head, element by element
      const uint32_t m0 = __shfl_sync(0xffffffffu, m, 0);
      if (lane < shift && lane < a.H) {
        dr_st(y + lane, value((m0 >> lane & 1) ? dr_ld(x + lane) : 0.f, RES ? dr_ld(r + lane) : 0.f));
      }
    }
    for (int i0 = 0; i0 < a.iters; i0 += B) {
      uint4 vx[B], vr[B];
      if constexpr (SAME) {
#pragma unroll
        for (int i = 0; i < B; ++i) {
          const int c = shift + N * (first + 32 * (i0 + i));
          if (c + N <= a.H) {
            vx[i] = *reinterpret_cast<const uint4*>(x + c);
            if constexpr (RES) vr[i] = *reinterpret_cast<const uint4*>(r + c);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < B; ++i) {
        const int k = first + 32 * (i0 + i);
        const int c = shift + N * k;
        if (i0 + i >= a.iters || c - N * lane >= a.H) break;  // the same for the whole warp
        const uint32_t next = bits(k + 32);
        uint32_t keep = m;
        if (shift) {  // a piece straddles two groups of N columns: the second one's bits are the next lane's
          const uint32_t beside = __shfl_down_sync(0xffffffffu, m, 1), over = __shfl_sync(0xffffffffu, next, 0);
          keep = (m | (lane == 31 ? over : beside) << N) >> shift;
        }
        m = next;
        if (c + N <= a.H) {
          float f[N], s[N];
          if constexpr (SAME) {
            unpack16<E>(vx[i], f);
            if constexpr (RES) unpack16<E>(vr[i], s);
          } else {
#pragma unroll
            for (int j = 0; j < N; ++j) {
              f[j] = dr_ld(x + c + j);
              if constexpr (RES) s[j] = dr_ld(r + c + j);
            }
          }
#pragma unroll
          for (int j = 0; j < N; ++j) f[j] = value((keep >> j & 1) ? f[j] : 0.f, RES ? s[j] : 0.f);  // a dropped infinity or NaN is gone
          *reinterpret_cast<uint4*>(y + c) = pack16<E>(f);
        } else {
          for (int j = 0; c + j < a.H && j < N; ++j)
            dr_st(y + c + j, value((keep >> j & 1) ? dr_ld(x + c + j) : 0.f, RES ? dr_ld(r + c + j) : 0.f));
        }
      }
    }
  }
}

// The same for rows of whole 16-byte pieces that all start on a 16-byte boundary: a piece is one or two generator groups, whose
// words select the values directly.
template <typename E, int ITERS, bool RES>
__global__ void __launch_bounds__(256) dropout_whole_kernel(const DropArgs a) {
  constexpr int N = 16 / sizeof(E);
  pdl_wait();
  pdl_trigger();
  const uint64_t off = a.offset + (a.offset_dev ? (uint64_t)*a.offset_dev : 0);
  const uint32_t k0 = a.key[0], k1 = a.key[1];
  const auto key = [=](int i) { return i & 1 ? k1 + (uint32_t)(i >> 1) * 0xBB67AE85u : k0 + (uint32_t)(i >> 1) * 0x9E3779B9u; };
  const uint32_t o0 = (uint32_t)off, o1 = (uint32_t)(off >> 32);
  const int64_t units = a.T * a.segs;
  const uint64_t scale = f2_splat(a.scale);
  for (int64_t unit = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); unit < units; unit += (int64_t)gridDim.x * 8) {
    const int64_t t = unit / a.segs;
    const int first = (int)(unit - t * a.segs) * 32 * ITERS + (threadIdx.x & 31);
    const E* x = static_cast<const E*>(a.x) + t * a.ldx;
    const E* r = RES ? static_cast<const E*>(a.r) + t * a.ldr : nullptr;
    E* y = static_cast<E*>(a.y) + t * a.H;
    uint4 vx[ITERS], vr[ITERS];
#pragma unroll
    for (int i = 0; i < ITERS; ++i) {
      const int c = N * (first + 32 * i);
      if (c < a.H) {
        vx[i] = *reinterpret_cast<const uint4*>(x + c);
        if constexpr (RES) vr[i] = *reinterpret_cast<const uint4*>(r + c);
      }
    }
#pragma unroll
    for (int i = 0; i < ITERS; ++i) {
      const int c = N * (first + 32 * i);
      if (c >= a.H) break;
      float f[N], s[N];
      unpack16<E>(vx[i], f);
      if constexpr (RES) unpack16<E>(vr[i], s);
#pragma unroll
      for (int g = 0; g < N / 4; ++g) {
        const uint4 w = philox((uint32_t)(c / 4 + g), (uint32_t)t, o0, o1, key);
        const uint32_t word[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; j += 2) {  // a dropped infinity or NaN is gone
          const uint64_t v = f2_pack(word[j] >= a.thr ? f[4 * g + j] : 0.f, word[j + 1] >= a.thr ? f[4 * g + j + 1] : 0.f);
          if constexpr (RES)
            f2_unpack(f2_fma(v, scale, f2_pack(s[4 * g + j], s[4 * g + j + 1])), f[4 * g + j], f[4 * g + j + 1]);
          else
            f2_unpack(f2_mul(v, scale), f[4 * g + j], f[4 * g + j + 1]);
        }
      }
      *reinterpret_cast<uint4*>(y + c) = pack16<E>(f);
    }
  }
}

template <typename E>
int launch(const DropArgs& a, bool same, bool whole, bool deep, int64_t blocks, cudaStream_t st) {
  auto k = whole ? (deep ? (a.r ? dropout_whole_kernel<E, 4, true> : dropout_whole_kernel<E, 4, false>)
                         : (a.r ? dropout_whole_kernel<E, 1, true> : dropout_whole_kernel<E, 1, false>))
           : a.r ? (same ? dropout_kernel<E, true, true> : dropout_kernel<E, true, false>)
                 : (same ? dropout_kernel<E, false, true> : dropout_kernel<E, false, false>);
  return launch_pdl(k, dim3((unsigned)blocks), dim3(256), 0, st, "dropout", a);
}

int dropout(const char* who, const void* x, int64_t ldx, const void* r, int64_t ldr, int dtype, int64_t T, int64_t H, double p,
            uint64_t seed, uint64_t offset, const int64_t* offset_dev, void* y, moe_stream_t stream) {
  clear_error();
  if (dtype != MOE_DT_BF16 && dtype != MOE_DT_F32) return fail(MOE_ERR_INVALID, "%s: bad dtype", who);
  if (T < 0 || H <= 0) return fail(MOE_ERR_INVALID, "%s: bad sizes", who);
  if (T > INT32_MAX || H > (1 << 28)) return fail(MOE_ERR_UNSUPPORTED, "%s: too large", who);
  if (!(p >= 0.0 && p < 1.0)) return fail(MOE_ERR_INVALID, "%s: p must be in [0, 1)", who);
  if (reinterpret_cast<uintptr_t>(offset_dev) & 7) return fail(MOE_ERR_INVALID, "%s: offset must be 8-byte aligned", who);
  if (T == 0) return MOE_OK;
  if (!x || !y) return fail(MOE_ERR_INVALID, "%s: null pointer", who);
  if ((ldx < H && T > 1) || (r && ldr < H && T > 1)) return fail(MOE_ERR_INVALID, "%s: row stride below H", who);
  const int es = dtype == MOE_DT_F32 ? 4 : 2;
  const uintptr_t ax = reinterpret_cast<uintptr_t>(x), ar = reinterpret_cast<uintptr_t>(r), ay = reinterpret_cast<uintptr_t>(y);
  if ((ax | ar | ay) % es) return fail(MOE_ERR_INVALID, "%s: tensors must be aligned to their element", who);
  const int n = 16 / es;
  auto beside = [&](uintptr_t p0, int64_t ld) { return (p0 - ay) % 16 == 0 && (T == 1 || (ld - H) % n == 0); };
  const bool same = beside(ax, ldx) && (!r || beside(ar, ldr));
  const bool whole = same && ay % 16 == 0 && H % n == 0;
  DropArgs a{};
  a.x = x; a.r = r; a.y = y; a.ldx = ldx; a.ldr = ldr; a.T = T; a.H = (int)H;
  a.thr = (uint32_t)std::min(4294967295.0, std::floor(p * 4294967296.0 + 0.5));
  a.scale = (float)(1.0 / (1.0 - p));
  a.offset = offset; a.offset_dev = offset_dev;
  for (uint32_t i = 0; i < 10; ++i) {
    a.key[2 * i] = (uint32_t)seed + i * 0x9E3779B9u;
    a.key[2 * i + 1] = (uint32_t)(seed >> 32) + i * 0xBB67AE85u;
  }
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // Whole rows: four pieces a lane where that still gives every SM its warps, else one (7 x 2048 bf16: more lanes at
  // work).  Rows off the 16-byte boundary: segments as long as that allows, since each begins with a step of the generator more
  // (fp32 16411 x 1111: 32 us with whole rows, 34 with segments of four steps).
  const int sms = device_sm_count();
  const int64_t steps = ((H + n - 1) / n + 31) / 32, want = (int64_t)sms * 32;
  const bool deep = T * ((steps + 3) / 4) >= want;
  const int64_t most = std::min(steps, (want + T - 1) / T);
  a.iters = whole ? (deep ? 4 : 1) : (int)((steps + most - 1) / most);
  a.segs = (int)((steps + a.iters - 1) / a.iters);
  const int64_t blocks = std::min<int64_t>((T * a.segs + 7) / 8, 1 << 30);
  return dtype == MOE_DT_F32 ? launch<float>(a, same, whole, deep, blocks, st) : launch<uint16_t>(a, same, whole, deep, blocks, st);
}

}  // namespace
}  // namespace moebwd

extern "C" int dropout_fwd(const void* x, int64_t ldx, const void* residual, int64_t ldr, int dtype, int64_t T, int64_t H,
                           double p, uint64_t seed, uint64_t offset, const int64_t* offset_dev, void* y, moe_stream_t stream) {
  return moebwd::dropout("dropout_fwd", x, ldx, residual, ldr, dtype, T, H, p, seed, offset, offset_dev, y, stream);
}

extern "C" int dropout_bwd(const void* dy, int64_t lddy, int dtype, int64_t T, int64_t H, double p, uint64_t seed,
                           uint64_t offset, const int64_t* offset_dev, void* dx, moe_stream_t stream) {
  return moebwd::dropout("dropout_bwd", dy, lddy, nullptr, 0, dtype, T, H, p, seed, offset, offset_dev, dx, stream);
}
