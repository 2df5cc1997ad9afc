// The gated feed-forward block on few tokens: one projection with the weights as the tensor core's M operand.
//
//   kGlu   a = act(x Wg + bg) * (x Wu + bu)   (64 features a CTA: 64 gate and 64 up columns are the 128 rows of its tile)
//   else   out = a W2 + b2                    (128 columns a CTA)
//
// A tile is 128 weight columns x NT tokens (16 .. 256, zero-filled above T), read as they lie: W [K, columns] is an
// MN-major operand.  The contraction is split over a cluster of up to 8 CTAs, whose fp32 partial tiles meet in distributed
// shared memory, every output summed in rank order by one thread (bit-reproducible, no atomics, no workspace).
//
// Bound: reading the weights once from HBM.  The 256-row pair tiles of ffn_kernel.cuh would keep I / 128 pairs busy; here
// columns / 128 x split CTAs read, each with its whole share of a projection in flight at once where it fits.  The
// second projection issues its weights' copies before it waits for the first (they are older than the first one's
// own start), so that only the activations' arrival is left on its critical path.
#include <cuda.h>
#include <algorithm>
#include <type_traits>

#include "ffn_kernel.cuh"
#include "ffn.h"

namespace moebwd {
namespace {

struct SmallParams {
  CUtensorMap w0, w1, x;  // gate and up columns (interleaved, or one projection: the same map), tokens
  int T, N, nk;           // tokens, output columns (features with GLU), k-blocks of 64
  int nt, stages;         // token tile, pipeline stages
  int glu, interleaved;
  int early;              // weights may be read before the previous kernel has ended
  const uint16_t* bias;   // [2 N] with GLU, else [N]; or null
  uint16_t* out;          // [T, N]
  uint16_t* h;            // GLU: [T, 2 N] or null
  int32_t* status;
  uint64_t wait_ns;
};

constexpr int kSmallThreads = 320;  // producer, MMA issue, eight warps that empty the accumulator; all of them sum
constexpr int kSmallABytes = 128 * 128;
constexpr int kSmallMaxStages = 8;

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

template <bool GLU, int SPLIT>
__global__ void __launch_bounds__(kSmallThreads, 1) ffn_small_kernel(const __grid_constant__ SmallParams P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int stage_bytes = kSmallABytes + P.nt * 128;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem);  // barriers first: the partial tile overlays the stages behind
  uint64_t* empty = full + kSmallMaxStages;
  uint64_t* done = empty + kSmallMaxStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint8_t* stages = smem + 1024;
  float* part = reinterpret_cast<float*>(stages);  // [nt][128]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr uint32_t split = SPLIT;
  const uint32_t rank = SPLIT > 1 ? cluster_ctarank() : 0;
  const int tile = blockIdx.x / split;
  const int t0 = blockIdx.y * P.nt;
  const int kb0 = (int)((int64_t)P.nk * rank / split);
  const int nk = (int)((int64_t)P.nk * (rank + 1) / split) - kb0;
  const int tmem_cols = P.nt < 32 ? 32 : P.nt;

  if (threadIdx.x == 0) {
    for (int s = 0; s < P.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&P.w0);
    prefetch_tmap(&P.w1);
    prefetch_tmap(&P.x);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      auto load_w = [&](int s, int kb) {
        uint8_t* a = stages + s * stage_bytes;
        const int k = (kb0 + kb) * 64;
        const int c = GLU && !P.interleaved ? tile * 64 : tile * 128;
        tma_load_2d(a, &P.w0, &full[s], c, k);
        tma_load_2d(a + 8192, &P.w1, &full[s], GLU && !P.interleaved ? c : c + 64, k);
      };
      const int first = nk < P.stages ? nk : P.stages;
      if (!P.early) pdl_wait();
      for (int kb = 0; kb < first; ++kb) {
        mbar_arrive_expect_tx(&full[kb], (uint32_t)stage_bytes);
        load_w(kb, kb);
      }
      if (P.early) pdl_wait();
      pdl_trigger();
      for (int kb = 0; kb < first; ++kb)
        tma_load_2d(stages + kb * stage_bytes + kSmallABytes, &P.x, &full[kb], (kb0 + kb) * 64, t0);
      int issued = first;
      int s = 0;
      uint32_t ph = 0;
      for (int kb = first; kb < nk; ++kb) {
        if (!mbar_wait_bounded(&empty[s], ph, P.status, abort_flag, P.wait_ns)) break;
        mbar_arrive_expect_tx(&full[s], (uint32_t)stage_bytes);
        load_w(s, kb);
        tma_load_2d(stages + s * stage_bytes + kSmallABytes, &P.x, &full[s], (kb0 + kb) * 64, t0);
        ++issued;
        if (++s == P.stages) {
          s = 0;
          ph ^= 1u;
        }
      }
      // every copy lands before the partial tile overlays the stages
      for (int i = 1; i <= (issued < P.stages ? issued : P.stages); ++i) {
        const int n = issued - i;
        mbar_wait_drain(&full[n % P.stages], (uint32_t)((n / P.stages) & 1), P.status);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      pdl_wait();  // the limit of the waits below does not count the kernel in front, whose end the tokens' copies wait for
      const uint32_t idesc = idesc_bf16(128, P.nt, 1, 0);
      int s = 0;
      uint32_t ph = 0;
      for (int kb = 0; kb < nk; ++kb) {
        if (!mbar_wait_bounded(&full[s], ph, P.status, abort_flag, P.wait_ns)) break;
        tc_fence_after();
        const uint32_t a0 = smem_u32(stages + s * stage_bytes), b0 = a0 + kSmallABytes;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_bf16(tmem, mnmajor_sw128_desc(a0 + kk * 2048, 8192), kmajor_sw128_desc(b0 + kk * 32), idesc, (kb | kk) != 0);
        mma_commit(&empty[s]);
        if (++s == P.stages) {
          s = 0;
          ph ^= 1u;
        }
      }
      mma_commit(done);
      mbar_wait_drain(done, 0, P.status);
    }
  }
  pdl_wait();  // every thread: outputs (and the bias) belong to earlier work until here
  __syncthreads();  // the products are in TMEM, no copy is in flight
  tc_fence_after();
  if (warp >= 2) {  // lane quarter `warp & 3`: weight columns 32 q + lane, one token a TMEM column; two warps a quarter
    const int q = warp & 3, sub = (warp - 2) >> 2;
    const uint32_t taddr = tmem + ((uint32_t)(32 * q) << 16);
    for (int c = 16 * sub; c < P.nt; c += 32) {
      uint32_t r[16];
      tmem_ld_32x32b_x16(taddr + c, r);
      tmem_ld_wait_regs<16>(r);
#pragma unroll
      for (int j = 0; j < 16; ++j) part[(c + j) * 128 + 32 * q + lane] = __uint_as_float(r[j]);
    }
  }
  tc_fence_before();
  if (SPLIT > 1)
    cluster_sync_all();  // every CTA's partial tile is complete
  else
    __syncthreads();

  // 4 output columns of one token a thread: a warp reads whole rows of partial tiles; the cluster's CTAs take turns
  constexpr int kPieces = GLU ? 16 : 32, V = GLU ? 8 : 4;
  const int tokens = P.T - t0 < P.nt ? P.T - t0 : P.nt;
  for (int i = (int)rank * kSmallThreads + threadIdx.x; i < tokens * kPieces; i += (int)split * kSmallThreads) {
    const int tok = i / kPieces, pc = i % kPieces;
    // floats of the tile row: with GLU 8 of them (gate 4 pc .. and up 64 + 4 pc .., or interleaved 8 pc ..)
    const int o0 = GLU && P.interleaved ? 8 * pc : 4 * pc;
    const int o1 = GLU && !P.interleaved ? 64 + 4 * pc : o0 + 4;
    float v[V];
    float4 f[SPLIT][V / 4];
    const uint32_t base = smem_u32(part + tok * 128);
#pragma unroll
    for (uint32_t r = 0; r < split; ++r) {
      const uint32_t pb = SPLIT > 1 ? mapa_shared(base, r) : base;
#pragma unroll
      for (int j = 0; j < V / 4; ++j)
        f[r][j] = SPLIT > 1 ? ld_cluster_f4(pb + 4 * (j ? o1 : o0))
                            : *reinterpret_cast<const float4*>(part + tok * 128 + (j ? o1 : o0));
    }
#pragma unroll
    for (int j = 0; j < V / 4; ++j) {
      v[4 * j] = f[0][j].x;
      v[4 * j + 1] = f[0][j].y;
      v[4 * j + 2] = f[0][j].z;
      v[4 * j + 3] = f[0][j].w;
#pragma unroll
      for (uint32_t r = 1; r < split; ++r) {
        v[4 * j] += f[r][j].x;
        v[4 * j + 1] += f[r][j].y;
        v[4 * j + 2] += f[r][j].z;
        v[4 * j + 3] += f[r][j].w;
      }
    }
    const int col = tile * (GLU ? 64 : 128) + 4 * pc;
    if (col >= P.N) continue;  // N is a multiple of 8
    const int64_t row = t0 + tok;
    auto add4 = [&](float* d, const uint16_t* b) {
      const uint2 x = *reinterpret_cast<const uint2*>(b);
      d[0] += bf_lo(x.x);
      d[1] += bf_hi(x.x);
      d[2] += bf_lo(x.y);
      d[3] += bf_hi(x.y);
    };
    auto pack4 = [](const float* d) { return make_uint2(pack_bf16x2(d[0], d[1]), pack_bf16x2(d[2], d[3])); };
    if constexpr (GLU) {
      if (P.bias) {
        add4(v, P.bias + (P.interleaved ? 2 * col : col));
        add4(v + 4, P.bias + (P.interleaved ? 2 * col + 4 : P.N + col));
      }
      float a[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        a[j] = P.interleaved ? glu_value(P.glu, v[2 * j], v[2 * j + 1]) : glu_value(P.glu, v[j], v[4 + j]);
      *reinterpret_cast<uint2*>(P.out + row * P.N + col) = pack4(a);
      if (P.h) {
        uint16_t* h = P.h + row * 2 * P.N;
        *reinterpret_cast<uint2*>(h + (P.interleaved ? 2 * col : col)) = pack4(v);
        *reinterpret_cast<uint2*>(h + (P.interleaved ? 2 * col + 4 : P.N + col)) = pack4(v + 4);
      }
    } else {
      if (P.bias) add4(v, P.bias + col);
      *reinterpret_cast<uint2*>(P.out + row * P.N + col) = pack4(v);
    }
  }
  __syncwarp();
  if (SPLIT > 1)
    cluster_sync_all();  // no CTA leaves while a peer may still read its partial tile
  else
    __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, tmem_cols);
  }
}

template <bool GLU, int SPLIT>
int launch_small(const SmallParams& P, int tiles, int token_tiles, cudaStream_t st) {
  auto kern = ffn_small_kernel<GLU, SPLIT>;
  constexpr int split = SPLIT;
  const size_t smem = 2048 + std::max<size_t>((size_t)P.stages * (kSmallABytes + P.nt * 128), (size_t)P.nt * 512);
  int rc = allow_smem(reinterpret_cast<const void*>(kern), kSmemLimit);
  if (rc) return rc;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see launch_pdl
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)(tiles * split), (unsigned)token_tiles, 1);
  cfg.blockDim = dim3(kSmallThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = option(MOE_OPT_PDL) ? 2 : 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, P);
  count_launch();
  if (e != cudaSuccess) return cuda_check(e, "ffn_small launch");
  return cuda_check(cudaGetLastError(), "ffn_small launch");
}

}  // namespace

// Microseconds of one projection on this kernel, fitted on one GB300 (T 1 .. 2048, K 768 .. 4096, weights in L2) within 15%:
// launch and load latency 2.5; 0.27 a k-block, whatever the token tile (with 16 tokens the issue of copies and
// products, with 256 the tensor core); emptying the accumulator 1 per 64 tokens; meeting in the cluster 1.1, with 8 CTAs
// 1.8.  Clusters need their SMs in one GPC, so the larger ones fill fewer of the 152: 8 CTAs with more than one token
// tile's shared memory each ran in two waves from 128 CTAs on (21.7 us where 4 took 10.1), and are not offered.
SmallPlan small_plan(int64_t T, int64_t columns, int64_t K, int per_tile, int sms) {
  SmallPlan best;
  best.us = 1e30f;
  const int64_t tiles = (columns + per_tile - 1) / per_tile, nk = (K + 63) / 64;
  for (int nt = 16; nt <= 256; nt *= 2) {
    if (nt < T && nt < 128) continue;  // one token tile, or tiles of 128 or 256
    const int64_t token_tiles = (T + nt - 1) / nt;
    for (int split = 1; split <= (nt == 16 ? 8 : 4); split *= 2) {
      if (split > nk) break;
      const int64_t room = split == 1 ? sms : split == 2 ? sms - 8 : sms - 16;
      const int64_t waves = (tiles * token_tiles * split + room - 1) / room;
      const float us = (float)waves * (2.5f + 0.0156f * nt + (split == 1 ? 0.f : split == 8 ? 1.8f : 1.1f) +
                                       0.27f * (float)((nk + split - 1) / split));
      if (us < best.us) best = SmallPlan{nt, split, tiles, token_tiles, us};
    }
    if (nt >= T) break;
  }
  return best;
}

int launch_ffn_small(bool glu_kernel, const SmallPlan& pl, const FfnSmallArgs& a, cudaStream_t st) {
  alignas(64) SmallParams P{};
  // weights [K, columns]: 64 x 64 boxes; the tokens' rows [T, K]: nt x 64
  const int64_t cols = glu_kernel && !a.interleaved ? a.N : glu_kernel ? 2 * a.N : a.N;
  if (!make_tmap_2d(&P.w0, a.W, 2, (uint64_t)a.K, (uint64_t)cols, (uint64_t)a.ldw * 2, 64, 64)) return MOE_ERR_INVALID;
  if (glu_kernel && !a.interleaved) {
    if (!make_tmap_2d(&P.w1, static_cast<const uint16_t*>(a.W) + a.N, 2, (uint64_t)a.K, (uint64_t)cols, (uint64_t)a.ldw * 2, 64, 64))
      return MOE_ERR_INVALID;
  } else {
    P.w1 = P.w0;
  }
  if (!make_tmap_2d(&P.x, a.x, 2, (uint64_t)a.T, (uint64_t)a.K, (uint64_t)a.ldx * 2, (uint32_t)pl.nt, 64)) return MOE_ERR_INVALID;
  P.T = (int)a.T;
  P.N = (int)a.N;
  P.nk = (int)((a.K + 63) / 64);
  P.nt = pl.nt;
  const int per = (P.nk + pl.split - 1) / pl.split;
  const int fit = (int)((kSmemLimit - 2048) / (kSmallABytes + pl.nt * 128));
  P.stages = std::min(std::min(per, fit), kSmallMaxStages);
  P.glu = a.glu;
  P.interleaved = a.interleaved;
  P.early = a.early;
  P.bias = a.bias;
  P.out = a.out;
  P.h = a.h;
  P.status = a.status;
  P.wait_ns = (uint64_t)option(MOE_OPT_WAIT_LIMIT_NS);
  auto go = [&](auto s) {
    constexpr int S = decltype(s)::value;
    return glu_kernel ? launch_small<true, S>(P, (int)pl.tiles, (int)pl.token_tiles, st)
                      : launch_small<false, S>(P, (int)pl.tiles, (int)pl.token_tiles, st);
  };
  switch (pl.split) {
    case 1: return go(std::integral_constant<int, 1>());
    case 2: return go(std::integral_constant<int, 2>());
    case 4: return go(std::integral_constant<int, 4>());
    default: return go(std::integral_constant<int, 8>());
  }
}

}  // namespace moebwd
