// Dense GEMMs of the gated feed-forward block on CTA pairs (clusters of two, cta_group::2 tcgen05 MMA, 256 x 256 tiles):
//
//   kFfnGlu    a = act(x Wg + bg) * (x Wu + bu): both projections in one tile (128 gate and 128 up columns of the same
//              features side by side in the accumulator), activation and product in the epilogue, the pre-activations
//              stored for the backward on request
//   kFfnDGlu   da = dout W2^T in the accumulator, and in the epilogue with the saved gate and up
//              dgate = da up act'(gate), dup = da act(gate), a = act(gate) up; dgate and dup overwrite the loaded slabs in
//              shared memory, and their fp32 column sums over 32 rows go out for the bias gradient
//   kFfnStore  C (+)= A B + bias of up to three problems of different shapes in one launch: dW1, dW2 and dx depend on the
//              same kernel only, and one persistent grid that takes the longest tiles first leaves no SM idle between them
//
// Bound: tensor cores.  An operand is read either K-major ([rows, K]) or MN-major ([K, rows]) as it lies in memory, so
// no operand is ever copied or transposed.  Sizes off the tile are zero-filled and clipped by the tensor maps.
//
// Roles, as in the grouped pair kernel: warp 0 TMA producer (the leader claims tiles and publishes them to both CTAs' rings),
// warp 1 MMA issue (leader), warps 2-17 epilogue.  The epilogue's two halves (warps 2-9: columns 0-127 of the accumulator,
// warps 10-17: 128-255) have staging buffers and barriers of their own and never meet; within a half, two groups of four
// warps take alternate 32-column pieces, one row of a 32-row quarter a lane.  The epilogues are bound by dependent
// steps, not by issue: sixteen warps instead of eight, paired fp32 arithmetic and a stored from registers took kFfnDGlu with
// bias sums (16384 x 2048 x 1024) from 149 to 81 us.
// Every wait is bounded; a timeout raises MOE_STATUS_TIMEOUT and the abort flags of both CTAs.
#pragma once
#include "gemm_pair_kernel.cuh"

namespace moebwd {

enum FfnEpi { kFfnGlu = 0, kFfnDGlu = 1, kFfnStore = 2 };

struct FfnProblem {
  int end;              // tiles of this problem and those before it
  int n_tiles, nk;      // column tiles; k-blocks of 64
  int M, N;             // rows, and columns of the output (kFfnGlu, kFfnDGlu: features)
  int a_mn, b_mn;       // operand stored [K, rows]: 1 its map is 2D, 2 in groups of 64 columns (see make_tmap_groups)
  int accumulate;       // add to the output
  const uint16_t* bias; // [N] or null
};

constexpr int kFfnMaps = 9;
struct FfnParams {
  // kFfnStore: A, B, C of problem i at 3 i.  kFfnGlu: x, Wg, Wu, a, h (gate part), h (up part).
  // kFfnDGlu: dout, W2, h (gate), h (up), dh (gate), dh (up).  Interleaved columns: one matrix, the two parts the same.
  CUtensorMap map[kFfnMaps];
  FfnProblem prob[3];
  int nprob;
  int glu, interleaved, save;
  const uint16_t* b1;     // kFfnGlu: [2I] or null
  int width;              // kFfnDGlu: features of a tile that are wanted, 256, 128 or 64 (of the product's first columns)
  uint16_t* a_out;        // kFfnDGlu: a [T, I]
  float* db1_part;        // kFfnDGlu: [4 * 128-row tiles, 2I] column sums, or null
  int32_t* tile_counter;  // null: tiles in turn; else zero before the launch, dynamic claims
  int32_t* zero_counter;  // set to 0 for the next kernel
  int32_t* status;
  uint64_t wait_ns;
};

template <int EPI>
struct FfnCfg {
  static constexpr int BN = 256, BKE = 64;
  static constexpr int A_BYTES = 128 * 128, B_BYTES = 128 * 128, STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int BUF_BYTES = 128 * 128;  // a slab of 128 rows x 64 bf16 columns, 128-byte swizzle
  // staging slabs of each half: one of C; two to alternate (a, gate, up); gate and up
  static constexpr int BUFS = EPI == kFfnStore ? 1 : 2;
  static constexpr int STAGES = EPI == kFfnStore ? 6 : 5;
  static constexpr int RING = 4;
  static constexpr int EPI_WARPS = 16;
  static constexpr int THREADS = 64 + 32 * EPI_WARPS;
  static constexpr int BAR_BYTES = 512;
  static constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + 2 * BUFS * BUF_BYTES + BAR_BYTES;
  static_assert(SMEM_BYTES <= kSmemLimit, "shared memory overflow");
};

struct FfnTile {
  int p, nt, mt, nk;
  bool valid;
};

__device__ __forceinline__ FfnTile ffn_decode(const FfnParams& P, int t, int rank) {
  FfnTile ti;
  ti.p = 0;
  int first = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (i + 1 < P.nprob && t >= P.prob[i].end) {
      ti.p = i + 1;
      first = P.prob[i].end;
    }
  const FfnProblem& pr = P.prob[ti.p];
  const int l = t - first;
  const int mp = l / pr.n_tiles;
  ti.nt = l - mp * pr.n_tiles;
  ti.mt = 2 * mp + rank;
  ti.nk = pr.nk;
  ti.valid = ti.mt * 128 < pr.M;  // an odd last row tile: the partner's rows are read as zeros and not stored
  return ti;
}

// Barrier over the 256 threads of one epilogue half, and the form that ORs a predicate over them.
__device__ __forceinline__ void half_bar(int half) { asm volatile("bar.sync %0, 256;" ::"r"(1 + half) : "memory"); }
__device__ __forceinline__ bool half_bar_any(int half, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "bar.red.or.pred q, %1, 256, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(1 + half), "r"((uint32_t)pred)
      : "memory");
  return r != 0;
}

// Wait for this thread's TMEM loads; no use of r can be scheduled before it.
__device__ __forceinline__ void tmem_ld_wait_32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14])
               :
               : "memory");
  asm volatile("" : "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                    "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                    "+r"(r[29]), "+r"(r[30]), "+r"(r[31]) : : "memory");
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// sigma(g) = 1 / (1 + 2^(-g log2 e)) from the exp2 and reciprocal approximations (2 ulp each, far below bf16's step; 0
// where 2^x overflows).
__device__ __forceinline__ float ffn_sigmoid(float g) {
  float e, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + e));
  return s;
}
__device__ __forceinline__ float glu_value(int glu, float g, float u) {
  if (glu == MOE_GLU_SWIGLU) return g * ffn_sigmoid(g) * u;
  return g * (0.5f * (1.f + erff(g * 0.70710678118654752f))) * u;
}
// Two features' act(g) and act'(g), in paired fp32 arithmetic where the formula allows.
__device__ __forceinline__ void glu_terms2(int glu, uint64_t G, uint64_t& act, uint64_t& slope) {
  float g0, g1;
  if (glu == MOE_GLU_SWIGLU) {  // s = sigma(g): g s and s (1 + g (1 - s))
    float e0, e1, s0, s1;
    f2_unpack(f2_mul(G, f2_splat(-1.4426950408889634f)), g0, g1);
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(g0));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(g1));
    f2_unpack(f2_add(f2_pack(e0, e1), f2_splat(1.f)), g0, g1);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s0) : "f"(g0));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s1) : "f"(g1));
    const uint64_t S = f2_pack(s0, s1);
    act = f2_mul(G, S);
    slope = f2_mul(S, f2_fma(G, f2_fma(S, f2_splat(-1.f), f2_splat(1.f)), f2_splat(1.f)));
  } else {
    f2_unpack(G, g0, g1);
    const float c0 = 0.5f * (1.f + erff(g0 * 0.70710678118654752f)), c1 = 0.5f * (1.f + erff(g1 * 0.70710678118654752f));
    act = f2_pack(g0 * c0, g1 * c1);
    slope = f2_pack(c0 + g0 * (0.39894228040143268f * __expf(-0.5f * g0 * g0)),
                    c1 + g1 * (0.39894228040143268f * __expf(-0.5f * g1 * g1)));
  }
}

// Two fp32 values rounded to bf16, in one instruction.
__device__ __forceinline__ uint32_t to_bf16x2(float lo, float hi) {
  uint32_t w;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}
__device__ __forceinline__ uint32_t to_bf16x2(uint64_t v) {
  float lo, hi;
  f2_unpack(v, lo, hi);
  return to_bf16x2(lo, hi);
}

// Sums over the warp's 32 rows of 8 columns: lanes j, j + 8, j + 16 and j + 24 get column j's.  Three halving exchanges,
// then two whole ones: 9 shuffles.
__device__ __forceinline__ float column_sums8(float (&v)[8], int lane) {
#pragma unroll
  for (int w = 4; w >= 1; w >>= 1) {
    const bool hi = lane & w;
#pragma unroll
    for (int j = 0; j < w; ++j) {
      const float send = hi ? v[j] : v[j + w];
      const float keep = hi ? v[j + w] : v[j];
      v[j] = keep + __shfl_xor_sync(0xffffffffu, send, w);
    }
  }
  v[0] += __shfl_xor_sync(0xffffffffu, v[0], 8);
  return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 16);
}

template <int EPI>
__global__ void __launch_bounds__(FfnCfg<EPI>::THREADS, 1) ffn_pair_kernel(const __grid_constant__ FfnParams P) {
  using C = FfnCfg<EPI>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* smA = smem;
  uint8_t* smB = smA + C::STAGES * C::A_BYTES;
  uint8_t* smBuf = smB + C::STAGES * C::B_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(smBuf + 2 * C::BUFS * C::BUF_BYTES);
  uint64_t* empty = full + C::STAGES;
  uint64_t* tfull = empty + C::STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* done = tempty + 2;
  uint64_t* hfull = done + 1;  // [2] kFfnDGlu: a half's gate and up slabs have landed
  uint64_t* tile_full = hfull + 2;
  uint64_t* tile_empty = tile_full + C::RING;
  volatile int* tile_ring = reinterpret_cast<volatile int*>(tile_empty + C::RING);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(const_cast<int*>(tile_ring) + C::RING);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);  // and the stages this CTA's producer has issued

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const uint32_t peer = rank ^ 1u;
  const uint32_t peer_abort = mapa_shared(smem_u32(const_cast<int*>(abort_flag)), peer);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 2 * C::EPI_WARPS);
      mbar_init(&hfull[a], 1);
    }
    mbar_init(done, 1);
    for (int r = 0; r < C::RING; ++r) {
      mbar_init(&tile_full[r], 1);
      mbar_init(&tile_empty[r], 2 + 2 * C::EPI_WARPS);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane < kFfnMaps) prefetch_tmap(&P.map[lane]);
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // barriers of both CTAs initialised before any cross-CTA signal
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // nothing written by earlier work is read, and nothing is written, before this point
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && threadIdx.x == 0 && P.zero_counter) *P.zero_counter = 0;
  const int total = P.prob[P.nprob - 1].end;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA producer (both CTAs) ----------------
      const uint32_t lead_full = mapa_shared(smem_u32(full), 0);
      int s = 0;
      uint32_t ph = 0;
      uint32_t issued = 0;
      int rs = 0;
      uint32_t rph = 0;
      int next = blockIdx.x >> 1;
      for (;;) {
        int t;
        if (leader) {
          if (P.tile_counter) {
            t = atomicAdd(P.tile_counter, 1);
          } else {
            t = next;
            next += gridDim.x >> 1;
          }
          if (t >= total) t = -1;
          if (!pair_wait(&tile_empty[rs], rph ^ 1u, P.status, abort_flag, peer_abort, P.wait_ns)) break;
          tile_ring[rs] = t;
          st_shared_cluster_u32(mapa_shared(smem_u32(const_cast<int*>(&tile_ring[rs])), peer), (uint32_t)t);
          mbar_arrive(&tile_full[rs]);
          mbar_arrive_cluster(mapa_shared(smem_u32(&tile_full[rs]), peer));
        } else {
          if (!pair_wait<true>(&tile_full[rs], rph, P.status, abort_flag, peer_abort, P.wait_ns)) break;
          t = tile_ring[rs];
          mbar_arrive_cluster(mapa_shared(smem_u32(&tile_empty[rs]), 0));
        }
        if (++rs == C::RING) {
          rs = 0;
          rph ^= 1u;
        }
        if (t < 0) break;
        const FfnTile ti = ffn_decode(P, t, (int)rank);
        const FfnProblem& pr = P.prob[ti.p];
        // A: this CTA's 128 rows.  B: its 128 of the tile's 256 columns; for kFfnGlu with gate and up apart, the leader
        // loads the gate columns of 128 features and its partner the up columns of the same.
        const CUtensorMap* ma = &P.map[EPI == kFfnStore ? 3 * ti.p : 0];
        const CUtensorMap* mb = &P.map[EPI == kFfnStore ? 3 * ti.p + 1 : EPI == kFfnGlu ? 1 + (int)rank : 1];
        const int a_row = ti.mt * 128;
        const int b_col = EPI == kFfnGlu && !P.interleaved ? ti.nt * 128 : ti.nt * (EPI == kFfnDGlu ? P.width : 256) + 128 * (int)rank;
        const int a_mn = EPI == kFfnStore ? pr.a_mn : 0;
        const int b_mn = EPI == kFfnDGlu ? 0 : pr.b_mn;
        bool ok = true;
        for (int kb = 0; kb < ti.nk; ++kb) {
          if (!pair_wait(&empty[s], ph ^ 1u, P.status, abort_flag, peer_abort, P.wait_ns)) {
            ok = false;
            break;
          }
          if (leader) mbar_arrive_expect_tx(&full[s], 2 * C::STAGE_BYTES);
          const uint32_t fb = lead_full + (uint32_t)(s * 8);
          const int kc = kb * C::BKE;
          // [K, rows]: two tiles of 64 rows, 8 KB apart
          if (a_mn == 2) {
            tma_load_3d_pair(smA + s * C::A_BYTES, ma, fb, 0, kc, a_row / 64);
          } else if (a_mn) {
#pragma unroll
            for (int j = 0; j < 2; ++j) tma_load_2d_pair(smA + s * C::A_BYTES + j * 8192, ma, fb, a_row + 64 * j, kc);
          } else {
            tma_load_2d_pair(smA + s * C::A_BYTES, ma, fb, kc, a_row);
          }
          if (b_mn == 2) {
            tma_load_3d_pair(smB + s * C::B_BYTES, mb, fb, 0, kc, b_col / 64);
          } else if (b_mn) {
#pragma unroll
            for (int j = 0; j < 2; ++j) tma_load_2d_pair(smB + s * C::B_BYTES + j * 8192, mb, fb, b_col + 64 * j, kc);
          } else {
            tma_load_2d_pair(smB + s * C::B_BYTES, mb, fb, kc, b_col);
          }
          ++issued;
          if (++s == C::STAGES) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (!ok) break;
      }
      abort_flag[1] = (int)issued;
    }
  } else if (warp == 1) {
    if (leader && lane == 0) {
      // ---------------- pair MMA issuer (leader) ----------------
      int s = 0, acc = 0;
      uint32_t ph = 0, aph = 0;
      bool ok = true;
      int rs = 0;
      uint32_t rph = 0;
      while (ok) {
        if (!pair_wait<true>(&tile_full[rs], rph, P.status, abort_flag, peer_abort, P.wait_ns)) break;
        const int t = tile_ring[rs];
        mbar_arrive(&tile_empty[rs]);
        if (++rs == C::RING) {
          rs = 0;
          rph ^= 1u;
        }
        if (t < 0) break;
        const FfnTile ti = ffn_decode(P, t, 0);
        const bool a_mn = EPI == kFfnStore && P.prob[ti.p].a_mn;
        const bool b_mn = EPI == kFfnGlu || (EPI == kFfnStore && P.prob[ti.p].b_mn);
        const uint32_t idesc = idesc_bf16(256, C::BN, (uint32_t)a_mn, (uint32_t)b_mn);
        if (!pair_wait(&tempty[acc], aph ^ 1u, P.status, abort_flag, peer_abort, P.wait_ns)) break;
        tc_fence_after();
        const uint32_t d = tmem_base + (uint32_t)(acc * C::BN);
        for (int kb = 0; kb < ti.nk; ++kb) {
          if (!pair_wait(&full[s], ph, P.status, abort_flag, peer_abort, P.wait_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a0 = smem_u32(smA + s * C::A_BYTES);
          const uint32_t b0 = smem_u32(smB + s * C::B_BYTES);
          // K step kk: 32 bytes into each 128-byte K-major row, or two 8-row atoms of an MN-major tile
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_bf16_pair(d, a_mn ? mnmajor_sw128_desc(a0 + kk * 2048, 8192) : kmajor_sw128_desc(a0 + kk * 32),
                          b_mn ? mnmajor_sw128_desc(b0 + kk * 2048, 8192) : kmajor_sw128_desc(b0 + kk * 32), idesc,
                          (kb | kk) != 0);
          mma_commit_pair(mapa_shared(smem_u32(&empty[s]), 0));
          mma_commit_pair(mapa_shared(smem_u32(&empty[s]), 1));
          if (++s == C::STAGES) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (!ok) break;
        mma_commit_pair(mapa_shared(smem_u32(&tfull[acc]), 0));
        mma_commit_pair(mapa_shared(smem_u32(&tfull[acc]), 1));
        if (++acc == 2) {
          acc = 0;
          aph ^= 1u;
        }
      }
      mma_commit_pair(mapa_shared(smem_u32(done), 0));
      mbar_wait_drain(done, 0, P.status);
    }
  } else {
    // ---------------- epilogue warps 2..17 (both CTAs) ----------------
    const int q = warp & 3;
    const int m = 32 * q + lane;
    const int half = (warp - 2) >> 3;
    const int sub = ((warp - 2) >> 2) & 1;
    const bool elect = (warp == 2 || warp == 10) && lane == 0;
    uint8_t* buf = smBuf + half * C::BUFS * C::BUF_BYTES;
    const uint32_t row_off = (uint32_t)m * 128;
    const uint32_t sw = (uint32_t)(m & 7);
    const uint32_t lead_tempty = mapa_shared(smem_u32(tempty), 0);
    const uint32_t lead_tile_empty = mapa_shared(smem_u32(tile_empty), 0);
    int acc = 0;
    uint32_t aph = 0;
    int rs = 0;
    uint32_t rph = 0;
    uint32_t hph = 0;       // kFfnDGlu: phase of the next slab load of this half
    bool h_flying = false;  // a slab load was issued and not yet seen to land (elected thread)
    int slot = 0;           // kFfnGlu: the buffer to use next
    for (;;) {
      const bool gt = pair_wait<true>(&tile_full[rs], rph, P.status, abort_flag, peer_abort, P.wait_ns);
      const int t = gt ? tile_ring[rs] : -1;
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(lead_tile_empty + (uint32_t)(rs * 8));
      if (++rs == C::RING) {
        rs = 0;
        rph ^= 1u;
      }
      // exit decisions are taken together: the OR of the abort flag over the half at a barrier
      if (half_bar_any(half, *abort_flag != 0)) break;
      if (t < 0) break;
      const FfnTile ti = ffn_decode(P, t, (int)rank);
      const FfnProblem& pr = P.prob[ti.p];
      const int row0 = ti.mt * 128;

      // kFfnDGlu: slab sl of this half is features f(sl) .. f(sl) + 63; the first is loaded while the tile is multiplied.
      // Tiles of 128 features are one slab a half, of 64 one of the first half.
      const int half_col = EPI == kFfnDGlu && P.width < 256 ? half * 64 : half * 128, slabs = EPI == kFfnDGlu && P.width < 256 ? 1 : 2;
      const bool idle = EPI == kFfnDGlu && half * 64 >= P.width;
      auto load_h = [&](int sl) {
        const int f = ti.nt * P.width + half_col + sl * 64;
        mbar_arrive_expect_tx(&hfull[half], 2 * C::BUF_BYTES);
        const int c = P.interleaved ? 2 * f : f;
        tma_load_2d(buf, &P.map[2], &hfull[half], c, row0);
        tma_load_2d(buf + C::BUF_BYTES, &P.map[3], &hfull[half], P.interleaved ? c + 64 : c, row0);
        h_flying = true;
      };
      if constexpr (EPI == kFfnDGlu) {
        if (elect && !idle) {
          bulk_wait_read_all();
          load_h(0);
        }
      }

      pair_wait(&tfull[acc], aph, P.status, abort_flag, peer_abort, P.wait_ns);
      if (half_bar_any(half, *abort_flag != 0)) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + ((uint32_t)(32 * q) << 16) + (uint32_t)(acc * C::BN);
      auto release = [&]() {  // this warp has read the accumulator
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (leader)
            mbar_arrive(&tempty[acc]);
          else
            mbar_arrive_remote(lead_tempty + (uint32_t)(acc * 8));
        }
      };
      // 16-byte piece `chunk` (8 columns) of this thread's row in a swizzled slab
      auto piece = [&](int b, int chunk) {
        return reinterpret_cast<uint4*>(buf + b * C::BUF_BYTES + row_off + (((uint32_t)chunk ^ sw) << 4));
      };

      if constexpr (EPI == kFfnStore) {
        uint32_t pk[2][16];
#pragma unroll
        for (int sl = 0; sl < 2; ++sl) {
          uint32_t r[32];
          const int c0 = half * 128 + sl * 64 + sub * 32;
          tmem_ld_32x32b_x32(taddr + c0, r);
          tmem_ld_wait_32(r);
          if (pr.bias) {
            const int n0 = ti.nt * 256 + c0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (n0 + 8 * j >= pr.N) break;  // N is a multiple of 8
              const uint4 b = *reinterpret_cast<const uint4*>(pr.bias + n0 + 8 * j);
              const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                r[8 * j + 2 * i] = __float_as_uint(__uint_as_float(r[8 * j + 2 * i]) + bf_lo(w[i]));
                r[8 * j + 2 * i + 1] = __float_as_uint(__uint_as_float(r[8 * j + 2 * i + 1]) + bf_hi(w[i]));
              }
            }
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) pk[sl][j] = to_bf16x2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
        }
        release();
#pragma unroll
        for (int sl = 0; sl < 2; ++sl) {
          const int n0 = ti.nt * 256 + half * 128 + sl * 64;
          if (elect) bulk_wait_read_all();
          half_bar(half);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *piece(0, 4 * sub + j) = make_uint4(pk[sl][4 * j], pk[sl][4 * j + 1], pk[sl][4 * j + 2], pk[sl][4 * j + 3]);
          fence_proxy_async_smem();
          half_bar(half);
          if (elect && ti.valid && n0 < pr.N) {
            if (pr.accumulate)
              tma_reduce_add_2d(&P.map[3 * ti.p + 2], buf, n0, row0);
            else
              tma_store_2d(&P.map[3 * ti.p + 2], buf, n0, row0);
            bulk_commit();
          }
        }
      } else if constexpr (EPI == kFfnGlu) {
        // 64 features of this half, 32 of them here: pa their a; hw their gate and up (interleaved: 64 columns of h)
        uint32_t pa[16], hw[32];
        const int f0 = ti.nt * 128 + half * 64;
#pragma unroll
        for (int c = 0; c < 2; ++c) {  // 16 features at a time
          const int k = sub * 32 + c * 16;
          float g[16], u[16];
          if (P.interleaved) {
            uint32_t r[32];
            tmem_ld_32x32b_x32(taddr + half * 128 + 2 * k, r);
            tmem_ld_wait_32(r);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              g[j] = __uint_as_float(r[2 * j]);
              u[j] = __uint_as_float(r[2 * j + 1]);
            }
          } else {
            uint32_t rg[16], ru[16];
            tmem_ld_32x32b_x16(taddr + half * 64 + k, rg);
            tmem_ld_32x32b_x16(taddr + 128 + half * 64 + k, ru);
            tmem_ld_wait_regs<16>(rg);
            tmem_ld_wait_regs<16>(ru);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              g[j] = __uint_as_float(rg[j]);
              u[j] = __uint_as_float(ru[j]);
            }
          }
          if (P.b1) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int f = f0 + k + 8 * j;
              if (f >= pr.N) break;  // N = I is a multiple of 8
              const uint16_t* pg = P.interleaved ? P.b1 + 2 * f : P.b1 + f;
              const uint16_t* pu = P.interleaved ? P.b1 + 2 * f + 8 : P.b1 + pr.N + f;
              const uint4 x = *reinterpret_cast<const uint4*>(pg), y = *reinterpret_cast<const uint4*>(pu);
              const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if (P.interleaved) {  // each word is one feature's gate and up
                  g[8 * j + i] += bf_lo(w[i]);
                  u[8 * j + i] += bf_hi(w[i]);
                  g[8 * j + 4 + i] += bf_lo(w[4 + i]);
                  u[8 * j + 4 + i] += bf_hi(w[4 + i]);
                } else {
                  g[8 * j + 2 * i] += bf_lo(w[i]);
                  g[8 * j + 2 * i + 1] += bf_hi(w[i]);
                  u[8 * j + 2 * i] += bf_lo(w[4 + i]);
                  u[8 * j + 2 * i + 1] += bf_hi(w[4 + i]);
                }
              }
            }
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            pa[8 * c + j] = to_bf16x2(glu_value(P.glu, g[2 * j], u[2 * j]), glu_value(P.glu, g[2 * j + 1], u[2 * j + 1]));
            if (P.interleaved) {
              hw[16 * c + 2 * j] = to_bf16x2(g[2 * j], u[2 * j]);
              hw[16 * c + 2 * j + 1] = to_bf16x2(g[2 * j + 1], u[2 * j + 1]);
            } else {
              hw[8 * c + j] = to_bf16x2(g[2 * j], g[2 * j + 1]);
              hw[16 + 8 * c + j] = to_bf16x2(u[2 * j], u[2 * j + 1]);
            }
          }
        }
        release();
        // `fill` writes this thread's pieces of a slab, which then goes to columns `col` ..
        auto put = [&](auto fill, const CUtensorMap* map, int col, int cols) {
          if (elect) bulk_wait_read<1>();  // the slab before the last has been read: this buffer is free
          half_bar(half);
          fill();
          fence_proxy_async_smem();
          half_bar(half);
          if (elect) {
            if (ti.valid && col < cols) tma_store_2d(map, buf + slot * C::BUF_BYTES, col, row0);
            bulk_commit();
          }
          slot ^= 1;
        };
        put([&]() {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *piece(slot, 4 * sub + j) = make_uint4(pa[4 * j], pa[4 * j + 1], pa[4 * j + 2], pa[4 * j + 3]);
        }, &P.map[3], f0, pr.N);
        if (P.save) {
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            const int col = P.interleaved ? 2 * f0 + 64 * part : f0;
            put([&]() {
              if (P.interleaved) {  // a slab is one group's 32 features
                if (sub == part) {
#pragma unroll
                  for (int j = 0; j < 8; ++j)
                    *piece(slot, j) = make_uint4(hw[4 * j], hw[4 * j + 1], hw[4 * j + 2], hw[4 * j + 3]);
                }
              } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  *piece(slot, 4 * sub + j) = make_uint4(hw[16 * part + 4 * j], hw[16 * part + 4 * j + 1],
                                                         hw[16 * part + 4 * j + 2], hw[16 * part + 4 * j + 3]);
              }
            }, &P.map[4 + part], col, P.interleaved ? 2 * pr.N : pr.N);
          }
        }
      } else {
        bool gone = false;
        const bool mine = row0 + m < pr.M;
        uint16_t* a_row = P.a_out + (int64_t)(row0 + m) * pr.N;
#pragma unroll 1
        for (int sl = 0; sl < (idle ? 0 : slabs); ++sl) {
          const int f0 = ti.nt * P.width + half_col + sl * 64;
          if (sl == 1 && elect) {
            bulk_wait_read_all();
            load_h(1);
          }
          const bool landed = pair_wait(&hfull[half], hph, P.status, abort_flag, peer_abort, P.wait_ns);
          if (landed) {  // a phase that was not seen to complete stays the one to drain
            h_flying = false;
            hph ^= 1u;
          }
          if (half_bar_any(half, !landed || *abort_flag != 0)) {
            gone = true;
            break;
          }
#pragma unroll
          for (int c = 0; c < 2; ++c) {  // 16 features at a time
            const int k = sub * 32 + c * 16;
            uint32_t r[16];
            tmem_ld_32x32b_x16(taddr + half_col + sl * 64 + k, r);
            tmem_ld_wait_regs<16>(r);
            if (sl == slabs - 1 && c == 1) release();
#pragma unroll
            for (int j = 0; j < 2; ++j) {  // 8 features: 16 bytes of gate and of up, or 32 interleaved
              const int f = f0 + k + 8 * j;
              const int i0 = 2 * c + j;  // eighth of the group's 32 features
              uint4* p0 = P.interleaved ? piece(sub, 2 * i0) : piece(0, 4 * sub + i0);
              uint4* p1 = P.interleaved ? piece(sub, 2 * i0 + 1) : piece(1, 4 * sub + i0);
              const uint4 x = *p0, y = *p1;
              const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
              uint32_t wa[4], wg[4], wu[4];
              float dg[8], du[8];
#pragma unroll
              for (int i = 0; i < 4; ++i) {  // features 2 i and 2 i + 1
                const uint64_t G = P.interleaved ? f2_pack(bf_lo(w[2 * i]), bf_lo(w[2 * i + 1])) : f2_pack(bf_lo(w[i]), bf_hi(w[i]));
                const uint64_t Up = P.interleaved ? f2_pack(bf_hi(w[2 * i]), bf_hi(w[2 * i + 1]))
                                                  : f2_pack(bf_lo(w[4 + i]), bf_hi(w[4 + i]));
                uint64_t act, slope;
                glu_terms2(P.glu, G, act, slope);
                const uint64_t da = f2_pack(__uint_as_float(r[8 * j + 2 * i]), __uint_as_float(r[8 * j + 2 * i + 1]));
                wa[i] = to_bf16x2(f2_mul(act, Up));
                f2_unpack(f2_mul(f2_mul(da, Up), slope), dg[2 * i], dg[2 * i + 1]);
                f2_unpack(f2_mul(da, act), du[2 * i], du[2 * i + 1]);
                if (P.interleaved) {
                  wg[i] = to_bf16x2(dg[2 * i], du[2 * i]);
                  wu[i] = to_bf16x2(dg[2 * i + 1], du[2 * i + 1]);
                } else {
                  wg[i] = to_bf16x2(dg[2 * i], dg[2 * i + 1]);
                  wu[i] = to_bf16x2(du[2 * i], du[2 * i + 1]);
                }
              }
              if (P.interleaved) {
                *p0 = make_uint4(wg[0], wu[0], wg[1], wu[1]);
                *p1 = make_uint4(wg[2], wu[2], wg[3], wu[3]);
              } else {
                *p0 = make_uint4(wg[0], wg[1], wg[2], wg[3]);
                *p1 = make_uint4(wu[0], wu[1], wu[2], wu[3]);
              }
              // a straight from registers: a lane's 32 bytes (both j) fill a sector, and no slab is needed for it
              if (mine && f < pr.N) *reinterpret_cast<uint4*>(a_row + f) = make_uint4(wa[0], wa[1], wa[2], wa[3]);
              if (P.db1_part) {  // sums of the unrounded values over this warp's 32 rows
                const float sg = column_sums8(dg, lane), su = column_sums8(du, lane);
                if (ti.valid && f < pr.N && lane < 16) {
                  float* dst = P.db1_part + ((int64_t)ti.mt * 4 + q) * 2 * pr.N;
                  const int fl = f + (lane & 7);
                  if (lane < 8)
                    dst[P.interleaved ? 2 * fl : fl] = sg;
                  else
                    dst[P.interleaved ? 2 * fl + 1 : pr.N + fl] = su;
                }
              }
            }
          }
          fence_proxy_async_smem();
          half_bar(half);
          if (elect && ti.valid && f0 < pr.N) {
            const int c = P.interleaved ? 2 * f0 : f0;
            tma_store_2d(&P.map[4], buf, c, row0);
            if (!P.interleaved || c + 64 < 2 * pr.N)
              tma_store_2d(&P.map[5], buf + C::BUF_BYTES, P.interleaved ? c + 64 : c, row0);
            bulk_commit();
          }
        }
        if (gone) break;
        if (idle) release();
      }
      if (++acc == 2) {
        acc = 0;
        aph ^= 1u;
      }
    }
    if (elect) {
      // a slab load still flying lands before this CTA exits (its barrier completes this phase)
      if (h_flying) mbar_wait_drain(&hfull[half], hph, P.status);
      bulk_wait_all();  // stores complete before exit
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // neither CTA leaves (or frees TMEM) while its partner may still signal it
  pair_land_copies<C::STAGES>(smem_raw, (uint32_t)(reinterpret_cast<uint8_t*>(full) - smem),
                              (uint32_t)(reinterpret_cast<uint8_t*>(const_cast<int*>(abort_flag)) - smem), C::STAGE_BYTES, P.status);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

}  // namespace moebwd
