// Low-rank adapters of many requests beside a shared projection, forward and backward.  Token t belongs to adapter a(t) or to
// none; A_a [r, H] and B_a [r, N] hold r rows each, contiguous along the features:
//
//   u_t = A_a x_t,  y_t = base_t + c_a B_a^T u_t
//   v_t = c_a B_a dy_t,  dx_t = base_t + A_a^T v_t,  dA_a = sum_t v_t x_t^T,  dB_a = sum_t (c_a u_t) dy_t^T
//
// With both matrices stored as r feature rows, the forward and the backward are the same two kernels: adapter_shrink
// contracts a token's features with r rows, adapter_expand adds r rows weighted by r numbers onto a token's row.
// adapter_grad is the third; its partial sums are joined by the expand kernel, which the backward runs last.  Tokens are taken in
// route_meta's order (expert_offsets, x_gather_idx with K = 1), so that the tokens of a tile share its adapter's matrices;
// tiles never mix adapters.
//
// Bound: HBM (2 r operations a byte; 16384 x 4096 at rank 16: shrink 26 us, 5.2 TB/s, expand 47, 5.7 TB/s).  The products run
// on the tensor core, one thread issuing them, so that the warps have nothing to do but copies and sums. Operands are
// gathered by token index with 16-byte asynchronous copies, which write the swizzled operand layouts directly and fill rows
// that are not there with zeros.  The r numbers of a token are summed in fp32; as operands of the next products they are two
// bf16 numbers each, the truncated value and what that leaves, together off by at most 2^-16.  Rounded to one they made
// gradients of adapters with few rows err by nearly twice their own rounding; two cost nothing up to rank 32 and 4% at rank
// 64 (backward of 16384 x (4096 + 4096): 149 us, 142 with one).  u stays fp32.
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "gemm_kernel.cuh"

namespace moebwd {
namespace {

constexpr int kThreads = 256;  // eight warps
constexpr int kMaxPer = 2048;  // rows of a gradient range at most

struct Groups {
  const int32_t* off;  // [n + 1]
  const int32_t* idx;  // [T] grouped row -> token
  int n, T;
};

__device__ __forceinline__ int clamp_row(int v, int T) { return v < 0 ? 0 : v > T ? T : v; }

struct Tile {
  int a, r0, rows;  // adapter, first grouped row, rows
};

// Tiles of ROWS rows before each adapter's, first[0 .. n]; the number of all is returned, at most T / ROWS + min(n, T): wrong
// offsets may name more.  All 256 threads call it.
template <int ROWS>
__device__ __forceinline__ int tile_table(const Groups& g, int* first, int* warp_sum) {
  const int tid = threadIdx.x, lane = tid & 31, each = (g.n + kThreads - 1) / kThreads, a0 = tid * each;
  int mine = 0;
  for (int i = a0; i < a0 + each && i < g.n; ++i) {
    const int c = clamp_row(g.off[i + 1], g.T) - clamp_row(g.off[i], g.T);
    first[i] = mine;
    mine += c > 0 ? (c + ROWS - 1) / ROWS : 0;
  }
  int sum = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, sum, o);
    if (lane >= o) sum += y;
  }
  if (lane == 31) warp_sum[tid >> 5] = sum;
  __syncthreads();
  int before = sum - mine, all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < (tid >> 5)) before += warp_sum[w];
    all += warp_sum[w];
  }
  for (int i = a0; i < a0 + each && i < g.n; ++i) first[i] += before;
  if (tid == 0) first[g.n] = all;
  __syncthreads();
  const int most = g.T / ROWS + (g.n < g.T ? g.n : g.T);
  return all < most ? all : most;
}
// A tile by its number.
template <int ROWS>
__device__ __forceinline__ Tile tile_of(const Groups& g, const int* first, int number) {
  int a = 0;  // the last adapter whose first tile is at or before this one
  for (int hi = g.n; hi - a > 1;) {
    const int mid = (a + hi) >> 1;
    if (first[mid] <= number) a = mid; else hi = mid;
  }
  const int64_t r0 = clamp_row(g.off[a], g.T) + (int64_t)(number - first[a]) * ROWS;
  const int left = (int)(clamp_row(g.off[a + 1], g.T) - r0);
  return Tile{a, (int)r0, left < ROWS ? left : ROWS};
}


// Token of a grouped row, -1 where the metadata names none.
__device__ __forceinline__ int token_of(const Groups& g, int row) {
  const int t = g.idx[row];
  return t >= 0 && t < g.T ? t : -1;
}

__device__ __forceinline__ void ld_shared_v4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
// Byte of 16-byte piece `c` of row `row` in a tile of PITCH-byte rows (PITCH >= 128): eight rows at one piece fall into
// eight bank groups.  Moving from piece c to c ^ d is an exclusive or of the byte with d << 4.
template <int PITCH>
__device__ __forceinline__ uint32_t at(int row, int c) {
  return (uint32_t)(row * PITCH + ((c ^ (row & 7)) << 4));
}
struct Waits {
  int32_t* status;
  uint64_t ns;
};

// The stages of a kernel whose threads copy operands with cp.async and one of which issues the products: a barrier a stage that
// its products arrive on, and the accumulator's TMEM.  All threads call the members; the issuing one commits in between.
// A wait that runs out is reported in the caller's status word, and every thread leaves the loop at its next barrier.
template <int STAGES>
struct PipeShared {
  uint64_t done[STAGES];
  uint32_t slot;
  int abort_flag;
};
template <int STAGES>
struct Pipe {
  PipeShared<STAGES>& sh;
  uint32_t at = 0, free = 0, parity = 0;  // stage in work, stage to refill; bit s: parity of stage s's next completion
  bool begun = false, fail = false;
  __device__ explicit Pipe(PipeShared<STAGES>& s) : sh(s) {}
  __device__ __forceinline__ uint32_t start(uint32_t cols) {
    if (threadIdx.x == 0) {
#pragma unroll
      for (int s = 0; s < STAGES; ++s) mbar_init(&sh.done[s], 1);
      sh.abort_flag = 0;
      fence_mbar_init();
    }
    if (threadIdx.x >> 5 == 1) {
      tmem_alloc(&sh.slot, cols);
      tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    return sh.slot;
  }
  __device__ __forceinline__ void commit() { mma_commit(&sh.done[at]); }
  __device__ __forceinline__ void wait(uint32_t s, const Waits& w) {
    if (!mbar_wait_bounded(&sh.done[s], (parity >> s) & 1u, w.status, &sh.abort_flag, w.ns)) fail = true;
  }
  // Waits for the products of the stage before the one just committed, which `free` then names.
  __device__ __forceinline__ void advance(const Waits& w) {
    free = at == 0 ? STAGES - 1 : at - 1;
    if (begun) {
      wait(free, w);
      parity ^= 1u << free;
    }
    begun = true;
    at = at == STAGES - 1 ? 0 : at + 1;
  }
  // Waits for all products committed.
  __device__ __forceinline__ void settle(const Waits& w) {
    const uint32_t last = at == 0 ? STAGES - 1 : at - 1;
    wait(last, w);
    if (fail) mbar_wait_drain(&sh.done[last], (parity >> last) & 1u, w.status);
  }
  // Behind a barrier after the last use of the TMEM.
  __device__ __forceinline__ void end(uint32_t tmem, uint32_t cols) {
    if (threadIdx.x >> 5 == 1) {
      tc_fence_after();
      tmem_dealloc(tmem, cols);
    }
  }
};

__device__ __forceinline__ float4 ld_peer_f4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

// ------------------------------------------------------------------------------------------
// shrink: w_t = W_a x_t, and from it v = c_a w (bf16, by grouped row), u = w (fp32, by token), su = c_a u_in (bf16)
// ------------------------------------------------------------------------------------------
struct ShrinkArgs {
  Groups g;
  const uint16_t* x;   // [T, K], row stride ld
  const uint16_t* W;   // [n, R, K]
  const float* scale;  // [n] or null
  uint16_t* v;         // [T, 2 RP]: truncated values, then what that leaves
  float* u;            // [T, R] or null
  const float* u_in;   // [T, R] with su [T, 2 RP], or null
  uint16_t* su;
  int64_t ld;
  int K, R;
  Waits w;
};

// A tile of tokens by all r rows, its contraction split over a cluster whose partial tiles meet in distributed shared memory,
// summed in rank order.  Stages of 64 features: asynchronous copies gather the tokens' 128-byte rows into the swizzled
// K-major layout (128 features and 64 tokens at ranks up to 32), one thread issues the tile's products, the accumulator stays
// in TMEM.  The form whose warps multiplied from registers spent its time on operand loads and their latency (rank 64, 16384
// x 4096: 38 us, now 33).  CTAs of a cluster take every SPLIT-th stage, not a contiguous part: they read a row's neighbouring
// pieces together (30 us instead of 32 at rank 16).  A thread copies the same four rows' pieces in every stage, so that a
// copy costs two additions beside it.
template <int RP>
struct ShrinkCfg {
  static constexpr int ROWS = RP <= 32 ? 64 : 128, KC = RP <= 32 ? 128 : 64, PIECES = KC / 8;
  static constexpr int X = ROWS * KC * 2, STAGE = X + RP * KC * 2;
  static constexpr int STAGES = RP <= 16 ? 5 : RP <= 64 ? 4 : 3;
  // Accumulators that the stages take turns with: the tensor core truncates its running sums, which shows in u (K 4096 at
  // rank 16: off by 4.4e-6 of its norm with one, 4.8e-7 with eight).
  static constexpr int ACCS = RP <= 32 ? 8 : 256 / RP, TMEM = ACCS * RP;
  static constexpr int PITCH = RP + 4;  // floats of a partial row: 16-byte pieces of 8 rows in 8 bank groups
  // a product reads 128 rows: with 64 the others are whatever lies behind them, and reach sums that nobody reads
  static constexpr int NEED = 1024 + STAGES * STAGE + (128 - ROWS) * 128;
  // Two CTAs may hold all of an SM's TMEM: their shared memory leaves no room for a CTA of another stream's cluster, which would
  // wait for TMEM while this cluster's other CTAs wait for its partners'.
  static constexpr int SMEM = TMEM > 128 && NEED < 108 * 1024 ? 108 * 1024 : NEED;
  static_assert(ROWS * PITCH * 4 <= STAGES * STAGE, "the partial tile overlays the stages");
};

// Four numbers as two bf16 each: truncated at p, what that leaves (rounded, at least 2^-133, bf16's smallest) RP further, together
// off by at most 2^-16 of the number or 2^-133.  Both have its sign and neither is 0 where the number reaches 2^-133: what they
// are multiplied with may be infinite, and as a rounded part and a rest of 0 or the other sign they made NaN of that infinity.
template <int RP>
__device__ __forceinline__ void store_split(uint16_t* p, const float (&y)[4]) {
  uint32_t hi[2], lo[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float rest[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float v = y[2 * i + j], h = __uint_as_float(__float_as_uint(v) & 0xFFFF0000u);
      rest[j] = v == 0.f ? 0.f : copysignf(fmaxf(fabsf(v - h), __uint_as_float(0x00010000u)), v);  // inf: NaN is not the maximum
    }
    hi[i] = __byte_perm(__float_as_uint(y[2 * i]), __float_as_uint(y[2 * i + 1]), 0x7632);
    lo[i] = pack_bf16x2(rest[0], rest[1]);
  }
  *reinterpret_cast<uint2*>(p) = make_uint2(hi[0], hi[1]);
  *reinterpret_cast<uint2*>(p + RP) = make_uint2(lo[0], lo[1]);
}

template <int RP, int SPLIT>
__global__ void __launch_bounds__(kThreads, 2) adapter_shrink_kernel(const ShrinkArgs p) {
  using C = ShrinkCfg<RP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ int tok[C::ROWS];
  __shared__ PipeShared<C::STAGES> pipe_shared;
  Pipe<C::STAGES> pipe(pipe_shared);
  const uint32_t tmem = pipe.start(C::TMEM);
  pdl_wait();
  pdl_trigger();  // after the allocation: the next kernel cannot take the TMEM that this one is still to get
  const uint32_t rank = SPLIT > 1 ? cluster_ctarank() : 0;
  // the table lies where the first stage will; the whole cluster works on one tile, so that all of it leaves here or none
  __shared__ int warp_sum[kThreads / 32];
  int* first = reinterpret_cast<int*>(smem);
  static_assert(C::STAGE >= (kMaxExperts + 1) * 4, "the table fits a stage");
  if ((int)blockIdx.x / SPLIT >= tile_table<C::ROWS>(p.g, first, warp_sum)) {
    pipe.end(tmem, C::TMEM);
    return;
  }
  const Tile t = tile_of<C::ROWS>(p.g, first, blockIdx.x / SPLIT);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid < C::ROWS) tok[tid] = tid < t.rows ? token_of(p.g, t.r0 + tid) : -1;
  __syncthreads();
  const int chunks = (p.K + C::KC - 1) / C::KC;
  const int mine = (chunks - (int)rank + SPLIT - 1) / SPLIT;  // chunks rank, rank + SPLIT, ...
  const uint32_t base = smem_u32(smem);
  const int pc = tid % C::PIECES, r0 = tid / C::PIECES;
  constexpr int STEP = kThreads / C::PIECES, XN = C::ROWS / STEP;  // rows of one pass of copies, passes over x's
  constexpr int WN = (RP + STEP - 1) / STEP;        // passes over W's rows
  const uint16_t* xs[XN];
  uint32_t xb[XN], xd[XN];
#pragma unroll
  for (int i = 0; i < XN; ++i) {
    const int row = r0 + STEP * i, tk = tok[row];
    xs[i] = p.x + (int64_t)(tk < 0 ? 0 : tk) * p.ld + 8 * pc + (int64_t)rank * C::KC;
    xb[i] = tk < 0 ? 0u : 16u;
    // other rows only reach their own sums, which nobody reads
    xd[i] = row < t.rows ? base + (pc >> 3) * C::ROWS * 128 + at<128>(row, pc & 7) : 0u;
  }
  const uint16_t* wsrc = p.W + ((int64_t)t.a * p.R + r0) * p.K + 8 * pc + (int64_t)rank * C::KC;
  auto load = [&](int c, uint32_t st) {
    const int64_t o = (int64_t)c * (C::KC * SPLIT);
    const uint32_t in = (int)rank * C::KC + o + 8 * pc < p.K ? 16u : 0u;  // K is a multiple of 8
#pragma unroll
    for (int i = 0; i < XN; ++i)
      if (xd[i]) cp_async_16_zfill(xd[i] + st, in ? xs[i] + o : p.x, xb[i] & in);
#pragma unroll
    for (int i = 0; i < WN; ++i) {
      const int row = r0 + STEP * i;
      if (RP % STEP == 0 || row < RP) {
        const bool ok = row < p.R && in;
        cp_async_16_zfill(base + st + C::X + (pc >> 3) * RP * 128 + at<128>(row, pc & 7),
                          ok ? wsrc + (int64_t)STEP * i * p.K + o : p.W, ok ? 16u : 0u);
      }
    }
  };
#pragma unroll
  for (int i = 0; i < C::STAGES - 1; ++i) {
    if (i < mine) load(i, i * C::STAGE);
    cp_async_commit();
  }
  constexpr uint32_t idesc = idesc_bf16(128, RP);
  for (int c = 0; c < mine; ++c) {
    cp_async_wait<C::STAGES - 2>();
    fence_proxy_async_smem();
    if (__syncthreads_or(pipe.fail)) break;  // stage c has landed for everyone
    if (tid == 0) {
      tc_fence_after();
      const uint32_t a0 = base + pipe.at * C::STAGE;
#pragma unroll
      for (int kk = 0; kk < C::KC / 16; ++kk)
        mma_bf16(tmem + (uint32_t)(c % C::ACCS) * RP, kmajor_sw128_desc(a0 + (kk >> 2) * C::ROWS * 128 + (kk & 3) * 32),
                 kmajor_sw128_desc(a0 + C::X + (kk >> 2) * RP * 128 + (kk & 3) * 32), idesc, (c >= C::ACCS || kk > 0) ? 1u : 0u);
      pipe.commit();
    }
    pipe.advance(p.w);  // the products of the step before are done with the stage refilled now
    if (c + C::STAGES - 1 < mine) load(c + C::STAGES - 1, pipe.free * C::STAGE);
    cp_async_commit();
  }
  cp_async_wait<0>();
  if (pipe.begun) pipe.settle(p.w);
  __syncthreads();  // the partial tiles overlay the stages
  tc_fence_after();
  float* part = reinterpret_cast<float*>(smem);  // [rows][PITCH]
  for (int c = 16 * (warp >> 2); c < RP && 32 * (warp & 3) < C::ROWS; c += 32) {
    float f[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) f[j] = 0.f;
    for (int i = 0; i < C::ACCS && i < mine; ++i) {
      uint32_t r[16];
      tmem_ld_32x32b_x16(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + i * RP + c, r);
      tmem_ld_wait_regs<16>(r);
#pragma unroll
      for (int j = 0; j < 16; ++j) f[j] += __uint_as_float(r[j]);
    }
    float* out = part + (32 * (warp & 3) + lane) * C::PITCH + c;
#pragma unroll
    for (int j = 0; j < 16; j += 4) *reinterpret_cast<float4*>(out + j) = make_float4(f[j], f[j + 1], f[j + 2], f[j + 3]);
  }
  tc_fence_before();
  if (SPLIT > 1)
    cluster_sync_all();
  else
    __syncthreads();
  pipe.end(tmem, C::TMEM);
  const float scale = p.scale ? p.scale[t.a] : 1.f;
  for (int i = (int)rank * kThreads + tid; i < t.rows * (RP / 4); i += SPLIT * kThreads) {
    const int row = i / (RP / 4), c = 4 * (i % (RP / 4));
    float4 f[SPLIT];
    const float* q = part + row * C::PITCH + c;
#pragma unroll
    for (int k = 0; k < SPLIT; ++k)
      f[k] = SPLIT > 1 ? ld_peer_f4(mapa_shared(smem_u32(q), (uint32_t)k)) : *reinterpret_cast<const float4*>(q);
    float4 s = f[0];
#pragma unroll
    for (int k = 1; k < SPLIT; ++k) {
      s.x += f[k].x;
      s.y += f[k].y;
      s.z += f[k].z;
      s.w += f[k].w;
    }
    const int tk = tok[row];
    const int64_t o = (int64_t)(t.r0 + row) * 2 * RP + c;
    const float w[4] = {s.x, s.y, s.z, s.w};
    float y[4];  // ranks behind r are zeros whatever x holds (0 times infinity)
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = c + j < p.R ? w[j] * scale : 0.f;
    store_split<RP>(p.v + o, y);
    if (p.u && tk >= 0)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c + j < p.R) p.u[(int64_t)tk * p.R + c + j] = w[j];
    if (p.su) {
      float z[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) z[j] = tk >= 0 && c + j < p.R ? p.u_in[(int64_t)tk * p.R + c + j] * scale : 0.f;
      store_split<RP>(p.su + o, z);
    }
  }
  __syncwarp();
  if (SPLIT > 1) cluster_sync_all();  // no CTA leaves while a peer may still read its partial tile
}

// ------------------------------------------------------------------------------------------
// the gradient's arguments, partial sums
// ------------------------------------------------------------------------------------------
struct GradProblem {
  const uint16_t* x;  // [T, K], row stride ld
  const uint16_t* v;  // [T, 2 RP] by grouped row
  uint16_t* dW;       // [n, R, K]
  float* part;        // [2 ranges, R, K]
  int64_t ld;
  int K, blocks;      // blocks of 256 features
};
struct GradArgs {
  Groups g;
  GradProblem pr[2];
  int R, ranges, accumulate;
  Waits w;
};

// The grouped rows are cut into `ranges` parts of equal cost: a row counts one and an adapter, whose sums have to be written,
// as many as kSegment rows.  (Parts of equal rows left the last one, with the many adapters of few rows, to work alone: the
// backward of 16384 rows of 1024 adapters of rank 16, 692 us, now 432; 2048 rows of 64 of rank 64, 123 us, now 94.)  Row r of
// adapter a lies at off[a] + kSegment a + (r - off[a]), and a part is `per` of these places. An adapter whose rows lie in one
// part is summed there; of any other each part holds a partial sum: at place 2 part + 1 for the one that has the adapter's
// first row (the part's last adapter), at 2 part for the others (the part's first), so that no two share one.
constexpr int kSegment = 32;  // 64 and 128 measured the same
__device__ __forceinline__ int rows_of_range(const Groups& g, int ranges, int& rows) {
  rows = clamp_row(g.off[g.n], g.T);
  const int per = (rows + kSegment * g.n + ranges - 1) / ranges;
  return per > 32 ? per : 32;
}
// The first row at or behind a place.  All threads call it.
__device__ __forceinline__ int row_at(const Groups& g, int64_t place, int rows) {
  int before = 0;  // adapters that begin at or before it
  for (int i0 = 0; i0 < g.n; i0 += (int)blockDim.x) {
    const int i = i0 + (int)threadIdx.x;
    before += __syncthreads_count(i < g.n && clamp_row(g.off[i < g.n ? i : 0], g.T) + (int64_t)kSegment * i <= place);
  }
  if (before == 0) return 0;
  const int o0 = clamp_row(g.off[before - 1], rows), o1 = clamp_row(g.off[before], rows);
  const int64_t r = o0 + (place - o0 - (int64_t)kSegment * (before - 1));
  return r < o0 ? o0 : r > o1 ? (o1 > o0 ? o1 : o0) : (int)r;
}

// Sums of the partial tiles of the adapters whose rows lie in several ranges, in order; zeros for those without rows.  The CTAs of
// the expand kernel, which runs behind the gradient's, share it out in pieces of 4096 numbers (as a kernel of its own it took
// 7 us more, 16384 x (4096 + 4096) at rank 64: 25 MB, but a launch and a start of its own).
__device__ __forceinline__ void sum_partials(const GradArgs& p, int64_t me, int64_t all) {
  int rows;
  const int per = rows_of_range(p.g, p.ranges, rows);
  const int64_t size0 = (int64_t)p.R * p.pr[0].K, size1 = (int64_t)p.R * p.pr[1].K;
  const int b0 = (int)((size0 + 4095) / 4096), each = b0 + (int)((size1 + 4095) / 4096);
  for (int64_t b = me; b < (int64_t)each * p.g.n; b += all) {
    const int a = (int)(b / each), piece = (int)(b - (int64_t)a * each);
    const int o0 = clamp_row(p.g.off[a], rows), o1 = clamp_row(p.g.off[a + 1], rows);
    const bool none = o1 <= o0;
    const int at_a = kSegment * a, s0 = (o0 + at_a) / per, s1 = none ? s0 : (o1 - 1 + at_a) / per;
    if (none ? p.accumulate != 0 : s0 == s1) continue;
    const GradProblem& q = p.pr[piece < b0 ? 0 : 1];
    const int64_t size = piece < b0 ? size0 : size1, i0 = (int64_t)(piece < b0 ? piece : piece - b0) * 4096 + 4 * threadIdx.x;
    uint16_t* dW = q.dW + a * size;
    float4 s[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = none ? s1 + 1 : s0; k <= s1; ++k) {
      const float* src = q.part + (2 * (int64_t)k + (k == s0)) * size;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t i = i0 + 1024 * j;  // K is a multiple of 8
        const float4 f = i < size ? *reinterpret_cast<const float4*>(src + i) : make_float4(0.f, 0.f, 0.f, 0.f);
        s[j].x += f.x;
        s[j].y += f.y;
        s[j].z += f.z;
        s[j].w += f.w;
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t i = i0 + 1024 * j;
      if (i >= size) continue;
      uint2* d = reinterpret_cast<uint2*>(dW + i);
      if (p.accumulate) {
        const uint2 w = *d;
        s[j].x += __uint_as_float(w.x << 16);
        s[j].y += __uint_as_float(w.x & 0xFFFF0000u);
        s[j].z += __uint_as_float(w.y << 16);
        s[j].w += __uint_as_float(w.y & 0xFFFF0000u);
      }
      *d = make_uint2(pack_bf16x2(s[j].x, s[j].y), pack_bf16x2(s[j].z, s[j].w));
    }
  }
}

// ------------------------------------------------------------------------------------------
// expand: out[token] = base[token] + v W_a
// ------------------------------------------------------------------------------------------
struct ExpandArgs {
  Groups g;
  const uint16_t* v;     // [T, 2 RP] by grouped row
  const uint16_t* W;     // [n, R, N]
  const uint16_t* base;  // [T, N], row stride ldb, or null
  uint16_t* out;         // [T, N] dense
  const int32_t* back;   // [T] token -> grouped row, negative: none
  float* u;              // [T, R] zeros for tokens without an adapter, or null
  int64_t ldb;
  int N, R, col_blocks;
  Waits w;
  GradArgs sums;  // with ranges: partial sums to join
};
constexpr int kExpandRows = 128;  // of a tile (64, which evens out short batches, leaves warps idle: 4096 x 4096, rank 16, 22 us instead of 17)

template <int RP>
struct ExpandCfg {
  static constexpr int DEPTH = RP == 64 ? 2 : 3;  // 16 tokens x 64 columns of base of a warp on their way, 2 KB each (2: two CTAs fit)
  static constexpr int V = 16384 * (RP <= 32 ? 1 : RP / 32), W = RP * 256;
  static constexpr int SMEM = 1024 + V + 2 * W + 8 * DEPTH * 2048;
};

// One wave of CTAs shares out the pieces of work (a tile of up to 128 tokens x 128 columns, a tile's pieces one behind
// another) in equal, contiguous parts.  (A CTA a piece, 7 waves of them, started anew each time: the forward at 16384 x 4096,
// rank 16, took 118 us, with equal parts 102.)  The product of the next piece runs on the tensor core, tokens x columns into
// one half of the TMEM, while the warps add this one's to the base: the tile's v stays in shared memory (K-major), W's
// columns come in two buffers (MN-major), and every warp has a few pieces of base on their way.  (Products from registers
// took their time beside the memory's: rank 64 62 us, now 53.)  The columns of W are permuted within 32 on their way to
// shared memory so that the four 8-column tiles of a TMEM load give a thread 8 neighbouring columns: base and out move in
// 16-byte pieces, four lanes to 64 bytes of a row.
// What the kernel reads before pdl_wait, and the rows without an adapter that it writes there, belong to the caller: whatever
// wrote or read them is complete before the kernel in front lets this one start (and that kernel leaves them alone).
template <int RP>
__global__ void __launch_bounds__(kThreads, RP <= 64 ? 2 : 1) adapter_expand_kernel(const ExpandArgs p) {
  using C = ExpandCfg<RP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ int tok[kExpandRows], first[kMaxExperts + 1], warp_sum[kThreads / 32];
  __shared__ PipeShared<2> sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t me = blockIdx.x, all = gridDim.x;
  Pipe<2> pipe(sh);
  const uint32_t tmem = pipe.start(2 * 128);
  // rows without an adapter keep their base
  const int t1 = (int)(p.g.T * (me + 1) / all);
  for (int t0 = (int)(p.g.T * me / all) + 32 * warp; t0 < t1; t0 += kThreads) {
    const bool mine = t0 + lane < t1 && p.back[t0 + lane] < 0;
    for (uint32_t left = __ballot_sync(0xFFFFFFFFu, mine); left; left &= left - 1) {
      const int64_t t = t0 + __ffs(left) - 1;
      if (p.u)
        for (int c = lane; c < p.R; c += 32) p.u[t * p.R + c] = 0.f;
      if (p.base == p.out) continue;
      for (int c = 8 * lane; c < p.N; c += 8 * 256) {
        uint4 q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          q[i] = p.base && c + 256 * i < p.N ? *reinterpret_cast<const uint4*>(p.base + t * p.ldb + c + 256 * i) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (c + 256 * i < p.N) *reinterpret_cast<uint4*>(p.out + t * p.N + c + 256 * i) = q[i];
      }
    }
  }
  const int64_t units = (int64_t)tile_table<kExpandRows>(p.g, first, warp_sum) * p.col_blocks;
  int64_t unit = units * me / all;
  const int64_t end = units * (me + 1) / all;
  const uint32_t bv = smem_u32(smem), bw = bv + C::V;
  const uint32_t slots = bw + 2 * C::W + (uint32_t)(warp * C::DEPTH * 2048 + lane * 16);
  const int qr = lane >> 2, qc = lane & 3, half = warp >> 2, first_row = 32 * (warp & 3);
  constexpr uint32_t idesc = idesc_bf16(128, 128, 0, 1);
  bool waited = false, stop = false;
  uint32_t issued = 0, k = 0;  // pieces whose product was issued, pieces done
  // everyone has stored its part of piece `issued`'s W (and v); one thread issues its product
  auto product = [&]() {
    fence_proxy_async_smem();
    tc_fence_before();  // this thread's loads of the half that is overwritten
    if (__syncthreads_or(pipe.fail)) return false;
    if (tid == 0) {
      tc_fence_after();
      const uint32_t w0 = bw + (issued & 1) * C::W;
#pragma unroll
      for (int kk = 0; kk < RP / 8; ++kk)  // v's two parts one behind the other along the sum, each with all of W
        mma_bf16(tmem + (issued & 1) * 128, kmajor_sw128_desc(bv + (kk >> 2) * 16384 + (kk & 3) * 32),
                 mnmajor_sw128_desc(w0 + kk % (RP / 16) * 2048, RP * 128), idesc, kk > 0 ? 1u : 0u);
      mma_commit(&sh.done[issued & 1]);
    }
    ++issued;
    return true;
  };
  int tile = (int)(unit / p.col_blocks), cb = (int)(unit - (int64_t)tile * p.col_blocks);
  for (; unit < end && !stop; ++tile, cb = 0) {
    const Tile t = tile_of<kExpandRows>(p.g, first, tile);
    const int a = t.a, rows = t.rows;
    const int64_t r0 = t.r0;
    __syncthreads();  // everyone is done with the last tile's
    if (tid < kExpandRows) tok[tid] = tid < rows ? token_of(p.g, (int)r0 + tid) : -1;
    const uint16_t* W = p.W + (int64_t)a * p.R * p.N + (int64_t)(tid >> 4) * p.N + 8 * (tid & 15);
    uint4 w[RP / 16];
    auto load_w = [&](int block) {
      const bool in = block * 128 + 8 * (tid & 15) < p.N;
#pragma unroll
      for (int i = 0; i < RP / 16; ++i)
        w[i] = in && (tid >> 4) + 16 * i < p.R ? *reinterpret_cast<const uint4*>(W + (int64_t)16 * i * p.N + block * 128)
                                               : make_uint4(0, 0, 0, 0);
    };
    auto store_w = [&](uint32_t buffer) {
#pragma unroll
      for (int i = 0; i < RP / 16; ++i) {
        const int row = (tid >> 4) + 16 * i, pc = tid & 15;
        const uint32_t ww[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
        // columns 8 pc + 2 j, + 1 of group pc / 4 of 32: columns 2 (pc % 4), + 1 of that group's tile j
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<uint32_t*>(smem + C::V + buffer * C::W + (pc >> 3) * RP * 128 + at<128>(row, (pc & 4) + j) +
                                       4 * (pc & 3)) = ww[j];
      }
    };
    // the warp's 16 tokens x 64 columns in order: (block, m); this thread's 64 bytes of them go to its own slot
    int fb = cb, fm = 0, fslot = 0;
    const int fb_end = first_row >= rows ? cb : p.col_blocks - cb < end - unit ? p.col_blocks : cb + (int)(end - unit);
    auto fetch = [&]() {
      if (p.base && fb < fb_end) {
        const int c = fb * 128 + 64 * half + 8 * qc;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int t = tok[first_row + 16 * fm + qr + 8 * h];
          const uint16_t* src = p.base + (t < 0 ? 0 : t) * p.ldb;
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const bool ok = t >= 0 && c + 32 * g < p.N;
            cp_async_16_zfill(slots + (uint32_t)(fslot * 4 + 2 * h + g) * 512, ok ? src + c + 32 * g : p.base, ok ? 16u : 0u);
          }
        }
      }
      cp_async_commit();
      fslot = fslot == C::DEPTH - 1 ? 0 : fslot + 1;
      fm ^= 1;
      fb += fm == 0;
    };
    load_w(cb);
    __syncthreads();  // tok
#pragma unroll
    for (int i = 0; i < C::DEPTH; ++i) fetch();
    store_w(issued & 1);
    if (!waited) {
      pdl_wait();  // v
      pdl_trigger();
      waited = true;
    }
    for (int i = tid; i < rows * (RP / 4); i += kThreads) {  // rows behind them only reach sums that nobody reads
      const int row = i / (RP / 4), c = i % (RP / 4);
      cp_async_16(bv + (c >> 3) * 16384 + at<128>(row, c & 7), p.v + (r0 + row) * 2 * RP + 8 * c);
    }
    cp_async_commit();
    cp_async_wait<0>();
    stop = !product();
    if (unit + 1 < end && cb + 1 < p.col_blocks) load_w(cb + 1);
    int slot = 0;
    for (; unit < end && cb < p.col_blocks && !stop; ++unit, ++cb, ++k) {
      if (unit + 1 < end && cb + 1 < p.col_blocks) {
        store_w(issued & 1);  // piece k - 1, whose buffer it is, is done
        stop = !product();
        if (stop) break;
        if (unit + 2 < end && cb + 2 < p.col_blocks) load_w(cb + 2);
      }
      if (!mbar_wait_bounded(&sh.done[k & 1], (k >> 1) & 1u, p.w.status, &sh.abort_flag, p.w.ns)) pipe.fail = true;
      if (first_row >= rows) continue;
      tc_fence_after();
      cp_async_wait<C::DEPTH - 2>();
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        uint32_t r[2][16];
        const uint32_t taddr = tmem + ((uint32_t)(first_row + 16 * m) << 16) + (k & 1) * 128 + 64 * half;
        tmem_ld_16x256b_x4(taddr, r[0]);
        tmem_ld_16x256b_x4(taddr + 32, r[1]);
        uint32_t o[2][2][4] = {};
        if (p.base) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int g = 0; g < 2; ++g) ld_shared_v4(o[h][g], slots + (uint32_t)(slot * 4 + 2 * h + g) * 512);
        }
        slot = slot == C::DEPTH - 1 ? 0 : slot + 1;
        tmem_ld_wait_regs<16>(r[0]);
        tmem_ld_wait_regs<16>(r[1]);
        const int c = cb * 128 + 64 * half + 8 * qc;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int t = tok[first_row + 16 * m + qr + 8 * h];
          if (t < 0) continue;
          uint16_t* out = p.out + (int64_t)t * p.N + c;
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            if (c + 32 * g >= p.N) continue;
            uint32_t y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              y[j] = pack_bf16x2(__uint_as_float(o[h][g][j] << 16) + __uint_as_float(r[g][4 * j + 2 * h]),
                                 __uint_as_float(o[h][g][j] & 0xFFFF0000u) + __uint_as_float(r[g][4 * j + 2 * h + 1]));
            *reinterpret_cast<uint4*>(out + 32 * g) = make_uint4(y[0], y[1], y[2], y[3]);
          }
        }
        __syncwarp();
        fetch();
      }
    }
  }
  if (!waited) {
    pdl_wait();
    pdl_trigger();
  }
  cp_async_wait<0>();
  if ((stop || pipe.fail) && issued) mbar_wait_drain(&sh.done[(issued - 1) & 1], ((issued - 1) >> 1) & 1u, p.w.status);
  tc_fence_before();
  __syncthreads();
  pipe.end(tmem, 2 * 128);
  if (p.sums.ranges) sum_partials(p.sums, me, all);
}

// ------------------------------------------------------------------------------------------
// grad: dW_a[R, K] = sum over the adapter's rows of v[row]^T x[token(row)]
// ------------------------------------------------------------------------------------------
// All r rows by 256 features over a range of tokens, 32 of one adapter a stage, as features x r on the tensor core: x and v
// are MN-major operands (a token's features are contiguous, the sum runs over tokens), gathered by asynchronous copies into the
// swizzled layout, one thread issues the products, two accumulators of 128 features stay in TMEM until the adapter changes.
// Equal ranges make one whole wave of CTAs whatever the adapters; tiles of one adapter's rows are uneven and do not fill
// their waves (backward of 16384 x (4096 + 4096) at rank 64: 181 us, with ranges 164).  Now 56 us; the copies alone take 43, the
// products 4 more, the partial sums at the end of the ranges 8.
template <int RP>
struct GradCfg {
  static constexpr int ROWS = 32, GROUP = ROWS * 128;  // 64 features (or ranks) of all tokens of a stage
  static constexpr int X = 4 * GROUP, STAGE = X + (RP <= 32 ? 1 : RP / 32) * GROUP;
  static constexpr int STAGES = RP <= 32 ? 5 : RP <= 64 ? 4 : 3;
  // v's truncated values and what they leave: columns of one product, joined at the end, or (rank 128) two products.  Twice the
  // products took 8 us more of 57 at rank 64.
  static constexpr int PARTS = RP <= 64 ? 2 : 1, N = PARTS * RP, TMEM = 2 * N;
  static constexpr int SMEM = 1024 + STAGES * STAGE;
};
struct Segment {
  int a, r, end;  // adapter, next row, row behind the adapter's last in the range
};
__device__ __forceinline__ void next_segment(const Groups& g, int hi, Segment& s) {
  while (s.end <= s.r && s.r < hi) {  // the last adapter takes what wrong offsets leave over
    ++s.a;
    const int o1 = s.a + 1 < g.n ? clamp_row(g.off[s.a + 1], g.T) : hi;
    s.end = o1 < hi ? o1 : hi;
  }
}
template <int RP>
__global__ void __launch_bounds__(kThreads, 2) adapter_grad_kernel(const GradArgs p) {
  using C = GradCfg<RP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ int tok[kMaxPer];
  __shared__ PipeShared<C::STAGES> pipe_shared;
  Pipe<C::STAGES> pipe(pipe_shared);
  const uint32_t tmem = pipe.start(C::TMEM);
  pdl_wait();
  pdl_trigger();  // after the allocation, as in the shrink kernel
  int rows;
  const int per = rows_of_range(p.g, p.ranges, rows);
  const int lo = row_at(p.g, (int64_t)blockIdx.y * per, rows), behind = row_at(p.g, (int64_t)(blockIdx.y + 1) * per, rows);
  const int hi = behind - lo < kMaxPer ? behind : lo + kMaxPer;  // less only with wrong offsets
  if (lo >= hi) {
    pipe.end(tmem, C::TMEM);
    return;
  }
  const GradProblem& q = p.pr[(int)blockIdx.x < p.pr[0].blocks ? 0 : 1];
  const int n0 = ((int)blockIdx.x < p.pr[0].blocks ? (int)blockIdx.x : (int)blockIdx.x - p.pr[0].blocks) * 256;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = smem_u32(smem);
  for (int i = tid; i < hi - lo; i += kThreads) tok[i] = token_of(p.g, lo + i);
  // the adapter of the range's first row: the last that begins at or before it
  int at_or_before = 0;
  for (int i0 = 0; i0 < p.g.n; i0 += kThreads)
    at_or_before += __syncthreads_count(i0 + tid < p.g.n && clamp_row(p.g.off[i0 + tid < p.g.n ? i0 + tid : 0], p.g.T) <= lo);
  Segment put{at_or_before > 0 ? at_or_before - 2 : -1, lo, lo};
  next_segment(p.g, hi, put);
  Segment get = put;
  // copies: a warp a token's 256 features, four tokens; v's rows one behind another
  const uint32_t in = n0 + 8 * lane < q.K ? 16u : 0u;
  const uint16_t* xcol = q.x + (in ? n0 + 8 * lane : 0);
  const int64_t ld = q.ld;
  const uint32_t xd = base + (lane >> 3) * C::GROUP + at<128>(4 * warp, lane & 7);
  constexpr int PIECES = RP / 4, VSTEP = kThreads / PIECES, VN = (C::ROWS + VSTEP - 1) / VSTEP;  // v rows of one pass, passes
  const int v0 = tid / PIECES, vc = tid % PIECES;
  const uint16_t* vcol = q.v + (int64_t)v0 * 2 * RP + 8 * vc;
  const uint32_t vd = base + C::X + (vc >> 3) * C::GROUP + at<128>(v0, vc & 7);  // VSTEP is a multiple of 8
  auto load = [&](uint32_t st) {  // the next rows, at most 32 of one adapter
    const int count = put.end - put.r;
    const int* tk = tok + (put.r - lo) + 4 * warp;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 4 * warp + i < count ? tk[i] : -1;
      cp_async_16_zfill((xd ^ (uint32_t)(i << 4)) + i * 128 + st, xcol + (int64_t)(t < 0 ? 0 : t) * ld, t < 0 ? 0u : in);
    }
#pragma unroll
    for (int i = 0; i < VN; ++i) {
      const int row = v0 + i * VSTEP;
      if (VSTEP * (i + 1) <= C::ROWS || row < C::ROWS) {
        const bool ok = row < count;
        cp_async_16_zfill(vd + i * VSTEP * 128 + st, vcol + (int64_t)(ok ? put.r + i * VSTEP : 0) * 2 * RP, ok ? 16u : 0u);
      }
    }
    put.r += C::ROWS;
    if (put.r >= put.end) {
      put.r = put.end;
      next_segment(p.g, hi, put);
    }
  };
#pragma unroll
  for (int i = 0; i < C::STAGES - 1; ++i) {
    if (put.r < hi) load(i * C::STAGE);
    cp_async_commit();
  }
  constexpr uint32_t idesc = idesc_bf16(128, C::N, 1, 1);
  bool more = false;  // the accumulators hold rows of this adapter
  while (get.r < hi) {
    cp_async_wait<C::STAGES - 2>();
    fence_proxy_async_smem();
    if (__syncthreads_or(pipe.fail)) break;
    if (tid == 0) {
      tc_fence_after();
      const uint32_t a0 = base + pipe.at * C::STAGE;
#pragma unroll
      for (int kk = 0; kk < C::ROWS / 16; ++kk)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int part = 0; part < 2; part += C::PARTS)
            mma_bf16(tmem + h * C::N, mnmajor_sw128_desc(a0 + h * 2 * C::GROUP + kk * 2048, C::GROUP),
                     mnmajor_sw128_desc(a0 + C::X + part * (RP / 64) * C::GROUP + kk * 2048, C::GROUP), idesc,
                     (more || kk > 0 || part > 0) ? 1u : 0u);
      pipe.commit();
    }
    more = true;
    pipe.advance(p.w);
    if (put.r < hi) load(pipe.free * C::STAGE);
    cp_async_commit();
    get.r += C::ROWS;
    if (get.r < get.end) continue;
    get.r = get.end;
    // the adapter's last rows of this range
    const bool starts = clamp_row(p.g.off[get.a], p.g.T) >= lo, ends = clamp_row(p.g.off[get.a + 1], p.g.T) <= hi;
    const bool whole = starts && ends;
    float* part = whole ? nullptr : q.part + (int64_t)(2 * (int)blockIdx.y + (starts ? 1 : 0)) * p.R * q.K;
    uint16_t* dW = q.dW + (int64_t)get.a * p.R * q.K;
    pipe.settle(p.w);
    tc_fence_after();
    // lanes are features: 32 of them a row of the result
    const int h = warp >> 2, f = n0 + 128 * h + 32 * (warp & 3) + lane;
    const uint32_t taddr = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + h * C::N;
    for (int m0 = 0; m0 < RP && m0 < p.R; m0 += 16) {
      uint32_t r[16];
      tmem_ld_32x32b_x16(taddr + m0, r);
      if constexpr (C::PARTS == 2) {
        uint32_t l[16];
        tmem_ld_32x32b_x16(taddr + RP + m0, l);
        tmem_ld_wait_regs<16>(r);
        tmem_ld_wait_regs<16>(l);
#pragma unroll
        for (int j = 0; j < 16; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) + __uint_as_float(l[j]));
      } else {
        tmem_ld_wait_regs<16>(r);
      }
      if (!whole) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (m0 + j < p.R && f < q.K) part[(int64_t)(m0 + j) * q.K + f] = __uint_as_float(r[j]);
      } else {
#pragma unroll
        for (int j = 0; j < 16; j += 2) {  // even lanes take row j of two features, odd ones row j + 1
          const bool odd = lane & 1;
          const float got = __shfl_xor_sync(0xFFFFFFFFu, __uint_as_float(odd ? r[j] : r[j + 1]), 1);
          const float own = __uint_as_float(odd ? r[j + 1] : r[j]);
          float f0 = odd ? got : own, f1 = odd ? own : got;
          const int m = m0 + j + (odd ? 1 : 0);
          if (m >= p.R || f >= q.K) continue;  // K is a multiple of 8
          uint32_t* d = reinterpret_cast<uint32_t*>(dW + (int64_t)m * q.K + (f & ~1));
          if (p.accumulate) {
            f0 += __uint_as_float(*d << 16);
            f1 += __uint_as_float(*d & 0xFFFF0000u);
          }
          *d = pack_bf16x2(f0, f1);
        }
      }
    }
    tc_fence_before();  // the next products wait for the next barrier
    more = false;
    next_segment(p.g, hi, get);
  }
  cp_async_wait<0>();
  if (pipe.begun) pipe.settle(p.w);
  tc_fence_before();
  __syncthreads();
  pipe.end(tmem, C::TMEM);
}

// ------------------------------------------------------------------------------------------
// host
// ------------------------------------------------------------------------------------------
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int padded_rank(int64_t r) { return r <= 16 ? 16 : r <= 32 ? 32 : r <= 64 ? 64 : 128; }
int64_t slots_of(int64_t T, int64_t n, int64_t per) { return T / per + std::min(n, T); }  // tiles at most

// Parts of the rows in the gradient: one wave of CTAs, but 64 rows a part at least and kMaxPer at most.
int grad_ranges(int64_t T, int64_t H, int64_t N, int64_t n, int sms) {
  const int64_t wave = 2 * sms / (cdiv(H, 256) + cdiv(N, 256));
  return (int)std::max(cdiv(T + kSegment * n, kMaxPer), std::min(wave, cdiv(T, 64)));
}
template <int RP, int SPLIT>
int launch_shrink(const ShrinkArgs& a, cudaStream_t st) {
  using C = ShrinkCfg<RP>;
  auto kern = adapter_shrink_kernel<RP, SPLIT>;
  const dim3 grid((unsigned)(slots_of(a.g.T, a.g.n, C::ROWS) * SPLIT));
  if constexpr (SPLIT == 1) {
    return launch_pdl(kern, grid, dim3(kThreads), C::SMEM, st, "adapter shrink", a);
  } else {
    const int rc = allow_smem(reinterpret_cast<const void*>(kern), C::SMEM);
    if (rc) return rc;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = SPLIT;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see launch_pdl
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = option(MOE_OPT_PDL) ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a);
    count_launch();
    if (e != cudaSuccess) return cuda_check(e, "adapter shrink");
    return cuda_check(cudaGetLastError(), "adapter shrink");
  }
}
// CTAs along the contraction: as many as still make one wave of two CTAs an SM.  (Tiles of fewer rows that fill the wave to the
// last SM, 111 instead of 128 at 16384 rows, measured the same, 33 us.)
template <int RP>
int run_shrink(const ShrinkArgs& a, int sms, cudaStream_t st) {
  using C = ShrinkCfg<RP>;
  const int64_t tiles = slots_of(a.g.T, a.g.n, C::ROWS), chunks = cdiv(a.K, C::KC);
  const auto fits = [&](int s) { return tiles * s <= 2 * sms && chunks >= s; };
  return fits(8) ? launch_shrink<RP, 8>(a, st) : fits(4) ? launch_shrink<RP, 4>(a, st) : fits(2) ? launch_shrink<RP, 2>(a, st)
                                                                                              : launch_shrink<RP, 1>(a, st);
}
template <int RP>
int run_expand(ExpandArgs a, int sms, cudaStream_t st) {
  const int64_t wave = (RP <= 64 ? 2 : 1) * sms;
  a.col_blocks = (int)cdiv(a.N, 128);
  int64_t most = std::max(slots_of(a.g.T, a.g.n, kExpandRows) * a.col_blocks, cdiv(a.g.T, 8));
  if (a.sums.ranges) most = std::max(most, (int64_t)a.g.n * cdiv((int64_t)a.R * (a.sums.pr[0].K + a.sums.pr[1].K), 4096));
  return launch_pdl(adapter_expand_kernel<RP>, dim3((unsigned)std::min(wave, most)), dim3(kThreads),
                    ExpandCfg<RP>::SMEM, st, "adapter expand", a);
}
template <int RP>
int run_grad(const GradArgs& a, cudaStream_t st) {
  return launch_pdl(adapter_grad_kernel<RP>, dim3((unsigned)(a.pr[0].blocks + a.pr[1].blocks), (unsigned)a.ranges), dim3(kThreads),
                    GradCfg<RP>::SMEM, st, "adapter gradient", a);
}
template <typename F>
int by_rank(int rp, F&& f) {
  switch (rp) {
    case 16: return f(std::integral_constant<int, 16>());
    case 32: return f(std::integral_constant<int, 32>());
    case 64: return f(std::integral_constant<int, 64>());
    default: return f(std::integral_constant<int, 128>());
  }
}

struct Layout {
  size_t v, su, grad0, grad1, total;
};
Layout layout(int64_t T, int64_t H, int64_t N, int64_t n, int64_t r, bool backward, int sms) {
  Layout L{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes, 256);
    return at;
  };
  const int rp = padded_rank(r);
  L.v = take((size_t)T * rp * 4);
  if (backward) {
    L.su = take((size_t)T * rp * 4);
    const size_t places = 2 * (size_t)grad_ranges(T, H, N, n, sms);
    L.grad0 = take(places * r * H * 4);
    L.grad1 = take(places * r * N * 4);
  }
  L.total = off;
  return L;
}

int check_sizes(const char* who, int64_t T, int64_t H, int64_t N, int64_t n, int64_t r) {
  if (T < 0 || H <= 0 || N <= 0 || n <= 0 || r <= 0) return fail(MOE_ERR_INVALID, "%s: bad sizes", who);
  if (H % 8 || N % 8) return fail(MOE_ERR_UNSUPPORTED, "%s: H and N must be multiples of 8", who);
  if (r > 128) return fail(MOE_ERR_UNSUPPORTED, "%s: rank above 128", who);
  if (n > kMaxExperts) return fail(MOE_ERR_UNSUPPORTED, "%s: more than %d adapters", who, kMaxExperts);
  if (T > (1 << 24) || H > (1 << 20) || N > (1 << 20)) return fail(MOE_ERR_UNSUPPORTED, "%s: too large", who);
  return MOE_OK;
}
bool off16(const void* p) { return reinterpret_cast<uintptr_t>(p) & 15; }
bool off4(const void* p) { return reinterpret_cast<uintptr_t>(p) & 3; }

}  // namespace
}  // namespace moebwd

using namespace moebwd;

extern "C" size_t adapter_workspace_size(int64_t T, int64_t H, int64_t N, int64_t n, int64_t r, int backward) {
  if (T <= 0 || H <= 0 || N <= 0 || n <= 0 || r <= 0 || r > 128) return 0;
  return layout(T, H, N, n, r, backward != 0, device_sm_count()).total;
}

extern "C" int adapter_fwd(const void* x, int64_t ldx, const void* A, const void* B, const float* scale, const void* base,
                           int64_t ldbase, const int32_t* expert_offsets, const int32_t* x_gather_idx,
                           const int32_t* s_reverse_scatter_idx, int64_t T, int64_t H, int64_t N, int64_t n, int64_t r, void* y,
                           float* u, int32_t* status_dev, void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  clear_error();
  int rc = check_sizes("adapter_fwd", T, H, N, n, r);
  if (rc || T == 0) return rc;
  if (!x || !A || !B || !expert_offsets || !x_gather_idx || !s_reverse_scatter_idx || !y || !workspace)
    return fail(MOE_ERR_INVALID, "adapter_fwd: null pointer");
  if (T == 1) ldx = H, ldbase = N;  // a row alone: its stride is never used
  if (ldx < H || ldx % 8 || (base && (ldbase < N || ldbase % 8)))
    return fail(MOE_ERR_INVALID, "adapter_fwd: row stride too small or not a multiple of 8");
  if (base == y && ldbase != N) return fail(MOE_ERR_INVALID, "adapter_fwd: y may be the base only where its row stride is N");
  if (off16(x) || off16(A) || off16(B) || off16(base) || off16(y)) return fail(MOE_ERR_INVALID, "adapter_fwd: tensors must be 16-byte aligned");
  if (off4(scale) || off4(expert_offsets) || off4(x_gather_idx) || off4(s_reverse_scatter_idx) || off4(u) || off4(status_dev))
    return fail(MOE_ERR_INVALID, "adapter_fwd: metadata, scales, u and status must be 4-byte aligned");
  if (reinterpret_cast<uintptr_t>(workspace) & 255) return fail(MOE_ERR_INVALID, "adapter_fwd: workspace must be 256-byte aligned");
  const int sms = device_sm_count();
  const Layout L = layout(T, H, N, n, r, false, sms);
  if (workspace_bytes < L.total) return fail(MOE_ERR_INVALID, "adapter_fwd: workspace too small (%zu < %zu)", workspace_bytes, L.total);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const Groups g{expert_offsets, x_gather_idx, (int)n, (int)T};
  ShrinkArgs s{};
  s.g = g; s.x = static_cast<const uint16_t*>(x); s.ld = ldx; s.W = static_cast<const uint16_t*>(A); s.scale = scale;
  s.v = reinterpret_cast<uint16_t*>(static_cast<char*>(workspace) + L.v); s.u = u;
  s.K = (int)H; s.R = (int)r;
  s.w = Waits{status_dev, (uint64_t)option(MOE_OPT_WAIT_LIMIT_NS)};
  ExpandArgs e{};
  e.g = g; e.v = s.v; e.W = static_cast<const uint16_t*>(B);
  e.base = static_cast<const uint16_t*>(base); e.ldb = ldbase; e.out = static_cast<uint16_t*>(y); e.back = s_reverse_scatter_idx;
  e.u = u; e.N = (int)N; e.R = (int)r; e.w = s.w;
  return by_rank(padded_rank(r), [&](auto k) {
    constexpr int RP = decltype(k)::value;
    const int rc1 = run_shrink<RP>(s, sms, st);
    return rc1 ? rc1 : run_expand<RP>(e, sms, st);
  });
}

extern "C" int adapter_bwd(const void* dy, int64_t lddy, const void* x, int64_t ldx, const float* u, const void* A, const void* B,
                           const float* scale, const void* base, int64_t ldbase, const int32_t* expert_offsets,
                           const int32_t* x_gather_idx, const int32_t* s_reverse_scatter_idx, int64_t T, int64_t H, int64_t N,
                           int64_t n, int64_t r, void* dx, void* dA, void* dB, int accumulate, int32_t* status_dev, void* workspace,
                           size_t workspace_bytes, moe_stream_t stream) {
  clear_error();
  int rc = check_sizes("adapter_bwd", T, H, N, n, r);
  if (rc) return rc;
  if (accumulate != 0 && accumulate != 1) return fail(MOE_ERR_INVALID, "adapter_bwd: accumulate must be 0 or 1");
  if (!dA || !dB) return fail(MOE_ERR_INVALID, "adapter_bwd: null pointer");
  if (off16(dA) || off16(dB)) return fail(MOE_ERR_INVALID, "adapter_bwd: tensors must be 16-byte aligned");
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0) {  // empty sums
    if (accumulate) return MOE_OK;
    if ((rc = cuda_check(cudaMemsetAsync(dA, 0, (size_t)n * r * H * 2, st), "memset dA"))) return rc;
    return cuda_check(cudaMemsetAsync(dB, 0, (size_t)n * r * N * 2, st), "memset dB");
  }
  if (!dy || !x || !u || !A || !B || !expert_offsets || !x_gather_idx || !s_reverse_scatter_idx || !dx || !workspace)
    return fail(MOE_ERR_INVALID, "adapter_bwd: null pointer");
  if (T == 1) ldx = ldbase = H, lddy = N;  // as in adapter_fwd
  if (ldx < H || ldx % 8 || lddy < N || lddy % 8 || (base && (ldbase < H || ldbase % 8)))
    return fail(MOE_ERR_INVALID, "adapter_bwd: row stride too small or not a multiple of 8");
  if (base == dx && ldbase != H) return fail(MOE_ERR_INVALID, "adapter_bwd: dx may be the base only where its row stride is H");
  if (off16(dy) || off16(x) || off16(A) || off16(B) || off16(base) || off16(dx))
    return fail(MOE_ERR_INVALID, "adapter_bwd: tensors must be 16-byte aligned");
  if (off4(scale) || off4(expert_offsets) || off4(x_gather_idx) || off4(s_reverse_scatter_idx) || off4(u) || off4(status_dev))
    return fail(MOE_ERR_INVALID, "adapter_bwd: metadata, scales, u and status must be 4-byte aligned");
  if (reinterpret_cast<uintptr_t>(workspace) & 255) return fail(MOE_ERR_INVALID, "adapter_bwd: workspace must be 256-byte aligned");
  const int sms = device_sm_count();
  const Layout L = layout(T, H, N, n, r, true, sms);
  if (workspace_bytes < L.total) return fail(MOE_ERR_INVALID, "adapter_bwd: workspace too small (%zu < %zu)", workspace_bytes, L.total);
  char* ws = static_cast<char*>(workspace);
  const Groups g{expert_offsets, x_gather_idx, (int)n, (int)T};
  ShrinkArgs s{};
  s.g = g; s.x = static_cast<const uint16_t*>(dy); s.ld = lddy; s.W = static_cast<const uint16_t*>(B); s.scale = scale;
  s.v = reinterpret_cast<uint16_t*>(ws + L.v); s.u_in = u; s.su = reinterpret_cast<uint16_t*>(ws + L.su);
  s.K = (int)N; s.R = (int)r;
  s.w = Waits{status_dev, (uint64_t)option(MOE_OPT_WAIT_LIMIT_NS)};
  ExpandArgs e{};
  e.g = g; e.v = s.v; e.W = static_cast<const uint16_t*>(A);
  e.base = static_cast<const uint16_t*>(base); e.ldb = ldbase; e.out = static_cast<uint16_t*>(dx); e.back = s_reverse_scatter_idx;
  e.N = (int)H; e.R = (int)r; e.w = s.w;
  GradArgs d{};
  d.g = g; d.R = (int)r; d.ranges = grad_ranges(T, H, N, n, sms); d.accumulate = accumulate;
  d.w = s.w;
  d.pr[0] = GradProblem{static_cast<const uint16_t*>(x), s.v, static_cast<uint16_t*>(dA), reinterpret_cast<float*>(ws + L.grad0), ldx,
                        (int)H, (int)cdiv(H, 256)};
  d.pr[1] = GradProblem{static_cast<const uint16_t*>(dy), s.su, static_cast<uint16_t*>(dB), reinterpret_cast<float*>(ws + L.grad1), lddy,
                        (int)N, (int)cdiv(N, 256)};
  e.sums = d;
  return by_rank(padded_rank(r), [&](auto k) {
    constexpr int RP = decltype(k)::value;
    int rc1 = run_shrink<RP>(s, sms, st);
    if (!rc1) rc1 = run_grad<RP>(d, st);  // right behind the kernel that read dy: an eighth of it (17 of 134 MB, rank 64) still comes from L2
    return rc1 ? rc1 : run_expand<RP>(e, sms, st);
  });
}
