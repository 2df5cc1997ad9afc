// Low-rank adapters of many requests beside a shared projection, forward and backward.  Token t belongs to adapter a(t) or to
// none; A_a [r, H] and B_a [r, N] hold r rows each, contiguous along the features:
//
//   u_t = A_a x_t,  y_t = base_t + c_a B_a^T u_t
//   v_t = c_a B_a dy_t,  dx_t = base_t + A_a^T v_t,  dA_a = sum_t v_t x_t^T,  dB_a = sum_t (c_a u_t) dy_t^T
//
// With both matrices stored as r feature rows, the forward and the backward are the same two kernels: adapter_shrink
// contracts a token's features with r rows, adapter_expand adds r rows weighted by r numbers onto a token's row.
// adapter_grad is the third.  Tokens are taken in route_meta's order (expert_offsets, x_gather_idx with K = 1), so that 64
// tokens of one adapter share its matrices; tiles never mix adapters.
//
// Bound: HBM (2 r operations a byte).  Products run on the warp-level matrix instruction (m16n8k16, bf16, fp32 sums): at r
// = 64 its rate is far from the bound, its operands come straight from the tiles that asynchronous copies gather by token
// index, and groups of one or two tokens (decoding) waste nothing but idle rows.
// r numbers a token go between the kernels in fp32; they are rounded to bf16 as operands of the next product.
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "ptx.cuh"
#include "mx_device.cuh"

namespace moebwd {
namespace {

constexpr int kRows = 64;      // tokens of a tile
constexpr int kChunk = 128;    // features of a pipeline stage
constexpr int kThreads = 128;  // four warps: 16 tokens each (shrink, expand), 32 features each (grad)
constexpr int kStages = 3;
constexpr int kMaxSplit = 16;
constexpr int kMaxPer = 1024;  // rows of a gradient tile at most

struct Groups {
  const int32_t* off;  // [n + 1]
  const int32_t* idx;  // [T] grouped row -> token
  int n, T;
};

__device__ __forceinline__ int clamp_row(int v, int T) { return v < 0 ? 0 : v > T ? T : v; }

struct Tile {
  int a, r0, rows, index, count;  // adapter, first grouped row, rows, tile of the adapter, its rows in all
};

// Tiles of `per` rows: adapter a's begin at slot off[a] / per + a, which leaves room for all of them whatever the counts, so
// that no prefix sum is needed: at most T / per + n slots, and a slot's adapter is the last one that begins at or before
// it.  Offsets are clamped to [0, T]: bad ones give wrong tiles, never rows outside.  All threads call it.
__device__ __forceinline__ bool find_tile(const Groups& g, int slot, int per, Tile& t) {
  int at = 0;
  for (int i0 = 0; i0 < g.n; i0 += blockDim.x) {
    const int i = i0 + (int)threadIdx.x;
    at += __syncthreads_count(i < g.n && clamp_row(g.off[i < g.n ? i : 0], g.T) / per + i <= slot);
  }
  if (at == 0) return false;
  t.a = at - 1;
  const int o0 = clamp_row(g.off[t.a], g.T), o1 = clamp_row(g.off[at], g.T);
  t.index = slot - (o0 / per + t.a);
  t.count = o1 - o0;
  const int64_t r0 = o0 + (int64_t)t.index * per;
  if (r0 >= o1) return false;
  t.r0 = (int)r0;
  t.rows = o1 - t.r0 < per ? o1 - t.r0 : per;
  return true;
}

// Token of a grouped row, -1 where the metadata names none.
__device__ __forceinline__ int token_of(const Groups& g, int row) {
  const int t = g.idx[row];
  return t >= 0 && t < g.T ? t : -1;
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Byte of 16-byte piece `c` of row `row` in a tile of 256-byte rows: eight rows at one piece fall into eight bank groups.
__device__ __forceinline__ uint32_t at256(int row, int c) { return (uint32_t)(row * 256 + ((c ^ (row & 7)) << 4)); }
// The same for rows of RP bf16 numbers.
template <int RP>
__device__ __forceinline__ uint32_t at_rank(int row, int c) {
  constexpr int mask = RP / 8 < 8 ? RP / 8 - 1 : 7;
  return (uint32_t)(row * RP * 2 + ((c ^ (row & mask)) << 4));
}

// ------------------------------------------------------------------------------------------
// shrink: part[split, row, :] = x[token(row), its features] W_a^T
// ------------------------------------------------------------------------------------------
struct ShrinkArgs {
  Groups g;
  const uint16_t* x;  // [T, K], row stride ld
  const uint16_t* W;  // [n, R, K]
  float* part;        // [splits, T, RP]
  int64_t ld;
  int K, R, splits;
};

template <int RP>
__global__ void __launch_bounds__(kThreads) adapter_shrink_kernel(const ShrinkArgs p) {
  extern __shared__ __align__(256) uint8_t smem[];
  __shared__ int tok[kRows];
  constexpr int kStage = (kRows + RP) * 256;
  pdl_wait();
  pdl_trigger();
  Tile t;
  if (!find_tile(p.g, blockIdx.x, kRows, t)) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid < kRows) tok[tid] = tid < t.rows ? token_of(p.g, t.r0 + tid) : -1;
  __syncthreads();
  const int chunks = (p.K + kChunk - 1) / kChunk;
  const int c0 = (int)((int64_t)chunks * blockIdx.y / p.splits), c1 = (int)((int64_t)chunks * (blockIdx.y + 1) / p.splits);
  const uint16_t* W = p.W + (int64_t)t.a * p.R * p.K;
  const uint32_t base = smem_u32(smem);
  const int pc = tid & 15;  // this thread's 16-byte piece of every row it copies
  auto load = [&](int c) {
    const uint32_t s = base + (uint32_t)((c - c0) % kStages) * kStage;
    const int k = c * kChunk + 8 * pc;
    const uint32_t in = k < p.K ? 16u : 0u;  // K is a multiple of 8
#pragma unroll
    for (int i = 0; i < kRows / 8; ++i) {
      const int row = (tid >> 4) + 8 * i, tk = tok[row];
      if (row < ((t.rows + 15) & ~15))  // tiles of 16 rows that no warp reads are not filled
        cp_async_16_zfill(s + at256(row, pc), tk >= 0 && in ? p.x + (int64_t)tk * p.ld + k : p.x, tk >= 0 ? in : 0u);
    }
#pragma unroll
    for (int i = 0; i < RP / 8; ++i) {
      const int row = (tid >> 4) + 8 * i;
      const bool ok = row < p.R && in;
      cp_async_16_zfill(s + kRows * 256 + at256(row, pc), ok ? W + (int64_t)row * p.K + k : p.W, ok ? 16u : 0u);
    }
  };
  float acc[RP / 8][4];
#pragma unroll
  for (int i = 0; i < RP / 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
  for (int i = 0; i < kStages - 1; ++i) {
    if (c0 + i < c1) load(c0 + i);
    cp_async_commit();
  }
  for (int c = c0; c < c1; ++c) {
    cp_async_wait<kStages - 2>();
    __syncthreads();  // stage c has landed for everyone, and everyone is done with the stage refilled now
    if (c + kStages - 1 < c1) load(c + kStages - 1);
    cp_async_commit();
    if (warp * 16 < t.rows) {
      const uint32_t s = base + (uint32_t)((c - c0) % kStages) * kStage;
#pragma unroll
      for (int kk = 0; kk < kChunk / 16; ++kk) {
        uint32_t a[4];
        ldsm4(a, s + at256(warp * 16 + (lane & 15), 2 * kk + (lane >> 4)));
#pragma unroll
        for (int nb = 0; nb < RP / 16; ++nb) {
          uint32_t b[4];
          ldsm4(b, s + kRows * 256 + at256(nb * 16 + (lane & 7) + ((lane >> 4) << 3), 2 * kk + ((lane >> 3) & 1)));
          mma16816(acc[2 * nb], a, b[0], b[1]);
          mma16816(acc[2 * nb + 1], a, b[2], b[3]);
        }
      }
    }
  }
  cp_async_wait<0>();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int row = warp * 16 + (lane >> 2) + 8 * h;
    if (row >= t.rows) continue;
    float* out = p.part + ((int64_t)blockIdx.y * p.g.T + t.r0 + row) * RP + 2 * (lane & 3);
#pragma unroll
    for (int i = 0; i < RP / 8; ++i) *reinterpret_cast<float2*>(out + 8 * i) = make_float2(acc[i][2 * h], acc[i][2 * h + 1]);
  }
}

// ------------------------------------------------------------------------------------------
// expand: out[token] = base[token] + v W_a, v = c_a sum over the splits
// ------------------------------------------------------------------------------------------
struct ExpandArgs {
  Groups g;
  const float* part;     // [splits, T, RP]
  const float* scale;    // [n] or null
  const uint16_t* W;     // [n, R, N]
  const uint16_t* base;  // [T, N], row stride ldb, or null
  uint16_t* out;         // [T, N] dense
  const int32_t* back;   // [T] token -> grouped row, negative: none
  float* u;              // [T, R] unscaled sums by token, or null
  uint16_t* v;           // [T, RP] bf16 v by grouped row, or null
  const float* u_in;     // [T, R] with su [T, RP]: bf16 c_a u_in by grouped row, or null
  uint16_t* su;
  int64_t ldb;
  int N, R, splits, cols, col_blocks, slots;  // columns of a block (a multiple of 128)
};

// A tile's 64 tokens x `cols` columns, 128 at a time.  The columns of W are permuted within 32 on their way to shared memory
// so that a thread's four 8-column matrix tiles give it 8 neighbouring columns: base and out move in 16-byte pieces,
// four lanes to 64 bytes of a row, with no pass through shared memory.
template <int RP>
__global__ void __launch_bounds__(kThreads) adapter_expand_kernel(const ExpandArgs p) {
  extern __shared__ __align__(256) uint8_t smem[];
  uint8_t* sW = smem;
  uint8_t* sV = smem + RP * 256;
  __shared__ int tok[kRows];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int work = p.slots * p.col_blocks;
  if ((int)blockIdx.x >= work) {  // 64 tokens: rows without an adapter keep their base
    const int64_t t0 = ((int64_t)blockIdx.x - work) * kRows;
    for (int i = warp; i < kRows; i += 4) {
      const int64_t t = t0 + i;
      if (t >= p.g.T || p.back[t] >= 0) continue;
      if (p.u)
        for (int c = lane; c < p.R; c += 32) p.u[t * p.R + c] = 0.f;
      if (p.base == p.out) continue;
      for (int c = 8 * lane; c < p.N; c += 256)
        *reinterpret_cast<uint4*>(p.out + t * p.N + c) =
            p.base ? *reinterpret_cast<const uint4*>(p.base + t * p.ldb + c) : make_uint4(0, 0, 0, 0);
    }
    return;
  }
  Tile t;
  const int slot = blockIdx.x / p.col_blocks, block = blockIdx.x % p.col_blocks;
  if (!find_tile(p.g, slot, kRows, t)) return;
  if (tid < kRows) tok[tid] = tid < t.rows ? token_of(p.g, t.r0 + tid) : -1;
  __syncthreads();
  const float scale = p.scale ? p.scale[t.a] : 1.f;
  for (int i = tid; i < kRows * RP / 4; i += kThreads) {
    const int row = i / (RP / 4), c = 4 * (i % (RP / 4));
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row < t.rows) {
      const float* q = p.part + (int64_t)(t.r0 + row) * RP + c;
      for (int k = 0; k < p.splits; ++k) {
        const float4 f = *reinterpret_cast<const float4*>(q + (int64_t)k * p.g.T * RP);
        s.x += f.x;
        s.y += f.y;
        s.z += f.z;
        s.w += f.w;
      }
    }
    const uint2 w = make_uint2(pack_bf16x2(s.x * scale, s.y * scale), pack_bf16x2(s.z * scale, s.w * scale));
    *reinterpret_cast<uint2*>(sV + at_rank<RP>(row, c >> 3) + (c & 4) * 2) = w;
    if (block == 0 && row < t.rows) {
      const int tk = tok[row];
      const float f[4] = {s.x, s.y, s.z, s.w};
      if (p.u && tk >= 0)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (c + j < p.R) p.u[(int64_t)tk * p.R + c + j] = f[j];
      if (p.v) *reinterpret_cast<uint2*>(p.v + (int64_t)(t.r0 + row) * RP + c) = w;
      if (p.su) {
        float z[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) z[j] = tk >= 0 && c + j < p.R ? p.u_in[(int64_t)tk * p.R + c + j] * scale : 0.f;
        *reinterpret_cast<uint2*>(p.su + (int64_t)(t.r0 + row) * RP + c) = make_uint2(pack_bf16x2(z[0], z[1]), pack_bf16x2(z[2], z[3]));
      }
    }
  }
  const uint16_t* W = p.W + (int64_t)t.a * p.R * p.N;
  const uint32_t bw = smem_u32(sW), bv = smem_u32(sV);
  const int n1 = min(p.N, (block + 1) * p.cols);
  const int qr = lane >> 2, qc = lane & 3;
  int64_t rows[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int row = warp * 16 + qr + 8 * h;
    rows[h] = row < t.rows ? tok[row] : -1;
  }
  for (int n0 = block * p.cols; n0 < n1; n0 += 128) {
    uint4 b[2][4];  // base: two rows, four groups of 32 columns
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int c = n0 + 32 * g + 8 * qc;
        b[h][g] = p.base && rows[h] >= 0 && c < n1 ? *reinterpret_cast<const uint4*>(p.base + rows[h] * p.ldb + c)
                                                  : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
    for (int i = 0; i < RP / 8; ++i) {
      const int row = (tid >> 4) + 8 * i, pc = tid & 15;
      const int c = n0 + 8 * pc;
      const uint4 w = row < p.R && c < p.N ? *reinterpret_cast<const uint4*>(W + (int64_t)row * p.N + c) : make_uint4(0, 0, 0, 0);
      const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
      // columns 8 pc + 2 j, + 1 of group pc / 4: columns 2 (pc % 4), + 1 of that group's matrix tile j
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<uint32_t*>(sW + at256(row, (pc & 12) + j) + 4 * (pc & 3)) = ww[j];
    }
    __syncthreads();
    if (warp * 16 < t.rows) {
      float acc[16][4];
#pragma unroll
      for (int i = 0; i < 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll
      for (int kk = 0; kk < RP / 16; ++kk) {
        uint32_t a[4];
        ldsm4(a, bv + at_rank<RP>(warp * 16 + (lane & 15), 2 * kk + (lane >> 4)));
#pragma unroll
        for (int np = 0; np < 8; ++np) {
          uint32_t w[4];
          ldsm4t(w, bw + at256(kk * 16 + (lane & 7) + (((lane >> 3) & 1) << 3), 2 * np + (lane >> 4)));
          mma16816(acc[2 * np], a, w[0], w[1]);
          mma16816(acc[2 * np + 1], a, w[2], w[3]);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (rows[h] < 0) continue;
        uint16_t* out = p.out + rows[h] * p.N;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int c = n0 + 32 * g + 8 * qc;
          if (c >= n1) continue;
          const uint32_t o[4] = {b[h][g].x, b[h][g].y, b[h][g].z, b[h][g].w};
          uint32_t r[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            r[j] = pack_bf16x2(__uint_as_float(o[j] << 16) + acc[4 * g + j][2 * h],
                               __uint_as_float(o[j] & 0xFFFF0000u) + acc[4 * g + j][2 * h + 1]);
          *reinterpret_cast<uint4*>(out + c) = make_uint4(r[0], r[1], r[2], r[3]);
        }
      }
    }
    __syncthreads();  // sW is read
  }
}

// ------------------------------------------------------------------------------------------
// grad: dW_a[R, K] = sum over the adapter's rows of v[row]^T x[token(row)]
// ------------------------------------------------------------------------------------------
struct GradProblem {
  const uint16_t* x;  // [T, K], row stride ld
  const uint16_t* v;  // [T, RP] by grouped row
  uint16_t* dW;       // [n, R, K]
  float* part;        // [2 (T / per + 1), R, K]
  int64_t ld;
  int K, blocks;      // blocks of 128 features
};
struct GradArgs {
  Groups g;
  GradProblem pr[2];
  int R, per, accumulate;
};

// Partial sums of adapters with more than `per` rows: tile `index` at grouped row r0 goes to 2 (r0 / per) + (index == 0).  Two
// such adapters' first rows, and any two other tiles, are more than `per` rows apart, so that no two share a place.
__device__ __forceinline__ int part_of(int r0, int per, int index) { return 2 * (r0 / per) + (index == 0 ? 1 : 0); }

template <int RP>
__global__ void __launch_bounds__(kThreads) adapter_grad_kernel(const GradArgs p) {
  extern __shared__ __align__(256) uint8_t smem[];
  __shared__ int tok[kMaxPer];
  constexpr int kStage = kRows * 256 + kRows * RP * 2;
  pdl_wait();
  pdl_trigger();
  Tile t;
  if (!find_tile(p.g, blockIdx.y, p.per, t)) return;
  const GradProblem& q = p.pr[(int)blockIdx.x < p.pr[0].blocks ? 0 : 1];
  const int n0 = ((int)blockIdx.x < p.pr[0].blocks ? (int)blockIdx.x : (int)blockIdx.x - p.pr[0].blocks) * 128;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = smem_u32(smem);
  for (int i = tid; i < t.rows; i += kThreads) tok[i] = token_of(p.g, t.r0 + i);
  __syncthreads();
  const int steps = (t.rows + kRows - 1) / kRows;
  const int pc = tid & 15;
  const uint32_t in = n0 + 8 * pc < q.K ? 16u : 0u;
  auto load = [&](int s) {
    const uint32_t st = base + (uint32_t)(s % kStages) * kStage;
    const int r = s * kRows;
#pragma unroll
    for (int i = 0; i < kRows / 8; ++i) {
      const int row = (tid >> 4) + 8 * i;
      const int tk = r + row < t.rows ? tok[r + row] : -1;
      cp_async_16_zfill(st + at256(row, pc), tk >= 0 && in ? q.x + (int64_t)tk * q.ld + n0 + 8 * pc : q.x, tk >= 0 ? in : 0u);
    }
    for (int i = tid; i < kRows * RP / 8; i += kThreads) {
      const int row = i / (RP / 8), c = i % (RP / 8);
      const bool ok = r + row < t.rows;
      cp_async_16_zfill(st + kRows * 256 + at_rank<RP>(row, c), ok ? q.v + (int64_t)(t.r0 + r + row) * RP + 8 * c : q.v,
                        ok ? 16u : 0u);
    }
  };
  float acc[RP / 16][4][4];
#pragma unroll
  for (int i = 0; i < RP / 16; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[i][j][k] = 0.f;
  for (int i = 0; i < kStages - 1; ++i) {
    if (i < steps) load(i);
    cp_async_commit();
  }
  for (int s = 0; s < steps; ++s) {
    cp_async_wait<kStages - 2>();
    __syncthreads();
    if (s + kStages - 1 < steps) load(s + kStages - 1);
    cp_async_commit();
    const uint32_t st = base + (uint32_t)(s % kStages) * kStage;
#pragma unroll
    for (int kk = 0; kk < kRows / 16; ++kk) {
      uint32_t b[2][4];
#pragma unroll
      for (int np = 0; np < 2; ++np)
        ldsm4t(b[np], st + at256(kk * 16 + (lane & 7) + (((lane >> 3) & 1) << 3), warp * 4 + 2 * np + (lane >> 4)));
#pragma unroll
      for (int mt = 0; mt < RP / 16; ++mt) {
        uint32_t a[4];
        ldsm4t(a, st + kRows * 256 + at_rank<RP>(kk * 16 + (lane & 7) + ((lane >> 4) << 3), 2 * mt + ((lane >> 3) & 1)));
#pragma unroll
        for (int j = 0; j < 4; ++j) mma16816(acc[mt][j], a, b[j >> 1][2 * (j & 1)], b[j >> 1][2 * (j & 1) + 1]);
      }
    }
  }
  cp_async_wait<0>();
  const bool whole = t.count <= p.per;
  float* part = whole ? nullptr : q.part + (int64_t)part_of(t.r0, p.per, t.index) * p.R * q.K;
  uint16_t* dW = q.dW + (int64_t)t.a * p.R * q.K;
#pragma unroll
  for (int mt = 0; mt < RP / 16; ++mt)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int m = mt * 16 + (lane >> 2) + 8 * h;
      if (m >= p.R) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = n0 + warp * 32 + 8 * j + 2 * (lane & 3);
        if (c >= q.K) continue;
        float f0 = acc[mt][j][2 * h], f1 = acc[mt][j][2 * h + 1];
        const int64_t o = (int64_t)m * q.K + c;
        if (!whole) {
          *reinterpret_cast<float2*>(part + o) = make_float2(f0, f1);
        } else {
          uint32_t* d = reinterpret_cast<uint32_t*>(dW + o);
          if (p.accumulate) {
            f0 += __uint_as_float(*d << 16);
            f1 += __uint_as_float(*d & 0xFFFF0000u);
          }
          *d = pack_bf16x2(f0, f1);
        }
      }
    }
}

// Sums of the partial tiles of an adapter with more than `per` rows, in order; zeros for one without rows.
__global__ void __launch_bounds__(256) adapter_reduce_kernel(const GradArgs p) {
  pdl_wait();
  pdl_trigger();
  const GradProblem& q = p.pr[blockIdx.z];
  const int a = blockIdx.y;
  const int o0 = clamp_row(p.g.off[a], p.g.T), o1 = clamp_row(p.g.off[a + 1], p.g.T);
  const int count = o1 - o0;
  if ((count > 0 && count <= p.per) || (count <= 0 && p.accumulate)) return;
  const int64_t size = (int64_t)p.R * q.K;
  const int tiles = count <= 0 ? 0 : (count + p.per - 1) / p.per;
  uint16_t* dW = q.dW + a * size;
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < size; i += (int64_t)gridDim.x * 1024) {  // K is a multiple of 8
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < tiles; ++k) {
      const float4 f = *reinterpret_cast<const float4*>(q.part + part_of(o0 + k * p.per, p.per, k) * size + i);
      s.x += f.x;
      s.y += f.y;
      s.z += f.z;
      s.w += f.w;
    }
    uint2* d = reinterpret_cast<uint2*>(dW + i);
    if (p.accumulate) {
      const uint2 w = *d;
      s.x += __uint_as_float(w.x << 16);
      s.y += __uint_as_float(w.x & 0xFFFF0000u);
      s.z += __uint_as_float(w.y << 16);
      s.w += __uint_as_float(w.y & 0xFFFF0000u);
    }
    *d = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
  }
}

// ------------------------------------------------------------------------------------------
// host
// ------------------------------------------------------------------------------------------
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int padded_rank(int64_t r) { return r <= 16 ? 16 : r <= 32 ? 32 : r <= 64 ? 64 : 128; }
int64_t slots_of(int64_t T, int64_t n, int64_t per) { return T / per + n; }

// CTAs along the contraction: enough for six an SM, no more than its chunks.
int splits_of(int64_t T, int64_t n, int64_t K, int sms) {
  const int64_t tiles = cdiv(T, kRows) + std::min<int64_t>(n, T) - 1;
  return (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(cdiv(K, kChunk), kMaxSplit), 6 * sms / std::max<int64_t>(tiles, 1)));
}
int grad_rows(int64_t T) { return T <= 4096 ? 256 : T <= 8192 ? 512 : kMaxPer; }

template <int RP>
int run_shrink(const ShrinkArgs& a, cudaStream_t st) {
  return launch_pdl(adapter_shrink_kernel<RP>, dim3((unsigned)slots_of(a.g.T, a.g.n, kRows), (unsigned)a.splits), dim3(kThreads),
                    (size_t)kStages * (kRows + RP) * 256, st, "adapter shrink", a);
}
template <int RP>
int run_expand(ExpandArgs a, int sms, cudaStream_t st) {
  a.slots = (int)slots_of(a.g.T, a.g.n, kRows);
  // 512 columns a CTA share the summation of a tile's r numbers; fewer where that leaves SMs without work
  const int64_t tiles = cdiv(a.g.T, kRows) + std::min<int64_t>(a.g.n, a.g.T) - 1;
  a.cols = 512;
  while (a.cols > 128 && tiles * cdiv(a.N, a.cols) < 4 * sms) a.cols /= 2;
  a.col_blocks = (int)cdiv(a.N, a.cols);
  const int64_t blocks = (int64_t)a.slots * a.col_blocks + cdiv(a.g.T, kRows);
  if (blocks > INT32_MAX) return fail(MOE_ERR_UNSUPPORTED, "adapter: too many tiles");
  return launch_pdl(adapter_expand_kernel<RP>, dim3((unsigned)blocks), dim3(kThreads), RP * 256 + kRows * RP * 2, st,
                    "adapter expand", a);
}
template <int RP>
int run_grad(const GradArgs& a, cudaStream_t st) {
  int rc = launch_pdl(adapter_grad_kernel<RP>, dim3((unsigned)(a.pr[0].blocks + a.pr[1].blocks), (unsigned)slots_of(a.g.T, a.g.n, a.per)),
                      dim3(kThreads), (size_t)kStages * (kRows * 256 + kRows * RP * 2), st, "adapter gradient", a);
  if (rc) return rc;
  const int64_t most = (int64_t)a.R * std::max(a.pr[0].K, a.pr[1].K);
  return launch_pdl(adapter_reduce_kernel, dim3((unsigned)std::min<int64_t>(cdiv(most, 1024), 64), (unsigned)a.g.n, 2), dim3(256), 0,
                    st, "adapter gradient sums", a);
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
  size_t part, v, su, grad0, grad1, total;
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
  L.part = take((size_t)splits_of(T, n, backward ? N : H, sms) * T * rp * 4);
  if (backward) {
    L.v = take((size_t)T * rp * 2);
    L.su = take((size_t)T * rp * 2);
    const size_t places = 2 * (size_t)(T / grad_rows(T) + 1);
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
                           float* u, void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  clear_error();
  int rc = check_sizes("adapter_fwd", T, H, N, n, r);
  if (rc || T == 0) return rc;
  if (!x || !A || !B || !expert_offsets || !x_gather_idx || !s_reverse_scatter_idx || !y || !workspace)
    return fail(MOE_ERR_INVALID, "adapter_fwd: null pointer");
  if (ldx < H || ldx % 8 || (base && (ldbase < N || ldbase % 8)))
    return fail(MOE_ERR_INVALID, "adapter_fwd: row stride too small or not a multiple of 8");
  if (base == y && ldbase != N) return fail(MOE_ERR_INVALID, "adapter_fwd: y may be the base only where its row stride is N");
  if (off16(x) || off16(A) || off16(B) || off16(base) || off16(y)) return fail(MOE_ERR_INVALID, "adapter_fwd: tensors must be 16-byte aligned");
  if (off4(scale) || off4(expert_offsets) || off4(x_gather_idx) || off4(s_reverse_scatter_idx) || off4(u))
    return fail(MOE_ERR_INVALID, "adapter_fwd: metadata, scales and u must be 4-byte aligned");
  if (reinterpret_cast<uintptr_t>(workspace) & 255) return fail(MOE_ERR_INVALID, "adapter_fwd: workspace must be 256-byte aligned");
  const int sms = device_sm_count();
  const Layout L = layout(T, H, N, n, r, false, sms);
  if (workspace_bytes < L.total) return fail(MOE_ERR_INVALID, "adapter_fwd: workspace too small (%zu < %zu)", workspace_bytes, L.total);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const Groups g{expert_offsets, x_gather_idx, (int)n, (int)T};
  float* part = reinterpret_cast<float*>(static_cast<char*>(workspace) + L.part);
  ShrinkArgs s{};
  s.g = g; s.x = static_cast<const uint16_t*>(x); s.ld = ldx; s.W = static_cast<const uint16_t*>(A); s.part = part;
  s.K = (int)H; s.R = (int)r; s.splits = splits_of(T, n, H, sms);
  ExpandArgs e{};
  e.g = g; e.part = part; e.scale = scale; e.W = static_cast<const uint16_t*>(B);
  e.base = static_cast<const uint16_t*>(base); e.ldb = ldbase; e.out = static_cast<uint16_t*>(y); e.back = s_reverse_scatter_idx;
  e.u = u; e.N = (int)N; e.R = (int)r; e.splits = s.splits;
  return by_rank(padded_rank(r), [&](auto k) {
    constexpr int RP = decltype(k)::value;
    const int rc1 = run_shrink<RP>(s, st);
    return rc1 ? rc1 : run_expand<RP>(e, sms, st);
  });
}

extern "C" int adapter_bwd(const void* dy, int64_t lddy, const void* x, int64_t ldx, const float* u, const void* A, const void* B,
                           const float* scale, const void* base, int64_t ldbase, const int32_t* expert_offsets,
                           const int32_t* x_gather_idx, const int32_t* s_reverse_scatter_idx, int64_t T, int64_t H, int64_t N,
                           int64_t n, int64_t r, void* dx, void* dA, void* dB, int accumulate, void* workspace,
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
  if (ldx < H || ldx % 8 || lddy < N || lddy % 8 || (base && (ldbase < H || ldbase % 8)))
    return fail(MOE_ERR_INVALID, "adapter_bwd: row stride too small or not a multiple of 8");
  if (base == dx && ldbase != H) return fail(MOE_ERR_INVALID, "adapter_bwd: dx may be the base only where its row stride is H");
  if (off16(dy) || off16(x) || off16(A) || off16(B) || off16(base) || off16(dx))
    return fail(MOE_ERR_INVALID, "adapter_bwd: tensors must be 16-byte aligned");
  if (off4(scale) || off4(expert_offsets) || off4(x_gather_idx) || off4(s_reverse_scatter_idx) || off4(u))
    return fail(MOE_ERR_INVALID, "adapter_bwd: metadata, scales and u must be 4-byte aligned");
  if (reinterpret_cast<uintptr_t>(workspace) & 255) return fail(MOE_ERR_INVALID, "adapter_bwd: workspace must be 256-byte aligned");
  const int sms = device_sm_count();
  const Layout L = layout(T, H, N, n, r, true, sms);
  if (workspace_bytes < L.total) return fail(MOE_ERR_INVALID, "adapter_bwd: workspace too small (%zu < %zu)", workspace_bytes, L.total);
  char* ws = static_cast<char*>(workspace);
  const Groups g{expert_offsets, x_gather_idx, (int)n, (int)T};
  ShrinkArgs s{};
  s.g = g; s.x = static_cast<const uint16_t*>(dy); s.ld = lddy; s.W = static_cast<const uint16_t*>(B);
  s.part = reinterpret_cast<float*>(ws + L.part);
  s.K = (int)N; s.R = (int)r; s.splits = splits_of(T, n, N, sms);
  ExpandArgs e{};
  e.g = g; e.part = s.part; e.scale = scale; e.W = static_cast<const uint16_t*>(A);
  e.base = static_cast<const uint16_t*>(base); e.ldb = ldbase; e.out = static_cast<uint16_t*>(dx); e.back = s_reverse_scatter_idx;
  e.v = reinterpret_cast<uint16_t*>(ws + L.v); e.u_in = u; e.su = reinterpret_cast<uint16_t*>(ws + L.su);
  e.N = (int)H; e.R = (int)r; e.splits = s.splits;
  GradArgs d{};
  d.g = g; d.R = (int)r; d.per = grad_rows(T); d.accumulate = accumulate;
  d.pr[0] = GradProblem{static_cast<const uint16_t*>(x), e.v, static_cast<uint16_t*>(dA), reinterpret_cast<float*>(ws + L.grad0), ldx,
                        (int)H, (int)cdiv(H, 128)};
  d.pr[1] = GradProblem{static_cast<const uint16_t*>(dy), e.su, static_cast<uint16_t*>(dB), reinterpret_cast<float*>(ws + L.grad1), lddy,
                        (int)N, (int)cdiv(N, 128)};
  return by_rank(padded_rank(r), [&](auto k) {
    constexpr int RP = decltype(k)::value;
    int rc1 = run_shrink<RP>(s, st);
    if (!rc1) rc1 = run_expand<RP>(e, sms, st);
    return rc1 ? rc1 : run_grad<RP>(d, st);
  });
}
