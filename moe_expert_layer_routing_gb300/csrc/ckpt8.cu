// Gated activation of the forward with the 8-bit gate/up checkpoint, and the checkpoint read back.
//
//   a = act(g) u (times the row's routing score when given), g and u the gate and up pre-activations
//   checkpoint: per feature, groups of 32 consecutive slots of the block layout share one power of two;
//     byte = max(1, exponent field of the group's largest magnitude - 6)      (E8M0, value 2^(byte - 127))
//     code = round(v 2^(127 - byte)), ties to even, clamped to +-127          (int8)
//   so a group's largest code is 64 .. 127, and a value (bf16: 8 significant bits, at most 127.5 steps) is off by at
//   most half a step, 1/128 of the group's largest magnitude.  A group with a NaN or an infinity gets byte 255 and reads as NaN.
//   Every value code 2^(byte - 127) has 7 significant bits: bf16 holds it exactly.
//
// Bound by HBM: at 131072 rows x I = 1024 the forward moves 1.08 GB (159 us at the measured copy rate) and the read-back
// 0.81 GB (120 us).  Measured 177 us (6.1 TB/s) and 119 us (6.8 TB/s); GeGLU's erff takes the forward to 248 us, bound by
// its arithmetic.  In moe_bwd the codes take 33/64 of the bf16 checkpoint's bytes; what their decoding costs G1 stands at
// its epilogue (gemm_kernel.cuh), and the whole pass takes 1 to 3% longer (BF16, 64 experts: 2.76 -> 2.79 to 2.84 ms;
// MXFP8, 128 experts: 3.33 -> 3.37 ms).
//
// Layout: codes int8 [N, 2, I, B], the bf16 checkpoint's; scale bytes [N, 2, B/128, I/32, 4, 32], so that the
// 32 features x 128 rows of a GEMM epilogue's chunk have their bytes in 128 consecutive ones, those of one
// 32-row quarter side by side.
//
// A CTA takes 128 slots (one GEMM tile's rows) and 64 features: the rows of h come into shared memory by
// 16-byte asynchronous copies (128 consecutive bytes of gate and of up per row), the activation is computed
// along rows (16-byte stores), the codes along columns: a thread owns one 32-bit word column, two values of
// each of 32 rows, so its two groups' maxima and codes need no exchange, and consecutive lanes read
// consecutive words.
#include <cuda_runtime.h>

#include <algorithm>
#include <initializer_list>

#include "moebwd_internal.h"
#include "mx_device.cuh"
#include "ptx.cuh"

namespace moebwd {

constexpr int kGluThreads = 256;
constexpr int kGluFeat = 64;  // features per CTA
constexpr int kGluRows = 128;

struct GluArgs {
  const uint16_t* h;  // [rows, 2I]
  int64_t ldh;
  uint16_t* a;        // [rows, I]
  int8_t* q;          // [N, 2, I, B] or null
  uint8_t* sf;        // [N, 2, B/128, I/32, 4, 32]
  const float* s;     // routing scores or null
  const int32_t* s_scatter_idx;
  const int32_t *expert_offsets, *block_offsets, *block_to_expert;
  int64_t rows;       // rows of h; no row at or past it is touched
  int64_t slots;      // T*K: scores
  int64_t items;      // 128-slot tiles x 64-feature chunks
  int I, B, E, glu, interleaved, tpb_shift;  // B = 128 << tpb_shift
};

// Rows [r0, r0 + n) of the grouped order that lie in the 128 slots of tile `tile`; n <= 0: none.
__device__ __forceinline__ void glu_tile_rows(const int32_t* eo, const int32_t* bo, const int32_t* b2e, int E, int B,
                                              int tpb_shift, int64_t rows, int tile, int64_t& r0, int& n) {
  const int blk = tile >> tpb_shift;
  const int e = b2e[blk];
  n = 0;
  if (e < 0 || e >= E) return;
  const int64_t j0 = (int64_t)(blk - bo[e]) * B + (tile - (blk << tpb_shift)) * kGluRows;
  r0 = eo[e] + j0;
  const int64_t r1 = min((int64_t)eo[e + 1], rows);
  if (j0 < 0 || r0 < 0) return;
  n = (int)max((int64_t)0, min((int64_t)kGluRows, r1 - r0));
}

// Scale byte of feature f, 32-slot group g of 128-slot tile tb of half `bu` (2 block + gate|up).
__device__ __forceinline__ int64_t sf_offset(int64_t bu, int tpb_shift, int tb, int I, int f, int g) {
  return ((((bu << tpb_shift) + tb) * (I >> 5) + (f >> 5)) * 4 + g) * 32 + (f & 31);
}

// a = act(g) u scaled by sv, for two (gate, up) pairs: SiLU(g) = g / (1 + e^-g) in paired arithmetic, with the
// exponential as 2^(-g log2 e) and the approximate reciprocal (2^-22 of the value each, and |g| 2^-24 from rounding the
// exponent: far below the rounding to bf16 that follows; one value at a time 184 instead of 177 us); or GELU(g) = g Phi(g).
__device__ __forceinline__ uint32_t glu_pair(uint32_t gw, uint32_t uw, float sv, int glu) {
  const uint64_t g = f2_pack(__uint_as_float(gw << 16), __uint_as_float(gw & 0xffff0000u));
  const uint64_t u = f2_pack(__uint_as_float(uw << 16), __uint_as_float(uw & 0xffff0000u));
  uint64_t act;
  float x0, x1, y0, y1;
  if (glu == MOE_GLU_GEGLU) {
    f2_unpack(g, x0, x1);
    act = f2_pack(x0 * (0.5f * (1.f + erff(x0 * 0.70710678118654752f))), x1 * (0.5f * (1.f + erff(x1 * 0.70710678118654752f))));
  } else {
    f2_unpack(f2_mul(g, f2_splat(-1.4426950408889634f)), x0, x1);
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y0) : "f"(x0));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y1) : "f"(x1));
    f2_unpack(f2_add(f2_pack(y0, y1), f2_splat(1.f)), x0, x1);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y0) : "f"(x0));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y1) : "f"(x1));
    act = f2_mul(g, f2_pack(y0, y1));
  }
  f2_unpack(f2_mul(f2_mul(act, u), f2_splat(sv)), x0, x1);
  return pack_bf16x2(x0, x1);
}

// Per half, max |x| over 32 words of two bf16 values each; a NaN or an infinity gives an exponent field of 255.
__device__ __forceinline__ uint32_t absmax32_nan(const uint32_t (&w)[32]) {
  uint32_t t[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(t[i]) : "r"(w[i]), "r"(w[i + 16]));
#pragma unroll
  for (int n = 8; n > 0; n >>= 1)
#pragma unroll
    for (int i = 0; i < n; ++i) asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(t[i]) : "r"(t[i]), "r"(t[i + n]));
  return t[0] & 0x7FFF7FFFu;
}

// Codes of the low (half 0) or high values of 32 words.  Adding 1.5 * 2^23 rounds to an integer (ties to even) in
// the low mantissa bits, two's complement in the low byte.
template <bool CLAMP>
__device__ __forceinline__ void codes32(const uint32_t (&v)[32], int half, uint64_t inv, uint32_t (&w)[8]) {
  const uint64_t magic = f2_splat(12582912.f);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const uint32_t x0 = v[4 * k + i], x1 = v[4 * k + i + 1];
      uint64_t f = f2_mul(f2_pack(__uint_as_float(half ? x0 & 0xffff0000u : x0 << 16),
                                  __uint_as_float(half ? x1 & 0xffff0000u : x1 << 16)), inv);
      if constexpr (CLAMP) {
        float a, c;
        f2_unpack(f, a, c);
        f = f2_pack(fminf(fmaxf(a, -127.f), 127.f), fminf(fmaxf(c, -127.f), 127.f));
      }
      float a, c;
      f2_unpack(f2_add(f, magic), a, c);
      b[i] = __float_as_uint(a);
      b[i + 1] = __float_as_uint(c);
    }
    w[k] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
  }
}

__device__ __forceinline__ void glu_tile(const GluArgs& p, int t, int f0, int64_t r0, int n,
                                         const uint32_t (*tile)[kGluFeat]) {
  // a: eight features of a row at a time
  for (int i = threadIdx.x; i < n * 8; i += kGluThreads) {
    const int r = i >> 3, c = i & 7;
    uint32_t g[4], u[4];
    if (p.interleaved) {
      const uint4 w0 = *reinterpret_cast<const uint4*>(&tile[r][c * 8]), w1 = *reinterpret_cast<const uint4*>(&tile[r][c * 8 + 4]);
      g[0] = __byte_perm(w0.x, w0.y, 0x5410);
      u[0] = __byte_perm(w0.x, w0.y, 0x7632);
      g[1] = __byte_perm(w0.z, w0.w, 0x5410);
      u[1] = __byte_perm(w0.z, w0.w, 0x7632);
      g[2] = __byte_perm(w1.x, w1.y, 0x5410);
      u[2] = __byte_perm(w1.x, w1.y, 0x7632);
      g[3] = __byte_perm(w1.z, w1.w, 0x5410);
      u[3] = __byte_perm(w1.z, w1.w, 0x7632);
    } else {
      const uint4 w0 = *reinterpret_cast<const uint4*>(&tile[r][c * 4]), w1 = *reinterpret_cast<const uint4*>(&tile[r][32 + c * 4]);
      g[0] = w0.x; g[1] = w0.y; g[2] = w0.z; g[3] = w0.w;
      u[0] = w1.x; u[1] = w1.y; u[2] = w1.z; u[3] = w1.w;
    }
    float sv = 1.f;
    if (p.s) {
      const int f = p.s_scatter_idx[r0 + r];
      sv = f >= 0 && f < p.slots ? p.s[f] : 0.f;
    }
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = glu_pair(g[k], u[k], sv, p.glu);
    *reinterpret_cast<uint4*>(p.a + (r0 + r) * (int64_t)p.I + f0 + c * 8) = make_uint4(o[0], o[1], o[2], o[3]);
  }
  if (!p.q) return;
  // codes: word column wc of the 32 rows of group gr
  const int wc = threadIdx.x & 63, gr = threadIdx.x >> 6;
  uint32_t v[32];
#pragma unroll
  for (int k = 0; k < 32; ++k) v[k] = tile[32 * gr + k][wc];
  const uint32_t am = absmax32_nan(v);
  const int64_t blk = t >> p.tpb_shift;
  const int tb = t & ((1 << p.tpb_shift) - 1);
  uint32_t bytes = 0;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int exponent = (half ? am >> 23 : am >> 7) & 0xff;
    const int byte = exponent == 255 ? 255 : max(1, exponent - 6);
    bytes |= (uint32_t)byte << (8 * half);
    // 2^(127 - byte); byte <= 248 for finite values
    const uint64_t inv = f2_splat(__uint_as_float((uint32_t)(254 - min(byte, 253)) << 23));
    uint32_t w[8];
    // a bf16 of 8 significant bits times 2^(127 - byte) is at most 127.5 in magnitude, and only that rounds to 128
    if (((half ? am >> 16 : am) & 0x7f) != 0x7f)
      codes32<false>(v, half, inv, w);
    else
      codes32<true>(v, half, inv, w);
    const int f = p.interleaved ? f0 + wc : f0 + 2 * (wc & 31) + half;  // feature
    const int up = p.interleaved ? half : wc >> 5;
    int8_t* dst = p.q + ((blk * 2 + up) * (int64_t)p.I + f) * p.B + tb * kGluRows + 32 * gr;
    st_global_32b_or_halves(dst, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
    if (p.interleaved) p.sf[sf_offset(blk * 2 + up, p.tpb_shift, tb, p.I, f, gr)] = (uint8_t)byte;
  }
  if (!p.interleaved)  // two features side by side
    *reinterpret_cast<uint16_t*>(p.sf + sf_offset(blk * 2 + (wc >> 5), p.tpb_shift, tb, p.I, f0 + 2 * (wc & 31), gr)) =
        (uint16_t)bytes;
}

constexpr int kGluBlocks = 3;  // resident blocks: two 32 KB tiles each

// Persistent: block i takes items i, i + grid, ... (an item is 64 features of a 128-slot tile, features fastest);
// the next item's rows are on their way while this one is computed.
__global__ void __launch_bounds__(kGluThreads, kGluBlocks) glu_fwd_kernel(const GluArgs p) {
  extern __shared__ __align__(16) uint32_t tiles[];  // two tiles [128][64] of words: 32 gate pairs | 32 up pairs, or 64 (gate, up)
  pdl_wait();
  const uint32_t chunks = p.I / kGluFeat;
  struct Item {
    int64_t r0;
    int t, f0, n;
  };
  auto fetch = [&](int64_t item, uint32_t* tile) {
    Item it{};
    if (item < p.items) {
      it.t = (int)((uint32_t)item / chunks);
      it.f0 = (int)((uint32_t)item - it.t * chunks) * kGluFeat;
      glu_tile_rows(p.expert_offsets, p.block_offsets, p.block_to_expert, p.E, p.B, p.tpb_shift, p.rows, it.t, it.r0,
                    it.n);
      if (it.n > 0) {
        // 16 pieces of 16 bytes per row; rows past the expert's last are zeros
        const int c = threadIdx.x & 15;
        const int col = p.interleaved ? 2 * it.f0 + c * 8 : c < 8 ? it.f0 + c * 8 : p.I + it.f0 + (c - 8) * 8;
        const uint16_t* src = p.h + it.r0 * p.ldh + col;
#pragma unroll
        for (int k = 0; k < kGluRows / 16; ++k) {
          const int r = k * 16 + (threadIdx.x >> 4);
          cp_async_16_zfill(smem_u32(tile + r * kGluFeat + c * 4), src + (r < it.n ? r : 0) * p.ldh, r < it.n ? 16 : 0);
        }
      }
    }
    cp_async_commit();
    return it;
  };
  int buf = 0;
  Item now = fetch(blockIdx.x, tiles);
  for (int64_t item = blockIdx.x; item < p.items; item += gridDim.x, buf ^= 1) {
    const Item next = fetch(item + gridDim.x, tiles + (buf ^ 1) * (kGluRows * kGluFeat));
    cp_async_wait<1>();
    __syncthreads();
    if (now.n > 0) glu_tile(p, now.t, now.f0, now.r0, now.n, reinterpret_cast<const uint32_t(*)[kGluFeat]>(tiles + buf * (kGluRows * kGluFeat)));
    __syncthreads();  // the buffer is read; it is filled again next time round
    now = next;
  }
  pdl_trigger();  // not earlier: the next kernel's blocks would take the place of this one's late ones
}

struct UnpackArgs {
  const int8_t* q;
  const uint8_t* sf;
  uint16_t* h;
  int64_t ldh, rows;
  const int32_t *expert_offsets, *block_offsets, *block_to_expert;
  int I, B, E, interleaved, tpb_shift;  // B = 128 << tpb_shift
};

// The checkpoint's values as rows [rows, 2I] in the grouped order.  The tile's 128 columns (64 gate | 64 up, or 64
// pairs) lie in shared memory as 128-byte rows of codes whose 16-byte pieces are swizzled by the column quad, so
// that a warp's four word loads (8 column quads x 4 slot quads) meet no bank twice; a thread turns 4 columns x 4
// slots and writes 8 bytes of each of four rows.
__global__ void __launch_bounds__(kGluThreads) ckpt8_unpack_kernel(const UnpackArgs p) {
  constexpr int COLS = 2 * kGluFeat;
  __shared__ __align__(16) uint32_t code[COLS][kGluRows / 4];
  __shared__ __align__(16) float scale[4][COLS];
  pdl_wait();  // (no early trigger: blocks of a persistent successor waiting beside this kernel's last ones cost 3%)
  const uint32_t chunks = p.I / kGluFeat;
  const int t = (int)(blockIdx.x / chunks);
  const int f0 = (int)(blockIdx.x - t * chunks) * kGluFeat;
  int64_t r0 = 0;
  int n;
  glu_tile_rows(p.expert_offsets, p.block_offsets, p.block_to_expert, p.E, p.B, p.tpb_shift, p.rows, t, r0, n);
  if (n == 0) return;
  const int64_t blk = t >> p.tpb_shift;
  const int tb = t & ((1 << p.tpb_shift) - 1);
  // column c of the tile: feature and half
  auto feature = [&](int c) { return f0 + (p.interleaved ? c >> 1 : c & (kGluFeat - 1)); };
  auto half = [&](int c) { return blk * 2 + (p.interleaved ? c & 1 : c / kGluFeat); };
  for (int i = threadIdx.x; i < COLS * 8; i += kGluThreads) {
    const int c = i >> 3, piece = i & 7;
    cp_async_16(smem_u32(&code[c][(piece ^ ((c >> 2) & 7)) * 4]),
                p.q + (half(c) * (int64_t)p.I + feature(c)) * p.B + tb * kGluRows + piece * 16);
  }
  cp_async_commit();
  for (int i = threadIdx.x; i < COLS * 4; i += kGluThreads) {
    const int c = i & (COLS - 1), g = i / COLS;
    const uint32_t byte = p.sf[sf_offset(half(c), p.tpb_shift, tb, p.I, feature(c), g)];
    scale[g][c] = __uint_as_float(byte == 255 ? 0x7fc00000u : byte << 23);
  }
  cp_async_wait<0>();
  __syncthreads();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    // warp w: column quads 8 (w & 3) .. + 7, slot quads 16 (w >> 2) + 4 k .. + 3
    const int cq = 8 * (w & 3) + (lane & 7), sq = 16 * (w >> 2) + 4 * k + (lane >> 3);
    if (4 * sq >= n) continue;
    const int c = 4 * cq;
    const float4 sc4 = *reinterpret_cast<const float4*>(&scale[sq >> 3][c]);
    const float sc[4] = {sc4.x, sc4.y, sc4.z, sc4.w};
    float x[4][4];  // [column][slot]
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t v = code[c + j][((sq >> 2) ^ (cq & 7)) * 4 + (sq & 3)] ^ 0x80808080u;
#pragma unroll
      for (int i = 0; i < 4; ++i)  // 2^23 + 128 + code
        x[j][i] = (__uint_as_float(__byte_perm(v, 0x4B000000u, 0x7650 + i)) - 8388736.f) * sc[j];
    }
    const int col = p.interleaved ? 2 * f0 + c : c < kGluFeat ? f0 + c : p.I + f0 + c - kGluFeat;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (4 * sq + i < n)
        *reinterpret_cast<uint2*>(p.h + (r0 + 4 * sq + i) * p.ldh + col) =
            make_uint2(pack_bf16x2(x[0][i], x[1][i]), pack_bf16x2(x[2][i], x[3][i]));
  }
}

static int tile_shift(int block_size) { return block_size == 128 ? 0 : block_size == 256 ? 1 : block_size == 512 ? 2 : 3; }

static int ckpt8_check(const char* who, int64_t rows, int I, int E, int block_size, int64_t num_blocks, int gate_up_layout) {
  if (rows < 0 || num_blocks < 0 || I <= 0 || E <= 0) return fail(MOE_ERR_INVALID, "%s: bad sizes", who);
  if (I % kGluFeat) return fail(MOE_ERR_UNSUPPORTED, "%s: I must be a multiple of %d", who, kGluFeat);
  if (E > kMaxExperts) return fail(MOE_ERR_UNSUPPORTED, "%s: E above %d", who, kMaxExperts);
  if (block_size != 128 && block_size != 256 && block_size != 512 && block_size != 1024)
    return fail(MOE_ERR_UNSUPPORTED, "%s: block_size must be 128, 256, 512 or 1024", who);
  if (gate_up_layout != MOE_GATE_UP_CONCAT && gate_up_layout != MOE_GATE_UP_INTERLEAVED)
    return fail(MOE_ERR_INVALID, "%s: bad gate_up_layout", who);
  if (num_blocks > INT32_MAX || num_blocks * (block_size / kGluRows) * (I / kGluFeat) > INT32_MAX)
    return fail(MOE_ERR_UNSUPPORTED, "%s: too many tiles", who);
  return MOE_OK;
}

// Routing metadata and scores: single 4-byte elements.
static int ckpt8_aligned(const char* who, std::initializer_list<const void*> meta) {
  for (const void* p : meta)
    if (reinterpret_cast<uintptr_t>(p) & 3)
      return fail(MOE_ERR_INVALID, "%s: routing metadata and scores must be 4-byte aligned", who);
  return MOE_OK;
}

}  // namespace moebwd

using namespace moebwd;

extern "C" int moe_glu_fwd(const void* h, int64_t ldh, int64_t rows, int I, int E, int block_size, int64_t num_blocks,
                           int glu, int gate_up_layout, const int32_t* expert_offsets, const int32_t* block_offsets,
                           const int32_t* block_to_expert, const float* s, const int32_t* s_scatter_idx,
                           int64_t num_slots, void* a, int8_t* ckpt_q, uint8_t* ckpt_sf, moe_stream_t stream) {
  clear_error();
  int rc = ckpt8_check("moe_glu_fwd", rows, I, E, block_size, num_blocks, gate_up_layout);
  if (rc) return rc;
  if (glu != MOE_GLU_SWIGLU && glu != MOE_GLU_GEGLU) return fail(MOE_ERR_INVALID, "moe_glu_fwd: bad glu");
  if ((ckpt_q == nullptr) != (ckpt_sf == nullptr))
    return fail(MOE_ERR_INVALID, "moe_glu_fwd: ckpt_q and ckpt_sf come together");
  if ((s == nullptr) != (s_scatter_idx == nullptr))
    return fail(MOE_ERR_INVALID, "moe_glu_fwd: s and s_scatter_idx come together");
  if (rows == 0 || num_blocks == 0) return MOE_OK;
  if (!h || !a || !expert_offsets || !block_offsets || !block_to_expert)
    return fail(MOE_ERR_INVALID, "moe_glu_fwd: null pointer");
  if (ldh < 2 * (int64_t)I || ldh % 8) return fail(MOE_ERR_INVALID, "moe_glu_fwd: row stride of h must be a multiple of 8, at least 2I");
  for (const void* q : {h, static_cast<const void*>(a), static_cast<const void*>(ckpt_q), static_cast<const void*>(ckpt_sf)})
    if (reinterpret_cast<uintptr_t>(q) & 15) return fail(MOE_ERR_INVALID, "moe_glu_fwd: tensors must be 16-byte aligned");
  if ((rc = ckpt8_aligned("moe_glu_fwd", {expert_offsets, block_offsets, block_to_expert, s, s_scatter_idx}))) return rc;
  GluArgs p{};
  p.h = static_cast<const uint16_t*>(h);
  p.ldh = ldh;
  p.a = static_cast<uint16_t*>(a);
  p.q = ckpt_q;
  p.sf = ckpt_sf;
  p.s = s;
  p.s_scatter_idx = s_scatter_idx;
  p.slots = num_slots;
  p.expert_offsets = expert_offsets;
  p.block_offsets = block_offsets;
  p.block_to_expert = block_to_expert;
  p.rows = rows;
  p.I = I;
  p.B = block_size;
  p.E = E;
  p.glu = glu;
  p.interleaved = gate_up_layout == MOE_GATE_UP_INTERLEAVED;
  p.tpb_shift = tile_shift(block_size);
  p.items = (num_blocks << p.tpb_shift) * (I / kGluFeat);
  constexpr size_t smem = 2 * sizeof(uint32_t) * kGluRows * kGluFeat;
  return launch_pdl(glu_fwd_kernel, dim3((unsigned)std::min<int64_t>(p.items, kGluBlocks * device_sm_count())),
                    dim3(kGluThreads), smem, reinterpret_cast<cudaStream_t>(stream), "glu_fwd", p);
}

extern "C" int moe_ckpt8_unpack(const int8_t* ckpt_q, const uint8_t* ckpt_sf, int64_t rows, int I, int E, int block_size,
                                int64_t num_blocks, int gate_up_layout, const int32_t* expert_offsets,
                                const int32_t* block_offsets, const int32_t* block_to_expert, void* h, int64_t ldh,
                                moe_stream_t stream) {
  clear_error();
  int rc = ckpt8_check("moe_ckpt8_unpack", rows, I, E, block_size, num_blocks, gate_up_layout);
  if (rc) return rc;
  if (rows == 0 || num_blocks == 0) return MOE_OK;
  if (!ckpt_q || !ckpt_sf || !h || !expert_offsets || !block_offsets || !block_to_expert)
    return fail(MOE_ERR_INVALID, "moe_ckpt8_unpack: null pointer");
  if (ldh < 2 * (int64_t)I || ldh % 8) return fail(MOE_ERR_INVALID, "moe_ckpt8_unpack: row stride of h must be a multiple of 8, at least 2I");
  for (const void* q : {static_cast<const void*>(ckpt_q), static_cast<const void*>(ckpt_sf), static_cast<const void*>(h)})
    if (reinterpret_cast<uintptr_t>(q) & 15) return fail(MOE_ERR_INVALID, "moe_ckpt8_unpack: tensors must be 16-byte aligned");
  if ((rc = ckpt8_aligned("moe_ckpt8_unpack", {expert_offsets, block_offsets, block_to_expert}))) return rc;
  UnpackArgs p{ckpt_q, ckpt_sf, static_cast<uint16_t*>(h), ldh, rows, expert_offsets, block_offsets, block_to_expert, I,
               block_size, E, gate_up_layout == MOE_GATE_UP_INTERLEAVED, tile_shift(block_size)};
  const int64_t grid = (num_blocks << p.tpb_shift) * (I / kGluFeat);
  return launch_pdl(ckpt8_unpack_kernel, dim3((unsigned)grid), dim3(kGluThreads), 0,
                    reinterpret_cast<cudaStream_t>(stream), "ckpt8_unpack", p);
}
