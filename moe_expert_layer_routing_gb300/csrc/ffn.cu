// The gated feed-forward block (a dense branch or shared expert beside the routed ones), forward and backward, BF16:
//
//   h = x W1 + b1 (gate and up columns as gate_up_layout says), a = act(gate) up, out = a W2 + b2
//   da = dout W2^T, dgate = da up act'(gate), dup = da act(gate), a recomputed from the saved h
//   dx = dh W1^T, dW1 = x^T dh, dW2 = a^T dout, db1 = sum_t dh, db2 = sum_t dout
//
// Two kernels forward (ffn_kernel.cuh, ffn_small.cu) and two backward, plus two small ones for the bias gradients.  All
// products accumulate in fp32; a and dh are rounded to bf16 between the kernels, since they are the next product's
// operands (the tensor core takes bf16; fp32 halves of them would double the products); out, dx, dW and h are rounded once.
#include <cuda.h>
#include <algorithm>
#include <atomic>

#include "ffn_kernel.cuh"
#include "ffn.h"

namespace moebwd {
namespace {

// ------------------------------------------------------------------------------------------
// column sums (bias gradients)
// ------------------------------------------------------------------------------------------
constexpr int kSumRows = 256;  // rows of a partial sum

// part[chunk, c] = sum of kSumRows rows of a bf16 matrix: 32 threads x 8 columns by 8 row groups, whole rows of 512 bytes
// a warp.  HBM-bound; the groups meet in shared memory in a fixed order.
__global__ void __launch_bounds__(256) column_part_kernel(const uint16_t* in, int64_t ld, int64_t T, int64_t H, float* part) {
  __shared__ float acc[8][256];
  const int cg = threadIdx.x & 31, rg = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 256 + 8 * cg;
  const int64_t r0 = (int64_t)blockIdx.y * kSumRows;
  pdl_wait();
  pdl_trigger();
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (c < H) {  // H is a multiple of 8
#pragma unroll 4
    for (int i = rg; i < kSumRows; i += 8) {
      if (r0 + i >= T) break;
      const uint4 v = *reinterpret_cast<const uint4*>(in + (r0 + i) * ld + c);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[2 * j] += bf_lo(w[j]);
        s[2 * j + 1] += bf_hi(w[j]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[rg][8 * cg + j] = s[j];
  __syncthreads();
  const int64_t col = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (col < H) {
    float t = 0.f;
#pragma unroll
    for (int g = 0; g < 8; ++g) t += acc[g][threadIdx.x];
    part[blockIdx.y * H + col] = t;
  }
}

// Rows up to which the bias gradient of the output is summed by column_reduce_kernel from the matrix itself: one launch less
// (333 rows: 40 us a backward pass without, 34 us with it; at 1024 rows a thread adds 32 numbers).
constexpr int64_t kDirectRows = 1024;

struct SumJob {
  const float* part;
  int64_t rows, cols;
  float* out;
  const uint16_t* in;  // a bf16 matrix of row stride ld in place of part, or null
  int64_t ld;
};
// out[c] (+)= sum over the rows of part[:, c]: 32 columns a block, 32 threads a column, fixed order
__global__ void __launch_bounds__(1024) column_reduce_kernel(SumJob j0, SumJob j1, int blocks0, int accumulate) {
  __shared__ float acc[32][33];
  const SumJob j = (int)blockIdx.x < blocks0 ? j0 : j1;
  const int64_t c = (int64_t)((int)blockIdx.x < blocks0 ? blockIdx.x : blockIdx.x - blocks0) * 32 + (threadIdx.x & 31);
  const int g = threadIdx.x >> 5;
  pdl_wait();
  pdl_trigger();
  float s = 0.f;
  if (c < j.cols) {
    if (j.in) {
#pragma unroll 8
      for (int64_t r = g; r < j.rows; r += 32) s += __uint_as_float((uint32_t)j.in[r * j.ld + c] << 16);
    } else {
#pragma unroll 4
      for (int64_t r = g; r < j.rows; r += 32) s += j.part[r * j.cols + c];
    }
  }
  acc[g][threadIdx.x & 31] = s;
  __syncthreads();
  if (g == 0 && c < j.cols) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += acc[i][threadIdx.x];
    j.out[c] = accumulate ? j.out[c] + t : t;
  }
}

// ------------------------------------------------------------------------------------------
// pair kernels
// ------------------------------------------------------------------------------------------
// Clusters of two that fit on the device at once, asked for once per device.  Without the kernel's shared-memory allowance the
// answer is none.
template <int EPI>
int pairs_resident() {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return device_sm_count() / 2;
  int n = known[dev].load(std::memory_order_relaxed);
  if (n > 0) return n;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(FfnCfg<EPI>::THREADS, 1, 1);
  cfg.dynamicSmemBytes = FfnCfg<EPI>::SMEM_BYTES;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(2, 1, 1);
  if (allow_smem(reinterpret_cast<const void*>(ffn_pair_kernel<EPI>), FfnCfg<EPI>::SMEM_BYTES) ||
      cudaOccupancyMaxActiveClusters(&n, ffn_pair_kernel<EPI>, &cfg) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    return std::max(1, device_sm_count() / 2);
  }
  known[dev].store(n, std::memory_order_relaxed);
  return n;
}

template <int EPI>
int launch_pair(FfnParams& P, cudaStream_t st) {
  using C = FfnCfg<EPI>;
  auto kern = ffn_pair_kernel<EPI>;
  const int rc = allow_smem(reinterpret_cast<const void*>(kern), C::SMEM_BYTES);
  if (rc) return rc;
  const int pairs = std::min(P.prob[P.nprob - 1].end, pairs_resident<EPI>());
  P.wait_ns = (uint64_t)option(MOE_OPT_WAIT_LIMIT_NS);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see launch_pdl
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)(2 * pairs), 1, 1);
  cfg.blockDim = dim3(C::THREADS, 1, 1);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = option(MOE_OPT_PDL) ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, P);
  count_launch();
  if (e != cudaSuccess) return cuda_check(e, "ffn pair launch");
  return cuda_check(cudaGetLastError(), "ffn pair launch");
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// operand [rows, K] (box 128 rows x 64) or [K, rows]: 64 x 128 in one copy where its columns are whole groups of 64, else
// two boxes of 64 x 64.  One producer thread issues every copy, and with three or four a k-block its issue bounds the
// kernel.
int mn_of(int64_t cols) { return cols % 64 ? 1 : 2; }
bool operand(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int64_t ld, bool mn) {
  if (mn && mn_of(cols) == 2) return make_tmap_groups(m, p, (uint64_t)rows, (uint64_t)cols, (uint64_t)ld * 2, 64, 2);
  return make_tmap_2d(m, p, 2, (uint64_t)rows, (uint64_t)cols, (uint64_t)ld * 2, mn ? 64 : 128, 64);
}
// a matrix moved in slabs of 128 rows x 64 columns
bool slabs(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int64_t ld) {
  return make_tmap_2d(m, p, 2, (uint64_t)rows, (uint64_t)cols, (uint64_t)ld * 2, 128, 64);
}
// the gate and up parts of a [rows, 2I] matrix: two of I columns, or one matrix twice
bool gate_up_slabs(CUtensorMap* m, const void* p, int64_t rows, int64_t I, bool interleaved) {
  const uint16_t* b = static_cast<const uint16_t*>(p);
  return interleaved ? slabs(m, b, rows, 2 * I, 2 * I) && slabs(m + 1, b, rows, 2 * I, 2 * I)
                     : slabs(m, b, rows, I, 2 * I) && slabs(m + 1, b + I, rows, I, 2 * I);
}

void add_problem(FfnParams& P, int64_t rows, int64_t cols, int64_t n_tiles, int64_t K, int a_mn, int b_mn) {
  FfnProblem& p = P.prob[P.nprob];
  const int64_t before = P.nprob ? P.prob[P.nprob - 1].end : 0;
  p.n_tiles = (int)n_tiles;
  p.nk = (int)cdiv(K, 64);
  p.M = (int)rows;
  p.N = (int)cols;
  p.a_mn = a_mn;
  p.b_mn = b_mn;
  p.end = (int)(before + cdiv(rows, 256) * n_tiles);
  ++P.nprob;
}

// Whether a projection of T rows runs on ffn_small_kernel (tiles as `plan` says) or on pair tiles.  Pair tiles: 7.5 us of
// launch, latency and epilogue, 0.36 a k-block in each wave of tiles (fitted like small_plan's estimate).  Measured on both
// sides of the border, both projections in a graph, H 2048, I 1024, h not kept: T 777 21 us against 29, T 2048 28 against 32,
// T 3000 54 against 51, T 4096 57 against 52; I 768: T 777 19 against 28, T 2048 26 against 30, T 4096 53 against 49.
bool use_small(const SmallPlan& plan, int64_t T, int64_t col_tiles, int64_t K, int sms) {
  const int64_t how = option(MOE_OPT_FFN_TILES);
  if (plan.token_tiles > 65535) return false;  // the grid's second dimension
  if (how) return how == 1;
  const int64_t waves = cdiv(cdiv(T, 256) * col_tiles, std::max(1, sms / 2));
  return plan.us < 7.5f + 0.36f * (float)(waves * cdiv(K, 64));
}

int check_common(const char* who, int64_t T, int64_t H, int64_t I, int glu, int layout) {
  if (T < 0 || H <= 0 || I <= 0) return fail(MOE_ERR_INVALID, "%s: bad sizes", who);
  if (H % 8 || I % 8) return fail(MOE_ERR_UNSUPPORTED, "%s: H and I must be multiples of 8", who);
  if (T > (1 << 30) || H > (1 << 24) || I > (1 << 24) ||
      cdiv(T, 256) * cdiv(std::max(2 * I, H), 256) > (1 << 30) || cdiv(H, 256) * cdiv(2 * I, 256) > (1 << 28))
    return fail(MOE_ERR_UNSUPPORTED, "%s: too large", who);
  if (glu != MOE_GLU_SWIGLU && glu != MOE_GLU_GEGLU) return fail(MOE_ERR_INVALID, "%s: bad glu", who);
  if (layout != MOE_GATE_UP_CONCAT && layout != MOE_GATE_UP_INTERLEAVED) return fail(MOE_ERR_INVALID, "%s: bad gate_up_layout", who);
  return MOE_OK;
}
bool off16(const void* p) { return reinterpret_cast<uintptr_t>(p) & 15; }

}  // namespace
}  // namespace moebwd

using namespace moebwd;

extern "C" size_t ffn_fwd_workspace_size(int64_t T, int64_t H, int64_t I) {
  if (T <= 0 || H <= 0 || I <= 0) return 0;
  return align_up((size_t)T * I * 2, 256);
}

extern "C" int ffn_fwd(const void* x, int64_t ldx, const void* W1, const void* b1, const void* W2, const void* b2, int64_t T,
                       int64_t H, int64_t I, int glu, int gate_up_layout, void* h, void* out, int32_t* status_dev,
                       void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  clear_error();
  int rc = check_common("ffn_fwd", T, H, I, glu, gate_up_layout);
  if (rc || T == 0) return rc;
  if (T == 1) ldx = H;  // a row alone: its stride is never used
  if (!x || !W1 || !W2 || !out || !workspace) return fail(MOE_ERR_INVALID, "ffn_fwd: null pointer");
  if (ldx < H || ldx % 8) return fail(MOE_ERR_INVALID, "ffn_fwd: row stride below H or not a multiple of 8");
  const void* al[] = {x, W1, W2, b1, b2, h, out};
  for (const void* p : al)
    if (off16(p)) return fail(MOE_ERR_INVALID, "ffn_fwd: tensors must be 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(status_dev) & 3) return fail(MOE_ERR_INVALID, "ffn_fwd: status must be 4-byte aligned");
  if (reinterpret_cast<uintptr_t>(workspace) & 255) return fail(MOE_ERR_INVALID, "ffn_fwd: workspace must be 256-byte aligned");
  const size_t need = ffn_fwd_workspace_size(T, H, I);
  if (workspace_bytes < need) return fail(MOE_ERR_INVALID, "ffn_fwd: workspace too small (%zu < %zu)", workspace_bytes, need);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint16_t* a = static_cast<uint16_t*>(workspace);
  const bool inter = gate_up_layout == MOE_GATE_UP_INTERLEAVED;
  const int sms = device_sm_count();

  const SmallPlan up = small_plan(T, I, H, 64, sms), down = small_plan(T, H, I, 128, sms);
  if (use_small(up, T, cdiv(I, 128), H, sms)) {
    FfnSmallArgs s{};
    s.W = W1; s.ldw = 2 * I; s.x = x; s.ldx = ldx; s.T = T; s.K = H; s.N = I;
    s.glu = glu; s.interleaved = inter; s.bias = static_cast<const uint16_t*>(b1);
    s.out = a; s.h = static_cast<uint16_t*>(h); s.status = status_dev;
    rc = launch_ffn_small(true, up, s, st);
  } else {
    alignas(64) FfnParams P{};
    add_problem(P, T, I, cdiv(I, 128), H, 0, mn_of(inter ? 2 * I : I));
    const uint16_t* w = static_cast<const uint16_t*>(W1);
    bool ok = operand(&P.map[0], x, T, H, ldx, false);
    ok = ok && (inter ? operand(&P.map[1], w, H, 2 * I, 2 * I, true) && operand(&P.map[2], w, H, 2 * I, 2 * I, true)
                      : operand(&P.map[1], w, H, I, 2 * I, true) && operand(&P.map[2], w + I, H, I, 2 * I, true));
    ok = ok && slabs(&P.map[3], a, T, I, I);
    ok = ok && (!h || gate_up_slabs(&P.map[4], h, T, I, inter));
    if (!ok) return MOE_ERR_INVALID;
    for (int i = h ? 6 : 4; i < kFfnMaps; ++i) P.map[i] = P.map[0];
    P.glu = glu; P.interleaved = inter; P.save = h != nullptr;
    P.b1 = static_cast<const uint16_t*>(b1);
    P.status = status_dev;
    rc = launch_pair<kFfnGlu>(P, st);
  }
  if (rc) return rc;

  if (use_small(down, T, cdiv(H, 256), I, sms)) {
    FfnSmallArgs s{};
    s.W = W2; s.ldw = H; s.x = a; s.ldx = I; s.T = T; s.K = I; s.N = H;
    s.early = 1;  // the first projection's kernel lets this one start once all that went before is complete
    s.bias = static_cast<const uint16_t*>(b2);
    s.out = static_cast<uint16_t*>(out); s.status = status_dev;
    return launch_ffn_small(false, down, s, st);
  }
  alignas(64) FfnParams P{};
  add_problem(P, T, H, cdiv(H, 256), I, 0, mn_of(H));
  P.prob[0].bias = static_cast<const uint16_t*>(b2);
  if (!operand(&P.map[0], a, T, I, I, false) || !operand(&P.map[1], W2, I, H, H, true) || !slabs(&P.map[2], out, T, H, H))
    return MOE_ERR_INVALID;
  for (int i = 3; i < kFfnMaps; ++i) P.map[i] = P.map[0];
  P.status = status_dev;
  return launch_pair<kFfnStore>(P, st);
}

namespace moebwd {
namespace {
struct BwdLayout {
  size_t a, dh, counter, part1, part2, total;
};
BwdLayout bwd_layout(int64_t T, int64_t H, int64_t I, bool bias) {
  BwdLayout L{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes, 256);
    return at;
  };
  L.a = take((size_t)T * I * 2);
  L.dh = take((size_t)T * I * 4);
  L.counter = take(4);
  L.part1 = take(bias ? (size_t)cdiv(T, 128) * 4 * 2 * I * 4 : 0);
  L.part2 = take(bias && T > kDirectRows ? (size_t)cdiv(T, kSumRows) * H * 4 : 0);
  L.total = off;
  return L;
}
}  // namespace
}  // namespace moebwd

extern "C" size_t ffn_bwd_workspace_size(int64_t T, int64_t H, int64_t I, int bias) {
  if (T <= 0 || H <= 0 || I <= 0) return 0;
  return bwd_layout(T, H, I, bias != 0).total;
}

extern "C" int ffn_bwd(const void* dout, int64_t lddout, const void* x, int64_t ldx, const void* h, const void* W1,
                       const void* W2, int64_t T, int64_t H, int64_t I, int glu, int gate_up_layout, void* dx, void* dW1,
                       void* dW2, float* db1, float* db2, int accumulate, int32_t* status_dev, void* workspace,
                       size_t workspace_bytes, moe_stream_t stream) {
  clear_error();
  int rc = check_common("ffn_bwd", T, H, I, glu, gate_up_layout);
  if (rc) return rc;
  if (accumulate != 0 && accumulate != 1) return fail(MOE_ERR_INVALID, "ffn_bwd: accumulate must be 0 or 1");
  if (!dW1 || !dW2) return fail(MOE_ERR_INVALID, "ffn_bwd: null pointer");
  if ((db1 == nullptr) != (db2 == nullptr)) return fail(MOE_ERR_INVALID, "ffn_bwd: db1 and db2 go together");
  if ((reinterpret_cast<uintptr_t>(db1) | reinterpret_cast<uintptr_t>(db2) | reinterpret_cast<uintptr_t>(status_dev)) & 3)
    return fail(MOE_ERR_INVALID, "ffn_bwd: db1, db2 and status must be 4-byte aligned");
  if (off16(dW1) || off16(dW2)) return fail(MOE_ERR_INVALID, "ffn_bwd: tensors must be 16-byte aligned");
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0) {  // empty sums
    if (accumulate) return MOE_OK;
    if ((rc = cuda_check(cudaMemsetAsync(dW1, 0, (size_t)H * I * 4, st), "memset dW1")) ||
        (rc = cuda_check(cudaMemsetAsync(dW2, 0, (size_t)H * I * 2, st), "memset dW2")))
      return rc;
    if (!db1) return MOE_OK;
    if ((rc = cuda_check(cudaMemsetAsync(db1, 0, (size_t)I * 8, st), "memset db1"))) return rc;
    return cuda_check(cudaMemsetAsync(db2, 0, (size_t)H * 4, st), "memset db2");
  }
  if (!dout || !x || !h || !W1 || !W2 || !dx || !workspace) return fail(MOE_ERR_INVALID, "ffn_bwd: null pointer");
  if (T == 1) ldx = lddout = H;  // as in ffn_fwd
  if (ldx < H || ldx % 8 || lddout < H || lddout % 8)
    return fail(MOE_ERR_INVALID, "ffn_bwd: row stride below H or not a multiple of 8");
  const void* al[] = {dout, x, h, W1, W2, dx};
  for (const void* p : al)
    if (off16(p)) return fail(MOE_ERR_INVALID, "ffn_bwd: tensors must be 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(workspace) & 255) return fail(MOE_ERR_INVALID, "ffn_bwd: workspace must be 256-byte aligned");
  const BwdLayout L = bwd_layout(T, H, I, db1 != nullptr);
  if (workspace_bytes < L.total) return fail(MOE_ERR_INVALID, "ffn_bwd: workspace too small (%zu < %zu)", workspace_bytes, L.total);
  char* ws = static_cast<char*>(workspace);
  void* a = ws + L.a;
  void* dh = ws + L.dh;
  int32_t* counter = reinterpret_cast<int32_t*>(ws + L.counter);
  float* part1 = db1 ? reinterpret_cast<float*>(ws + L.part1) : nullptr;
  float* part2 = db1 ? reinterpret_cast<float*>(ws + L.part2) : nullptr;
  const bool inter = gate_up_layout == MOE_GATE_UP_INTERLEAVED;

  const bool direct = T <= kDirectRows;
  if (db2 && !direct) {
    if (cdiv(T, kSumRows) > 65535) return fail(MOE_ERR_UNSUPPORTED, "ffn_bwd: too many rows for the bias gradients");
    rc = launch_pdl(column_part_kernel, dim3((unsigned)cdiv(H, 256), (unsigned)cdiv(T, kSumRows)), dim3(256), 0, st, "column sums",
                    static_cast<const uint16_t*>(dout), lddout, T, H, part2);
    if (rc) return rc;
  }
  {
    alignas(64) FfnParams P{};
    // A tile's epilogue (two activations' derivatives a number) takes 13 us with 256 features: narrower tiles, whose product
    // is as wide, while all of them run at once (333 x 520 x 264: 34 us, now 28).
    P.width = 256;
    while (P.width > 64 && cdiv(T, 256) * cdiv(I, P.width / 2) <= pairs_resident<kFfnDGlu>()) P.width /= 2;
    add_problem(P, T, I, cdiv(I, P.width), H, 0, 0);
    if (!operand(&P.map[0], dout, T, H, lddout, false) || !operand(&P.map[1], W2, I, H, H, false) ||
        !gate_up_slabs(&P.map[2], h, T, I, inter) || !gate_up_slabs(&P.map[4], dh, T, I, inter))
      return MOE_ERR_INVALID;
    for (int i = 6; i < kFfnMaps; ++i) P.map[i] = P.map[0];
    P.glu = glu; P.interleaved = inter;
    P.a_out = static_cast<uint16_t*>(a);
    P.db1_part = part1;
    P.zero_counter = counter;
    P.status = status_dev;
    if ((rc = launch_pair<kFfnDGlu>(P, st))) return rc;
  }
  {
    // dW1 = x^T dh and dW2 = a^T dout over the tokens, dx = dh W1^T over the features: the longer contraction first
    alignas(64) FfnParams P{};
    auto weights = [&]() {
      const int i = 3 * P.nprob;
      add_problem(P, H, 2 * I, cdiv(2 * I, 256), T, mn_of(H), mn_of(2 * I));
      P.prob[P.nprob - 1].accumulate = accumulate;
      bool ok = operand(&P.map[i], x, T, H, ldx, true) && operand(&P.map[i + 1], dh, T, 2 * I, 2 * I, true) &&
                slabs(&P.map[i + 2], dW1, H, 2 * I, 2 * I);
      add_problem(P, I, H, cdiv(H, 256), T, mn_of(I), mn_of(H));
      P.prob[P.nprob - 1].accumulate = accumulate;
      return ok && operand(&P.map[i + 3], a, T, I, I, true) && operand(&P.map[i + 4], dout, T, H, lddout, true) &&
             slabs(&P.map[i + 5], dW2, I, H, H);
    };
    auto rows = [&]() {
      const int i = 3 * P.nprob;
      add_problem(P, T, H, cdiv(H, 256), 2 * I, 0, 0);
      return operand(&P.map[i], dh, T, 2 * I, 2 * I, false) && operand(&P.map[i + 1], W1, H, 2 * I, 2 * I, false) &&
             slabs(&P.map[i + 2], dx, T, H, H);
    };
    if (!(T >= 2 * I ? weights() && rows() : rows() && weights())) return MOE_ERR_INVALID;
    P.tile_counter = counter;
    P.status = status_dev;
    if ((rc = launch_pair<kFfnStore>(P, st))) return rc;
  }
  if (!db1) return MOE_OK;
  const SumJob j1{part1, cdiv(T, 128) * 4, 2 * I, db1, nullptr, 0};
  const SumJob j2{part2, direct ? T : cdiv(T, kSumRows), H, db2, direct ? static_cast<const uint16_t*>(dout) : nullptr, lddout};
  const int blocks0 = (int)cdiv(2 * I, 32);
  return launch_pdl(column_reduce_kernel, dim3((unsigned)(blocks0 + cdiv(H, 32))), dim3(1024), 0, st, "bias gradients", j1, j2,
                    blocks0, accumulate);
}
