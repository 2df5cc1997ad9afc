// BF16 instantiations of the tcgen05 grouped GEMM (kind::f16, FP32 accumulation in TMEM).
#include "gemm_kernel.cuh"

namespace moebwd {

int launch_gemm_bf16(int BN, const GemmParams& p, const void* tmA, const void* tmB, const void* tmC, int grid,
                     cudaStream_t st) {
  if (p.epi == kEpiCkpt)  // G0 (recomputed pre-activations): 2I is a multiple of 256
    return gemm_launch_instance<false, 256, kEpiCkpt>(p, tmA, tmB, tmC, grid, st);
  if (p.epi == kEpiStore)
    return BN == 256 ? gemm_launch_instance<false, 256, kEpiStore>(p, tmA, tmB, tmC, grid, st)
                     : gemm_launch_instance<false, 128, kEpiStore>(p, tmA, tmB, tmC, grid, st);
  if (p.epi == kEpiDSwiGLU8)  // G1 on an 8-bit checkpoint
    return BN == 256 ? gemm_launch_instance<false, 256, kEpiDSwiGLU8>(p, tmA, tmB, tmC, grid, st)
                     : gemm_launch_instance<false, 128, kEpiDSwiGLU8>(p, tmA, tmB, tmC, grid, st);
  return BN == 256 ? gemm_launch_instance<false, 256, kEpiDSwiGLU>(p, tmA, tmB, tmC, grid, st)
                   : gemm_launch_instance<false, 128, kEpiDSwiGLU>(p, tmA, tmB, tmC, grid, st);
}

}  // namespace moebwd
