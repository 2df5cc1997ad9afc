// Declarations shared by the translation units of the gated feed-forward block.
#pragma once
#include "moebwd_internal.h"

namespace moebwd {

// Tiling of a projection on few tokens (ffn_small.cu): token tile, CTAs along the contraction.
struct SmallPlan {
  int nt, split;
  int64_t tiles, token_tiles;
  float us;  // estimate
};
SmallPlan small_plan(int64_t T, int64_t columns, int64_t K, int per_tile, int sms);

struct FfnSmallArgs {
  const void* W;  // [K, columns], row stride ldw
  int64_t ldw;
  const void* x;  // [T, K], row stride ldx
  int64_t ldx, T, K, N;
  int glu, interleaved, early;
  const uint16_t* bias;
  uint16_t* out;
  uint16_t* h;
  int32_t* status;
};
int launch_ffn_small(bool glu_kernel, const SmallPlan& plan, const FfnSmallArgs& a, cudaStream_t st);

}  // namespace moebwd
