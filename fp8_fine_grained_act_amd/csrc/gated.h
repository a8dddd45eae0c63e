// A gated feed-forward block's forward pass (gated.hip, skinny.hip, gemm.hip).
#pragma once

#include "skinny.h"

namespace fp8bs {

struct GatedArgs {
  SkinnyArgs p;              // gated, seg for expert segments; c = h in bf16 or null, hf = h in FP32 or null
  uint8_t* qh;               // E4M3 codes of h's 1x128 tiles [m, n], row stride ldqh, or null
  int64_t ldqh;
  float* sh;                 // their scales [m, n/128]
};

// The kernel of a gated product (gemm.hip): 0 for the few-row tiles of skinny.hip, else the
// weight rows of a warp-specialized tile, 128 (64 columns of h) or 256 (128 columns, whose rows' codes it makes itself).
int gated_tile_cols(const GatedArgs& a, int64_t cus);
int launch_gated_tiles(const GatedArgs& a, int bn, hipStream_t s);

}  // namespace fp8bs
