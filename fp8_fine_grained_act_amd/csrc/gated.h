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

}  // namespace fp8bs
