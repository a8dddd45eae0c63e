// Block-scaled products with few rows (skinny.hip).
#pragma once

#include "common.h"

namespace fp8bs {

struct SkinnyArgs {
  const uint8_t* qa;
  const float* sa;
  const uint8_t* qb;
  const float* sb;
  uint16_t* c;
  int64_t ldc;
  int64_t m, n, k;
  const int32_t* seg;        // ragged expert segments, or null: one product of m rows
  int64_t num_experts;
  Epilogue epi;
  int gated;                 // qb, sb hold two weights [2n, .]: c = act(z_gate) * z_up, epi.z [m, 2n] (b_layout 0)
  float* hf;                 // gated: h in FP32 [m, n] as well, or null (c may be null then)
};

// What the product takes on the best shape of skinny.hip, in us per 56 blocks of
// the contraction (the comparison's unit; gemm.hip knows its own kernels').
int64_t skinny_cost(const SkinnyArgs& a, int b_layout, int64_t cus);

// Enqueues the product; sizes and alignment as the callers have checked them.
int launch_skinny(const SkinnyArgs& a, int b_layout, int64_t cus, hipStream_t s);

}  // namespace fp8bs
