// Backward pass of a linear layer's epilogue y = act(z) + residual, z = x W^T + bias:
//
//   dz[i, j] = dy[i, j] * act'(z[i, j]),   dbias[j] (+)= sum_i dz[i, j]
//
// (the residual's gradient is dy itself).  dz goes on to the quantizers and the
// dgrad and wgrad products.  One pass over dy and z, bound by HBM (6 bytes per
// element): a workgroup owns a strip of columns and a run of rows, each lane sums
// its 8 columns' FP32 dz in registers, the waves' sums meet in LDS in wave order.
//   more than kNarrowRows rows: strips of 512 columns, a wave's 64 lanes on one
//     row; wave w takes rows w, w + 8, ... of its run.  With one run of rows the
//     workgroup writes dbias itself; otherwise its sums go to the caller's
//     workspace [runs][n] and bias_sum_kernel adds the runs in order.
//   up to kNarrowRows rows: strips of 64 columns, one run; 8 lanes on a row, a
//     wave's step 8 rows (wave w rows 8 w .. 8 w + 7, then every 64th row from
//     each), so a column's sums of 8 lanes are added across the wave first, lanes
//     8, 16 and 32 apart in turn.
// No atomics: the bits depend on (m, n) only.  dbias sums the FP32 dz, before its
// bf16 rounding.
//
// About 512 workgroups of 8 waves with 2 rows each in flight: 16384 x 4096 with
// GELU in 75 us, both launches (403 MB, 5.4 TB/s).  2048 workgroups of 4 waves with 4
// rows each took 107 us, 1024 of them 89 us, 256 of 8 waves 76 us; without the
// non-temporal hint the shipped form takes 82 us (4096 x 4096, which the
// last-level cache holds, 23.8 us without and 27 us with it).

#include "common.h"
#include "launch.h"

namespace fp8bs {

constexpr int kBwdWaves = 8;
constexpr int kBwdUnroll = 2;                  // rows of a wave in flight

struct BwdArgs {
  const uint16_t* dy;
  int64_t ldy;
  const uint16_t* z;
  int64_t ldz;
  uint16_t* dz;
  int64_t lddz;
  float* sums;                                 // dbias (one run) or the workspace [runs][n], or null
  int64_t m, n, run_rows;
  int accumulate;                              // one run: add to sums
};

// STREAM: the call's bytes are larger than half the last-level cache, and pass
// through with the non-temporal hint.
// LPR: lanes per row, 64 (strips of 512 columns) or 8 (strips of 64, a wave's step 8 rows).
template <int ACT, bool STREAM, int LPR>
__global__ __launch_bounds__(64 * kBwdWaves) void epilogue_bwd_kernel(BwdArgs p) {
  constexpr int kCols = 8 * LPR, kRows = 64 / LPR;
  __shared__ float part[kBwdWaves][kCols];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t col = (int64_t)blockIdx.x * kCols + 8 * (lane % LPR);
  const bool live = col < p.n;
  const int64_t r0 = (int64_t)blockIdx.y * p.run_rows;
  const int64_t r1 = min(p.m, r0 + p.run_rows);
  auto load = [](const uint16_t* a) { return STREAM ? load_nt(a) : *reinterpret_cast<const uint4*>(a); };
  float sum[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sum[i] = 0.0f;

  if (live) {
    for (int64_t r = r0 + wave * kRows + lane / LPR; r < r1; r += kBwdWaves * kRows * kBwdUnroll) {
      uint4 d[kBwdUnroll], zv[kBwdUnroll];
#pragma unroll
      for (int u = 0; u < kBwdUnroll; ++u) {
        const int64_t row = r + u * kBwdWaves * kRows;
        d[u] = zv[u] = make_uint4(0, 0, 0, 0);
        if (row < r1) {
          d[u] = load(p.dy + row * p.ldy + col);
          if (ACT != FP8BS_ACT_NONE) zv[u] = load(p.z + row * p.ldz + col);
        }
      }
#pragma unroll
      for (int u = 0; u < kBwdUnroll; ++u) {
        const int64_t row = r + u * kBwdWaves * kRows;
        if (row >= r1) break;
        const uint32_t dd[4] = {d[u].x, d[u].y, d[u].z, d[u].w};
        const uint32_t zz[4] = {zv[u].x, zv[u].y, zv[u].z, zv[u].w};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float lo = bf16_lo(dd[i]) * act_slope<ACT>(bf16_lo(zz[i]));
          const float hi = bf16_hi(dd[i]) * act_slope<ACT>(bf16_hi(zz[i]));
          sum[2 * i] += lo;
          sum[2 * i + 1] += hi;
          o[i] = pack_bf16(lo, hi);
        }
        if (!p.dz) continue;
        uint16_t* const dst = p.dz + row * p.lddz + col;
        if (STREAM) store_nt(dst, make_uint4(o[0], o[1], o[2], o[3]));
        else *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
  if (!p.sums) return;
#pragma unroll
  for (int d = LPR; d < 64; d <<= 1)           // the wave's rows
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] += __shfl_xor(sum[i], d);
  if (lane < LPR) {
#pragma unroll
    for (int i = 0; i < 8; ++i) part[wave][8 * lane + i] = sum[i];
  }
  __syncthreads();
  for (int c = threadIdx.x; c < kCols; c += 64 * kBwdWaves) {
    const int64_t j = (int64_t)blockIdx.x * kCols + c;
    if (j >= p.n) continue;
    float s = part[0][c];
#pragma unroll
    for (int w = 1; w < kBwdWaves; ++w) s += part[w][c];
    float* dst = p.sums + (int64_t)blockIdx.y * p.n + j;
    *dst = p.accumulate ? *dst + s : s;
  }
}

// dbias[j] (+)= the runs' sums in order: 16 groups of runs per column, each
// added in order, then the groups in order.
__global__ __launch_bounds__(1024) void bias_sum_kernel(const float* __restrict__ sums, int64_t runs, int64_t n,
                                                        float* __restrict__ dbias, int accumulate) {
  __shared__ float part[16][64];
  const int c = threadIdx.x & 63, grp = threadIdx.x >> 6;
  const int64_t j = (int64_t)blockIdx.x * 64 + c;
  const int64_t per = (runs + 15) / 16;
  float s = 0.0f;
  if (j < n)
    for (int64_t r = grp * per; r < min(runs, (grp + 1) * per); ++r) s += sums[r * n + j];
  part[grp][c] = s;
  __syncthreads();
  if (grp == 0 && j < n) {
    for (int g = 1; g < 16; ++g) s += part[g][c];
    dbias[j] = accumulate ? dbias[j] + s : s;
  }
}

// Up to here a workgroup takes all rows of a strip of 64 columns: one launch and no
// workspace, which saves a short call's host time too (on strips of 512 columns against these:
// 37 x 1536 4.5 and 3.1 us on the device, 256 x 4096 8.4 and 4.7, 15.3 and 10.7 with
// the host's call, 512 x 16384 12.3 and 10.1; at 1024 rows the two launches win).
constexpr int64_t kNarrowRows = 512;

// Rows per run: about 512 workgroups over the strips, 64 rows or more each.
static int64_t bwd_run_rows(int64_t m, int64_t n) {
  if (m <= kNarrowRows) return m;
  const int64_t strips = (n + 511) / 512;
  const int64_t want = strips < 512 ? 512 / strips : 1;
  int64_t rows = (m + want - 1) / want;
  rows = (rows + 15) / 16 * 16;
  if (rows < 64) rows = 64;
  const int64_t least = (m + 65534) / 65535;   // gridDim.y
  return rows < least ? least : rows;
}
static int64_t bwd_runs(int64_t m, int64_t n) { return (m + bwd_run_rows(m, n) - 1) / bwd_run_rows(m, n); }

template <int ACT>
static void launch_bwd(const BwdArgs& a, int64_t runs, hipStream_t s) {
  if (a.m <= kNarrowRows) {
    const dim3 strips((unsigned)((a.n + 63) / 64)), threads(64 * kBwdWaves);
    hipLaunchKernelGGL((epilogue_bwd_kernel<ACT, false, 8>), strips, threads, 0, s, a);
    return;
  }
  const dim3 grid((unsigned)((a.n + 511) / 512), (unsigned)runs), block(64 * kBwdWaves);
  if (6 * a.m * a.n > kStreamBytes)
    hipLaunchKernelGGL((epilogue_bwd_kernel<ACT, true, 64>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((epilogue_bwd_kernel<ACT, false, 64>), grid, block, 0, s, a);
}

}  // namespace fp8bs

using namespace fp8bs;

static bool bwd_sizes_ok(int64_t m, int64_t n) {
  return m > 0 && n > 0 && n % 8 == 0 && m <= 0x7FFFFFFFLL && n <= 0x7FFFFFFFLL;
}

extern "C" int64_t fp8bs_epilogue_backward_workspace(int64_t m, int64_t n) {
  if (!bwd_sizes_ok(m, n)) return FP8BS_ERR_SHAPE;
  const int64_t runs = bwd_runs(m, n);
  return runs > 1 ? runs * n * (int64_t)sizeof(float) : 0;
}

extern "C" int fp8bs_epilogue_backward(const uint16_t* dy, int64_t ldy, const uint16_t* z, int64_t ldz, int64_t m,
                                       int64_t n, int act, uint16_t* dz, int64_t lddz, float* dbias, int accumulate,
                                       float* workspace, int64_t workspace_bytes, void* stream) {
  if (act < FP8BS_ACT_NONE || act > FP8BS_ACT_SILU || (accumulate != 0 && accumulate != 1)) return FP8BS_ERR_FLAG;
  if (!dy || (act != FP8BS_ACT_NONE && !z) || (!dz && !dbias)) return FP8BS_ERR_NULL;
  if (!bwd_sizes_ok(m, n) || ldy < n || (act != FP8BS_ACT_NONE && ldz < n) || (dz && lddz < n)) return FP8BS_ERR_SHAPE;
  if (!aligned(dy, 16) || ldy % 8 || (act != FP8BS_ACT_NONE && (!aligned(z, 16) || ldz % 8)) ||
      (dz && (!aligned(dz, 16) || lddz % 8)) || !aligned(dbias, 4) || !aligned(workspace, 4))
    return FP8BS_ERR_ALIGN;
  const int64_t rows = bwd_run_rows(m, n), runs = bwd_runs(m, n);
  const bool two = dbias && runs > 1;
  if (two && (!workspace || workspace_bytes < fp8bs_epilogue_backward_workspace(m, n))) return FP8BS_ERR_SCRATCH;
  BwdArgs a{dy, ldy, z, ldz, dz, lddz, two ? workspace : dbias, m, n, rows, two ? 0 : accumulate};
  hipStream_t s = (hipStream_t)stream;
  switch (act) {
    case FP8BS_ACT_RELU: launch_bwd<FP8BS_ACT_RELU>(a, runs, s); break;
    case FP8BS_ACT_GELU_TANH: launch_bwd<FP8BS_ACT_GELU_TANH>(a, runs, s); break;
    case FP8BS_ACT_SILU: launch_bwd<FP8BS_ACT_SILU>(a, runs, s); break;
    default: launch_bwd<FP8BS_ACT_NONE>(a, runs, s); break;
  }
  if (two)
    hipLaunchKernelGGL(bias_sum_kernel, dim3((unsigned)((n + 63) / 64)), dim3(1024), 0, s, workspace, runs, n, dbias,
                       accumulate);
  return launch_status();
}
