// A gated feed-forward block, h = act(x Wg^T) * (x Wu^T): the entry points of its
// forward pass and the kernels of its backward pass.
//
// Backward, element by element from dh and the kept z = [g, u] (bf16):
//   dg = dh * u * act'(g),   du = dh * act(g),   h = act(g) * u
// with act(g) and act'(g) from one sigma (common.h).  What the products of the
// backward pass read is made in the same pass, from the unrounded FP32 values: the
// 1x128 tiles of dz = [dg, du] along the columns (activation gradient), and along the
// rows, transposed (weight gradients of both weights; h's for the down projection).
// Bound by HBM: 6 bytes read per element of h, 2 to 10 written.  Without transposed outputs
// 32768 x 2048 in 140 us with dz, h and codes (6.7 TB/s), 16384 x 2048 with codes alone in 43
// us (6.2 TB/s); with both orientations and h's, 16384 x 2048 in 78-82 us (4.7 TB/s), where the
// arithmetic (38 VALU instructions per element, 37 us of issue) and the phases between
// barriers of only two squares per CU come on top.

#include <type_traits>

#include "common.h"
#include "f32_codes.h"
#include "gated.h"
#include "launch.h"

namespace fp8bs {

__device__ __forceinline__ float top8(const float (&x)[8]) {
  float t = top_of(x[0], x[1]);
#pragma unroll
  for (int i = 2; i < 8; ++i) t = top_of(t, x[i]);
  return t;
}

// ---- codes of h from its FP32 values -----------------------------------------------
// Whether some segment holds row first + i, bit i for i < 16, for the whole workgroup of 256 threads: an expert per
// thread and step.  Offsets outside the rows need no clipping, a segment that runs backwards holds none.
__device__ __forceinline__ uint32_t rows_of_segments(const int32_t* __restrict__ seg, int64_t num_experts, int64_t first) {
  __shared__ uint32_t held;
  if (threadIdx.x == 0) held = 0;
  __syncthreads();
  uint32_t mine = 0;
  for (int64_t e = threadIdx.x; e < num_experts; e += 256) {
    const int64_t lo = max((int64_t)seg[e] - first, (int64_t)0), hi = min((int64_t)seg[e + 1] - first, (int64_t)16);
    if (lo < hi) mine |= (1u << hi) - (1u << lo);
  }
  if (mine) atomicOr(&held, mine);
  __syncthreads();
  return held;
}

// h [m, n] FP32 contiguous -> 1x128 tiles along the columns.  16 lanes per tile, 8 values each.  With
// seg only the rows of segments.  Every row from the first offset to the last is one: offsets lead from the one to
// the other and pass it upwards somewhere.  The others are looked for in all segments (rows behind the last one are
// in none, but where offsets run backwards they may be).  A launch of its
// own, 2 us for a few rows, 8 us (4.7 TB/s) for 4096 x 2048.
__global__ __launch_bounds__(256) void quant_h_kernel(const float* __restrict__ hf, int64_t m, int64_t n,
                                                      const int32_t* __restrict__ seg, int64_t num_experts,
                                                      uint8_t* __restrict__ q, int64_t ldq, float* __restrict__ s) {
  const int lane16 = threadIdx.x & 15;
  const uint32_t tiles_n = (uint32_t)(n / kGroup);
  const uint32_t t = blockIdx.x * 16u + (threadIdx.x >> 4);
  const int64_t row = t / tiles_n, tb = t - (uint32_t)row * tiles_n;
  if (seg) {
    const int64_t first = blockIdx.x * 16u / tiles_n, last = (blockIdx.x * 16u + 15u) / tiles_n;   // at most 16 rows
    if (first < seg[0] || last >= seg[num_experts]) {      // the same for the whole workgroup
      const uint32_t held = rows_of_segments(seg, num_experts, first);
      if (!(held >> (row - first) & 1)) return;
    }
  }
  if (row >= m) return;                        // the 16 lanes of a tile together
  const float4* const src = reinterpret_cast<const float4*>(hf + row * n + tb * kGroup + 8 * lane16);
  const float4 a = src[0], b = src[1];
  const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  const F32Scale g = f32_scale(max16_f32(top8(x)));
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = f32_quotient<true>(x[i], g);
  *reinterpret_cast<uint2*>(q + row * ldq + tb * kGroup + 8 * lane16) =
      make_uint2(code4_f32(v[0], v[1], v[2], v[3]), code4_f32(v[4], v[5], v[6], v[7]));
  if (lane16 == 0) s[t] = g.s;
}

static int quant_h(const GatedArgs& a, hipStream_t s) {
  const int64_t tiles = a.p.m * (a.p.n / kGroup);
  hipLaunchKernelGGL(quant_h_kernel, dim3((unsigned)((tiles + 15) / 16)), dim3(256), 0, s, a.p.hf, a.p.m, a.p.n, a.p.seg,
                     a.p.num_experts, a.qh, a.ldqh, a.sh);
  return launch_status();
}

// ---- backward ----------------------------------------------------------------------
struct GatedBwdArgs {
  const uint16_t* dh;
  int64_t lddh;
  const uint16_t* z;
  int64_t ldz;
  int64_t m, n;
  uint16_t* dz;              // [m, 2n] or null
  int64_t lddz;
  uint8_t* q;                // [m, 2n] or null
  int64_t ldq;
  float* s;                  // [m, 2n/128]
  uint8_t* qt;               // [2n, m] or null
  int64_t ldqt;
  float* st;                 // [2n, m/128]
  uint16_t* h;               // [m, n] or null
  int64_t ldh;
  uint8_t* qht;              // [n, m] or null
  int64_t ldqht;
  float* sht;                // [n, m/128]
  const int32_t* row_end;    // rows from *row_end on are left alone, or null
};

// 8 columns of one row: dg, du and h from the packed bf16 inputs
template <int ACT>
__device__ __forceinline__ void gated_slopes(uint4 dh, uint4 g, uint4 u, float (&dg)[8], float (&du)[8], float (&h)[8]) {
  const uint32_t d4[4] = {dh.x, dh.y, dh.z, dh.w}, g4[4] = {g.x, g.y, g.z, g.w}, u4[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float d = i & 1 ? bf16_hi(d4[i / 2]) : bf16_lo(d4[i / 2]);
    const float gv = i & 1 ? bf16_hi(g4[i / 2]) : bf16_lo(g4[i / 2]);
    const float uv = i & 1 ? bf16_hi(u4[i / 2]) : bf16_lo(u4[i / 2]);
    float a, slope;
    act_both<ACT>(gv, a, slope);
    dg[i] = d * uv * slope;
    du[i] = d * a;
    h[i] = a * uv;
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// 8 codes of one row's tile piece of dg and of du, their scales stored by the tiles' first lane (16 lanes a
// tile).  Where every group of the wave is of ordinary size, a scale takes three operations and its reciprocal three.
template <bool SLOW>
__device__ __forceinline__ uint2 row_codes(const float (&x)[8], const F32Scale& g) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = f32_quotient<SLOW>(x[i], g);
  return make_uint2(code4_f32(v[0], v[1], v[2], v[3]), code4_f32(v[4], v[5], v[6], v[7]));
}
struct RowCodes {
  uint2 g, u;                // codes of dg and du
  float sg, su;
};
template <bool SLOW>
__device__ __forceinline__ RowCodes code_row_by(const float (&dg)[8], const float (&du)[8], const F32Scale& g, const F32Scale& u) {
  return RowCodes{row_codes<SLOW>(dg, g), row_codes<SLOW>(du, u), g.s, u.s};
}
__device__ __forceinline__ RowCodes code_row(const float (&dg)[8], const float (&du)[8]) {
  const float a = max16_f32(top8(dg)), b = max16_f32(top8(du));
  if (__ballot(fminf(a, b) < kTinyGroup)) return code_row_by<true>(dg, du, f32_scale(a), f32_scale(b));
  return code_row_by<false>(dg, du, f32_scale_ordinary(a), f32_scale_ordinary(b));
}

// Without transposed outputs: 16 lanes per piece of 128 columns of a row.
template <int ACT, bool STREAM>
__global__ __launch_bounds__(256) void gated_bwd_rows_kernel(GatedBwdArgs p, uint32_t pieces_n, uint32_t pieces) {
  const int lane16 = threadIdx.x & 15;
  const uint32_t t = blockIdx.x * 16u + (threadIdx.x >> 4);
  if (t >= pieces) return;
  const uint32_t row = t / pieces_n, tb = t - row * pieces_n;
  const int64_t col = (int64_t)tb * kGroup + 8 * lane16;
  if (col >= p.n || (p.row_end && (int64_t)row >= *p.row_end)) return;   // n % 128 != 0 has no codes: no lane is waited for
  auto load = [](const uint16_t* a) { return STREAM ? load_nt(a) : *reinterpret_cast<const uint4*>(a); };
  auto store = [](uint16_t* a, uint4 v) {
    if (STREAM) store_nt(a, v);
    else *reinterpret_cast<uint4*>(a) = v;
  };
  const uint16_t* const zr = p.z + row * p.ldz + col;
  const uint4 dhv = load(p.dh + row * p.lddh + col), gv = load(zr), uv = load(zr + p.n);
  float dg[8], du[8], h[8];
  gated_slopes<ACT>(dhv, gv, uv, dg, du, h);
  if (p.dz) {
    store(p.dz + row * p.lddz + col, pack8(dg));
    store(p.dz + row * p.lddz + p.n + col, pack8(du));
  }
  if (p.h) store(p.h + row * p.ldh + col, pack8(h));
  if (p.q) {
    uint8_t* const qr = p.q + row * p.ldq + col;
    float* const sr = p.s + row * (int64_t)(2 * pieces_n) + tb;
    const RowCodes o = code_row(dg, du);
    *reinterpret_cast<uint2*>(qr) = o.g;
    *reinterpret_cast<uint2*>(qr + p.n) = o.u;
    if (lane16 == 0) {
      sr[0] = o.sg;
      sr[pieces_n] = o.su;
    }
  }
}

// The square (column, row) of workgroup b.  Each XCD (they take workgroups in turn) owns one
// range of squares, in bands of 8 squares down: neighbours in both directions then
// meet in one L2, and with them the scales' lines, of which a square writes 4 bytes,
// and the transposed rows' pages (8192 x 7168 139 -> 125 us; by now 117, with bands of 4 119, of 32 122).
__device__ __forceinline__ uint2 square_of(uint32_t b, uint32_t nx, uint32_t ny) {
  const uint32_t per = (nx * ny + 7) / 8, full = nx * ny - 8 * (per - 1), x = b % 8, j = b / 8;
  const uint32_t l = x < full ? x * per + j : full * per + (x - full) * (per - 1) + j;
  const uint32_t band = l / (8 * nx), r = l - band * 8 * nx, rows = min(8u, ny - 8 * band);
  return make_uint2(r / rows, 8 * band + r % rows);
}

// With transposed outputs: a workgroup of 8 waves owns a square of 128 rows and 128
// columns of h.  Thread (cg, rg) = (tid % 16, tid / 16) holds columns 8 cg .. 8 cg + 7 of rows
// 4 rg .. 4 rg + 3 in FP32 registers, so both tile directions are coded from the
// same values without staging them: a row's amax crosses its 16 lanes (DPP), a
// column's the wave (two lane swaps) and then the waves in LDS.  The transposed
// codes, 4 bytes of a column per thread, meet in LDS and leave as whole 128-byte
// rows of the output: dword d of column c is stored at d ^ (4 * ((c / 8) % 8)), which
// keeps 16-byte chunks whole and puts a wave's 64 writes on 32 banks, two each.
// 128 registers (the FP32 values are 96 of them), so that two squares share a CU: 140 us
// for 16384 x 2048 with 136 registers and one, 86 with two.  An address is the wave's, in
// scalar registers, plus the lane's 32-bit offset, at most 15 rows away: strides are below
// 2^28 elements (81 -> 78.5 us, with the ordinary groups' shorter scales).
constexpr int64_t kMaxSquareStride = (1 << 28) - 1;

template <int ACT, int STREAM>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(4, 4))) void gated_bwd_square_kernel(GatedBwdArgs p) {
  __shared__ float tops[3][8][128];            // [dg, du, h][wave][column]
  __shared__ float2 rcps[3][128];              // a column's r and rl
  __shared__ float ups[3][128];                // and its up
  __shared__ int tiny;                         // some up is not 1
  __shared__ __attribute__((aligned(16))) uint32_t codes[3][128 * 32];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int cg = tid & 15, rg = tid >> 4;
  const uint2 square = square_of(blockIdx.x, (uint32_t)(p.n / kGroup), (uint32_t)(p.m / kGroup));
  const uint32_t bx = square.x, by = square.y;
  const int64_t c0 = (int64_t)bx * 128, r0 = (int64_t)by * 128;
  const int64_t rw = r0 + 16 * wave;           // the wave's first row
  const uint32_t r4 = 4 * (rg & 3);            // the lane's first row from there
  const int nq = p.qht ? 3 : 2, q0 = p.qt ? 0 : 2;
  auto load = [](const uint16_t* a) { return STREAM ? load_nt(a) : *reinterpret_cast<const uint4*>(a); };
  auto store = [](void* a, uint4 v, int from) {  // past the caches from that degree on
    if (STREAM >= from) store_nt(a, v);
    else *reinterpret_cast<uint4*>(a) = v;
  };
  uint4 dhv[4], gv[4], uv[4];
  {
    const uint32_t od = r4 * (uint32_t)p.lddh + 8 * cg, oz = r4 * (uint32_t)p.ldz + 8 * cg;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint16_t *const dr = p.dh + (rw + i) * p.lddh + c0, *const zr = p.z + (rw + i) * p.ldz + c0;
      dhv[i] = load(dr + od);
      gv[i] = load(zr + oz);
      uv[i] = load(zr + p.n + oz);
    }
  }
  float x[3][4][8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    gated_slopes<ACT>(dhv[i], gv[i], uv[i], x[0][i], x[1][i], x[2][i]);
    if (p.dz) {
      uint16_t* const zr = p.dz + (rw + i) * p.lddz + c0;
      const uint32_t o = r4 * (uint32_t)p.lddz + 8 * cg;
      store(zr + o, pack8(x[0][i]), 3);
      store(zr + p.n + o, pack8(x[1][i]), 3);
    }
    if (p.h) store(p.h + (rw + i) * p.ldh + c0 + (r4 * (uint32_t)p.ldh + 8 * cg), pack8(x[2][i]), 3);
    if (p.q) {
      const RowCodes o = code_row(x[0][i], x[1][i]);
      uint8_t* const qr = p.q + (rw + i) * p.ldq + c0;
      const uint32_t oq = r4 * (uint32_t)p.ldq + 8 * cg;
      *reinterpret_cast<uint2*>(qr + oq) = o.g;
      *reinterpret_cast<uint2*>(qr + p.n + oq) = o.u;
      if (cg == 0) {
        const uint32_t lds = 2 * (uint32_t)p.n / kGroup;
        float* const sr = p.s + (rw + i) * lds + bx;
        sr[r4 * lds] = o.sg;
        sr[r4 * lds + lds / 2] = o.su;
      }
    }
    __builtin_amdgcn_sched_barrier(0);         // a row at a time: few live temporaries
  }
  // columns' maxima
  if (tid == 0) tiny = 0;
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    float t[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      t[j] = top_of(top_of(x[q][0][j], x[q][1][j]), top_of(x[q][2][j], x[q][3][j]));
    // over the wave's four groups of 16 lanes, two columns to a swap: afterwards group gr holds
    // columns 4 (gr % 2) + 2 (gr / 2) and the next of its 8
#pragma unroll
    for (int j = 0; j < 4; ++j) t[j] = max_swap16_f32(t[j], t[j + 4]);
#pragma unroll
    for (int j = 0; j < 2; ++j) t[j] = max_swap32_f32(t[j], t[j + 2]);
    *reinterpret_cast<float2*>(&tops[q][wave][8 * cg + 4 * ((lane >> 4) & 1) + 2 * (lane >> 5)]) = make_float2(t[0], t[1]);
  }
  __syncthreads();
  if (tid < 384) {
    const int q = tid >> 7, c = tid & 127;
    float t = tops[q][0][c];
#pragma unroll
    for (int w = 1; w < 8; ++w) t = top_of(t, tops[q][w][c]);
    const F32Scale g = f32_scale(t);
    rcps[q][c] = make_float2(g.r, g.rl);
    ups[q][c] = g.up;
    if (g.up != 1.0f) tiny = 1;
    if (q >= q0 && q < nq) {
      float* const s = q == 2 ? p.sht : p.st + (q * p.n) * (p.m / kGroup);
      s[(c0 + c) * (p.m / kGroup) + by] = g.s;
    }
  }
  __syncthreads();
  auto code_columns = [&](auto slow) {
    constexpr bool SLOW = decltype(slow)::value;
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      if (q < q0 || q >= nq) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 r = rcps[q][8 * cg + j];
        const F32Scale col{0.0f, r.x, r.y, SLOW ? ups[q][8 * cg + j] : 1.0f};
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = f32_quotient<SLOW>(x[q][i][j], col);
        codes[q][(8 * cg + j) * 32 + (rg ^ ((cg & 7) << 2))] = code4_f32(v[0], v[1], v[2], v[3]);
        __builtin_amdgcn_sched_barrier(0);     // a column at a time: few live scales
      }
    }
  };
  if (tiny) code_columns(std::true_type{});
  else code_columns(std::false_type{});
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    if (q < q0 || q >= nq) continue;
    uint8_t* const out = q == 2 ? p.qht : p.qt + q * p.n * p.ldqt;
    const int64_t ld = q == 2 ? p.ldqht : p.ldqt;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int cw = 64 * i + 8 * wave, cl = lane >> 3, k = lane & 7;
      const uint4 v = *reinterpret_cast<const uint4*>(&codes[q][(cw + cl) * 32 + 4 * (k ^ wave)]);
      store(out + (c0 + cw) * ld + r0 + (cl * (uint32_t)ld + 16 * k), v, 2);
    }
  }
}

template <int ACT>
static int launch_gated_bwd(const GatedBwdArgs& a, hipStream_t s) {
  const int64_t size = a.m * a.n;
  // What passes through with the non-temporal hint, by degrees (kStreamBytes is half the last-level cache):
  //   1  reads and writes exceed it: the inputs, and without transposed outputs dz and h
  //   2  the writes alone do: the transposed codes too (the codes along the columns stay: the
  //      activation gradient reads them next)
  //   3  the writes exceed twice that, the whole cache: dz and h of the squares too
  // Squares with codes alone, outputs in new memory / in one place: 8192 x 2048 53 / 49 us at degree 0, 47 / 47 at
  // 1, 48 / 48 at 2; 16384 x 2048 85 / 76 at 1, 75 / 76 at 2; 8192 x 7168 144 / 125 and 117 / 117; 65536 x 1408
  // 230 / 221 and 207 / 186; every store past the caches 87, 124 and 191.  4096 x 2048, 93 MB in all, 18.6 at 0 and
  // 21.4 at 1.  With dz and h, 11008 x 2048 73 at 2 and 78 at 3, 8192 x 7168 220 and 180.  (Measured with the codes
  // from one product with the reciprocal; they take up to 6 us more now, at any degree.)
  const int64_t writes = size * ((a.dz ? 4 : 0) + (a.q ? 2 : 0) + (a.qt ? 2 : 0) + (a.h ? 2 : 0) + (a.qht ? 1 : 0));
  const int stream = 6 * size + writes <= kStreamBytes ? 0 : writes <= kStreamBytes ? 1 : writes <= 2 * kStreamBytes ? 2 : 3;
  if (a.qt || a.qht) {
    const dim3 grid((unsigned)((a.n / kGroup) * (a.m / kGroup)));
    if (stream == 3) hipLaunchKernelGGL((gated_bwd_square_kernel<ACT, 3>), grid, dim3(512), 0, s, a);
    else if (stream == 2) hipLaunchKernelGGL((gated_bwd_square_kernel<ACT, 2>), grid, dim3(512), 0, s, a);
    else if (stream) hipLaunchKernelGGL((gated_bwd_square_kernel<ACT, 1>), grid, dim3(512), 0, s, a);
    else hipLaunchKernelGGL((gated_bwd_square_kernel<ACT, 0>), grid, dim3(512), 0, s, a);
    return launch_status();
  }
  const int64_t pieces_n = (a.n + kGroup - 1) / kGroup, pieces = a.m * pieces_n;
  const dim3 grid((unsigned)((pieces + 15) / 16));
  if (stream) hipLaunchKernelGGL((gated_bwd_rows_kernel<ACT, true>), grid, dim3(256), 0, s, a, (uint32_t)pieces_n, (uint32_t)pieces);
  else hipLaunchKernelGGL((gated_bwd_rows_kernel<ACT, false>), grid, dim3(256), 0, s, a, (uint32_t)pieces_n, (uint32_t)pieces);
  return launch_status();
}

}  // namespace fp8bs

using namespace fp8bs;

// Checks shared by the two forward entry points (m, n, k known to be non-negative).
static int gated_check(const GatedArgs& a, float* workspace) {
  const SkinnyArgs& p = a.p;
  if ((a.qh == nullptr) != (a.sh == nullptr) || (p.m > 0 && !p.c && !a.qh)) return FP8BS_ERR_NULL;
  if (p.epi.act < FP8BS_ACT_NONE || p.epi.act > FP8BS_ACT_SILU) return FP8BS_ERR_FLAG;
  if (p.n <= 0 || p.k <= 0 || p.n % 128 || p.k % BK || (p.c && p.ldc < p.n) || (p.epi.z && p.epi.ldz < 2 * p.n) ||
      (a.qh && a.ldqh < p.n) || p.k >= 1 << 24 || p.n > 0xFFFFFFFFLL / (2 * p.k) || p.m > kMaxGrid / (p.n / 16))
    return FP8BS_ERR_SHAPE;
  if (!aligned(p.qa, 16) || !aligned(p.qb, 16) || !aligned(p.sa, 4) || !aligned(p.sb, 4) || !aligned(p.seg, 4) ||
      (p.c && (!aligned(p.c, 16) || p.ldc % 8)) || (p.epi.z && (!aligned(p.epi.z, 16) || p.epi.ldz % 8)) ||
      (a.qh && (!aligned(a.qh, 16) || a.ldqh % 16 || !aligned(a.sh, 4))) || !aligned(workspace, 16))
    return FP8BS_ERR_ALIGN;
  return FP8BS_OK;
}

// h in FP32, for the kernels whose tiles do not hold a row's 128 columns
static int64_t gated_workspace(const GatedArgs& a, int bn) { return a.qh && bn != 256 ? 4 * a.p.m * a.p.n : 0; }

static int gated_run(GatedArgs a, float* workspace, int64_t workspace_bytes, hipStream_t s) {
  const int64_t cus = cu_count();
  const int bn = gated_tile_cols(a, cus);
  const int64_t need = gated_workspace(a, bn);
  if (need > 0 && (!workspace || workspace_bytes < need)) return FP8BS_ERR_SCRATCH;
  a.p.hf = need > 0 ? workspace : nullptr;
  int st = bn ? launch_gated_tiles(a, bn, s) : launch_skinny(a.p, 0, cus, s);
  if (st == FP8BS_OK && need > 0) st = quant_h(a, s);
  return st;
}

// The workspace of sizes alone: seg for expert segments (its contents do not count).
static int64_t gated_workspace_of(int64_t m, int64_t n, int64_t k, int64_t num_experts, const int32_t* seg) {
  GatedArgs a{};
  if (m <= 0 || k <= 0) return FP8BS_ERR_SHAPE;
  a.p.m = m;
  a.p.n = n;
  a.p.k = k;
  a.p.gated = 1;
  a.p.num_experts = num_experts;
  a.p.seg = seg;
  a.qh = reinterpret_cast<uint8_t*>(16);       // any aligned address: not used
  a.sh = reinterpret_cast<float*>(16);
  a.ldqh = n > 0 ? n : 0;
  const int st = gated_check(a, nullptr);
  return st == FP8BS_OK ? gated_workspace(a, gated_tile_cols(a, cu_count())) : st;
}

extern "C" int64_t fp8bs_gemm_gated_workspace(int64_t m, int64_t n, int64_t k) {
  return gated_workspace_of(m, n, k, 1, nullptr);
}

extern "C" int64_t fp8bs_grouped_gemm_gated_ragged_workspace(int64_t num_experts, int64_t total_rows, int64_t n, int64_t k) {
  if (num_experts < 1 || num_experts > 65536 || total_rows < 0 || total_rows > 0x3FFFFFFFLL || k <= 0 || n <= 0 || n % 128 ||
      k % BK)
    return FP8BS_ERR_SHAPE;
  return total_rows == 0 ? 0 : gated_workspace_of(total_rows, n, k, num_experts, reinterpret_cast<const int32_t*>(16));
}

extern "C" int fp8bs_gemm_gated(const uint8_t* qa, const float* sa, const uint8_t* qb, const float* sb, int64_t m, int64_t n,
                                int64_t k, int act, uint16_t* z, int64_t ldz, uint16_t* h, int64_t ldh, uint8_t* qh,
                                int64_t ldqh, float* sh, float* workspace, int64_t workspace_bytes, void* stream) {
  if (!qa || !sa || !qb || !sb) return FP8BS_ERR_NULL;
  if (m <= 0 || k <= 0) return FP8BS_ERR_SHAPE;
  GatedArgs a{{qa, sa, qb, sb, h, ldh, m, n, k, nullptr, 1, Epilogue{nullptr, nullptr, 0, z, ldz, act}, 1, nullptr}, qh, ldqh, sh};
  const int chk = gated_check(a, workspace);
  return chk != FP8BS_OK ? chk : gated_run(a, workspace, workspace_bytes, (hipStream_t)stream);
}

extern "C" int fp8bs_grouped_gemm_gated_ragged(const uint8_t* qa, const float* sa, const int32_t* seg_offsets,
                                               int64_t num_experts, int64_t total_rows, const uint8_t* qb, const float* sb,
                                               int64_t n, int64_t k, int act, uint16_t* z, int64_t ldz, uint16_t* h,
                                               int64_t ldh, uint8_t* qh, int64_t ldqh, float* sh, float* workspace,
                                               int64_t workspace_bytes, void* stream) {
  if (!seg_offsets || !qb || !sb || (total_rows > 0 && (!qa || !sa))) return FP8BS_ERR_NULL;
  if (num_experts < 1 || num_experts > 65536 || total_rows < 0 || total_rows > 0x3FFFFFFFLL || k <= 0) return FP8BS_ERR_SHAPE;
  GatedArgs a{{qa, sa, qb, sb, h, ldh, total_rows, n, k, seg_offsets, num_experts, Epilogue{nullptr, nullptr, 0, z, ldz, act},
               1, nullptr}, qh, ldqh, sh};
  const int chk = gated_check(a, workspace);
  if (chk != FP8BS_OK || total_rows == 0) return chk;
  return gated_run(a, workspace, workspace_bytes, (hipStream_t)stream);
}

extern "C" int fp8bs_gated_backward(const uint16_t* dh, int64_t lddh, const uint16_t* z, int64_t ldz, int64_t m, int64_t n,
                                    int act, uint16_t* dz, int64_t lddz, uint8_t* q, int64_t ldq, float* scales, uint8_t* qt,
                                    int64_t ldqt, float* scales_t, uint16_t* h, int64_t ldh, uint8_t* qht, int64_t ldqht,
                                    float* scales_ht, const int32_t* row_end, void* stream) {
  if ((m > 0 && (!dh || !z || (!dz && !q && !qt && !h && !qht))) || (q == nullptr) != (scales == nullptr) ||
      (qt == nullptr) != (scales_t == nullptr) || (qht == nullptr) != (scales_ht == nullptr))
    return FP8BS_ERR_NULL;
  if (act < FP8BS_ACT_NONE || act > FP8BS_ACT_SILU) return FP8BS_ERR_FLAG;
  const bool cols = qt || qht;
  if (m < 0 || n <= 0 || n % 8 || n > 0x3FFFFFFFLL || m > 0x7FFFFFFFLL || ((q || cols) && n % kGroup) ||
      (cols && (m % kGroup || row_end || m / kGroup > 65535)) || m > (kMaxGrid - 16) / ((n + kGroup - 1) / kGroup) || lddh < n ||
      ldz < 2 * n || (dz && lddz < 2 * n) || (q && ldq < 2 * n) || (qt && ldqt < m) || (h && ldh < n) || (qht && ldqht < m) ||
      (cols && (lddh > kMaxSquareStride || ldz > kMaxSquareStride || (dz && lddz > kMaxSquareStride) ||
                (q && ldq > kMaxSquareStride) || (qt && ldqt > kMaxSquareStride) || (h && ldh > kMaxSquareStride) ||
                (qht && ldqht > kMaxSquareStride))))
    return FP8BS_ERR_SHAPE;
  if (!aligned(dh, 16) || lddh % 8 || !aligned(z, 16) || ldz % 8 || (dz && (!aligned(dz, 16) || lddz % 8)) ||
      (q && (!aligned(q, 16) || ldq % 16)) || (qt && (!aligned(qt, 16) || ldqt % 16)) || (h && (!aligned(h, 16) || ldh % 8)) ||
      (qht && (!aligned(qht, 16) || ldqht % 16)) || !aligned(scales, 4) || !aligned(scales_t, 4) || !aligned(scales_ht, 4) ||
      !aligned(row_end, 4))
    return FP8BS_ERR_ALIGN;
  if (m == 0) return FP8BS_OK;
  const GatedBwdArgs a{dh, lddh, z, ldz, m, n, dz, lddz, q, ldq, scales, qt, ldqt, scales_t, h, ldh, qht, ldqht, scales_ht, row_end};
  hipStream_t s = (hipStream_t)stream;
  switch (act) {
    case FP8BS_ACT_RELU: return launch_gated_bwd<FP8BS_ACT_RELU>(a, s);
    case FP8BS_ACT_GELU_TANH: return launch_gated_bwd<FP8BS_ACT_GELU_TANH>(a, s);
    case FP8BS_ACT_SILU: return launch_gated_bwd<FP8BS_ACT_SILU>(a, s);
    default: return launch_gated_bwd<FP8BS_ACT_NONE>(a, s);
  }
}
