// Experts' weight gradients over row segments of any length:
//
//   dW[e][i, j] (+)= sum over rows t of segment e of dy[t, i] * x[t, j]
//
// bf16 rows in, FP32 out.  In an unpadded layout a 128-token FP8 tile would
// cross experts, and the FP8 MFMA's in-block summation is only good to about
// 1e-5 of an FP32 output, so the operands stay bf16: their products are exact
// in FP32 and the matrix cores add them in FP32.
//
// Both operands have the contraction (rows t) as their slow index.  A slab of
// kT rows by 128 columns of each is copied as it lies straight into LDS
// (buffer_load ... lds); the fragments, which need consecutive t per lane, are
// gathered with ds_read_b64_tr_b16: in a group of 16 lanes that each point at 4
// bf16, lane i receives element i mod 4 of the words of lanes 4r + i div 4, r =
// 0..3; lane j therefore points at row t = 8g + j div 4 (+ 4 for the second
// read), columns 4 (j mod 4) of the tile's 16, and lane i ends with column i at
// t = 8g .. 8g + 7.
// LDS rows are 256 bytes = 8 units of 32 bytes (one 16-column tile each); unit
// u of row t is stored at u ^ f(t), f = (t & 3) | ((t >> 1) & 4), so the 8 rows
// that 32 lanes read together (t = 0..3 and 8..11 of a half slab) fall on 64
// distinct banks.
// Rows past the segment's end read as zeros (buffer range check).

#include "common.h"
#include "launch.h"

namespace fp8bs {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef short v4i16 __attribute__((ext_vector_type(4)));

struct RaggedWgradArgs {
  const uint16_t* dy;
  int64_t ldy;
  const uint16_t* x;
  int64_t ldx;
  const int32_t* seg;
  int64_t total_rows, m, n;
  float* c;
  int64_t tiles_m, tiles_n;
  int accumulate;
};

constexpr int kT = 64;                         // rows of a slab

__device__ __forceinline__ int tswz(int t) { return (t & 3) | ((t >> 1) & 4); }

struct WgStage {
  uint8_t a[kT * 256];
  uint8_t b[kT * 256];
};
template <int IDX>
__device__ __forceinline__ WgStage& wg_stage() {
  __shared__ __attribute__((aligned(16))) WgStage st;
  return st;
}

__global__ __launch_bounds__(256) void ragged_wgrad_kernel(RaggedWgradArgs p) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int l16 = lane & 15, g = lane >> 4;

  const int64_t tiles = p.tiles_m * p.tiles_n;
  const int64_t e = (int64_t)blockIdx.x / tiles, tb = (int64_t)blockIdx.x - e * tiles;
  const int64_t m0 = tb / p.tiles_n * 128, n0 = tb % p.tiles_n * 128;
  const int cap = (int)p.total_rows;
  const int s0 = min(max(p.seg[e], 0), cap);
  const int rows = max(0, min(max(p.seg[e + 1], 0), cap) - s0);
  if (rows == 0 && p.accumulate) return;
  const int slabs = (rows + kT - 1) / kT;

  const uint16_t* const a0 = p.dy + (int64_t)s0 * p.ldy + m0;
  const uint16_t* const b0 = p.x + (int64_t)s0 * p.ldx + n0;
  const int64_t mw = min((int64_t)128, p.m - m0), nw = min((int64_t)128, p.n - n0);

  // one copy instruction fills 4 rows; lane: row r4, stored chunk pc of 16
  const int r4 = lane >> 4, pc = lane & 15;
  auto issue = [&](int s, WgStage& st) {
    const int64_t t0 = (int64_t)s * kT;
    const int64_t left = rows - t0;
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(a0 + t0 * p.ldy, ((left - 1) * p.ldy + mw) * 2);
    const __amdgpu_buffer_rsrc_t rb = make_rsrc(b0 + t0 * p.ldx, ((left - 1) * p.ldx + nw) * 2);
#pragma unroll
    for (int i = 0; i < kT / 16; ++i) {
      const int q = wave + 4 * i, t = 4 * q + r4;
      const int chunk = (((pc >> 1) ^ tswz(t)) << 1) | (pc & 1);
      dma16(ra, st.a + q * 1024, (uint32_t)((int64_t)t * p.ldy * 2 + chunk * 16), 0);
      dma16(rb, st.b + q * 1024, (uint32_t)((int64_t)t * p.ldx * 2 + chunk * 16), 0);
    }
  };
  auto frag = [&](const uint8_t* base, int k0, int tile) -> v8bf {
    v4i16 h[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int t = k0 + 8 * g + 4 * u + (l16 >> 2);
      h[u] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (__attribute__((address_space(3))) v4i16*)(base + t * 256 + ((tile ^ tswz(t)) << 5) + ((l16 & 3) << 3)));
    }
    typedef short v8i16 __attribute__((ext_vector_type(8)));
    const v8i16 r = {h[0][0], h[0][1], h[0][2], h[0][3], h[1][0], h[1][1], h[1][2], h[1][3]};
    return __builtin_bit_cast(v8bf, r);
  };

  v4f acc[4][4];                               // [n tile][m tile]
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  auto barrier = [&]() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  auto slab = [&](int s, WgStage& cur, WgStage& nxt) {
    if (s + 1 < slabs) {
      issue(s + 1, nxt);
      wait_vmcnt<2 * (kT / 16)>();             // this slab's copies have landed, the next one's may fly
    } else {
      wait_vmcnt<0>();
    }
    barrier();
#pragma unroll
    for (int k0 = 0; k0 < kT; k0 += 32) {
      v8bf af[4], bf[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) af[j] = frag(cur.a, k0, 4 * wm + j);
#pragma unroll
      for (int i = 0; i < 4; ++i) bf[i] = frag(cur.b, k0, 4 * wn + i);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[i], af[j], acc[i][j], 0, 0, 0);
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);        // lgkmcnt(0): the slab is read before it is refilled
    barrier();
  };
  if (slabs > 0) issue(0, wg_stage<0>());
  for (int s = 0; s < slabs; s += 2) {
    slab(s, wg_stage<0>(), wg_stage<1>());
    if (s + 1 < slabs) slab(s + 1, wg_stage<1>(), wg_stage<0>());
  }

  float* const ce = p.c + e * p.m * p.n;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t row = m0 + 64 * wm + 16 * j + l16;
    if (row >= p.m) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t col = n0 + 64 * wn + 16 * i + 4 * g;
      if (col >= p.n) continue;
      float* dst = ce + row * p.n + col;
      float4 o = make_float4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
      if (p.accumulate) {
        const float4 old = *reinterpret_cast<const float4*>(dst);
        o.x += old.x; o.y += old.y; o.z += old.z; o.w += old.w;
      }
      *reinterpret_cast<float4*>(dst) = o;
    }
  }
}

}  // namespace fp8bs

using namespace fp8bs;

extern "C" int fp8bs_grouped_wgrad_ragged(const uint16_t* dy, int64_t ldy, const uint16_t* x, int64_t ldx,
                                          const int32_t* seg_offsets, int64_t num_experts, int64_t total_rows,
                                          int64_t m, int64_t n, float* c, int accumulate, void* stream) {
  if (!seg_offsets || !c || (total_rows > 0 && (!dy || !x))) return FP8BS_ERR_NULL;
  if (accumulate != 0 && accumulate != 1) return FP8BS_ERR_FLAG;
  if (num_experts < 1 || num_experts > 65536 || total_rows < 0 || total_rows > 0x3FFFFFFFLL || m <= 0 || n <= 0 ||
      m % 8 || n % 8 || ldy < m || ldx < n || ldy > (1 << 24) || ldx > (1 << 24))
    return FP8BS_ERR_SHAPE;
  if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(c, 16) || !aligned(seg_offsets, 4) || ldy % 8 || ldx % 8)
    return FP8BS_ERR_ALIGN;
  RaggedWgradArgs a{dy, ldy, x, ldx, seg_offsets, total_rows, m, n, c, (m + 127) / 128, (n + 127) / 128, accumulate};
  const int64_t grid = num_experts * a.tiles_m * a.tiles_n;
  if (grid > kMaxGrid) return FP8BS_ERR_SHAPE;
  hipLaunchKernelGGL(ragged_wgrad_kernel, dim3((unsigned)grid), dim3(256), 0, (hipStream_t)stream, a);
  return launch_status();
}
