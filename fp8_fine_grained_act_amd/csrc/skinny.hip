// Block-scaled FP8 products with few rows: decode steps of a linear layer and
// of the experts.  Bound by the weights' bytes, each read once: there is
// nothing to reuse across tiles, so no barrier and no shared staging stands in
// the main loop.  A workgroup owns 16 MT rows by NB columns of the output; its
// waves split the contraction (wave w takes blocks w, w + W, ...), each with its
// own loads in flight, and meet once, at the end, in LDS: the waves' partial
// sums are added in wave order, then the epilogue is applied and the row pieces
// stored.
//   b_layout 0 (weight rows along k): NB = 16; the MFMA fragments are 32
//     consecutive bytes of a weight row per lane, loaded straight into
//     registers, the next kU blocks while the current ones multiply.
//   b_layout 1 (weight rows along n): NB = 128, so that a row's piece is a whole
//     128-byte line.  The fragments need 32 consecutive k of one column: each
//     wave copies its 128 x 128 blocks into its own two LDS slabs
//     (buffer_load ... lds) and gathers them with ds_read_b64_tr_b8 (the layout
//     of the dgrad slabs in gemm.hip).
// Rows past the end are read as the last row again and not stored.

#include "launch.h"
#include "skinny.h"

namespace fp8bs {

// z for 4 consecutive columns of one row -> z out, activation, residual, bf16
__device__ __forceinline__ void finish4(const SkinnyArgs& p, int64_t row, int64_t col, float4 s) {
  const Epilogue& ep = p.epi;
  float x[4] = {s.x, s.y, s.z, s.w};
  if (ep.bias) {
#pragma unroll
    for (int v = 0; v < 4; ++v) x[v] += ep.bias[col + v];
  }
  auto pack = [&]() { return make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])); };
  if (ep.z) *reinterpret_cast<uint2*>(ep.z + row * ep.ldz + col) = pack();
  act_forward4(ep.act, x);
  if (ep.res) {
    const uint2 r = *reinterpret_cast<const uint2*>(ep.res + row * ep.ldr + col);
    x[0] += bf16_lo(r.x);
    x[1] += bf16_hi(r.x);
    x[2] += bf16_lo(r.y);
    x[3] += bf16_hi(r.y);
  }
  *reinterpret_cast<uint2*>(p.c + row * p.ldc + col) = pack();
}

// The workgroup's rows and weight: a tile of a ragged segment, or of the one product.
template <int MT, bool RAGGED>
__device__ __forceinline__ RaggedTile skinny_tile(const SkinnyArgs& p, int tm, int lane) {
  if constexpr (RAGGED) return ragged_tile(p.seg, (int)p.num_experts, p.m, tm, 16 * MT, lane);
  const int64_t m0 = (int64_t)tm * 16 * MT;
  return RaggedTile{0, m0, p.m - m0 < 16 * MT ? p.m - m0 : 16 * MT};
}

__device__ __forceinline__ v8i load32(const uint8_t* p) {
  const uint4 x = reinterpret_cast<const uint4*>(p)[0], y = reinterpret_cast<const uint4*>(p)[1];
  return v8i{(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)y.x, (int)y.y, (int)y.z, (int)y.w};
}

// Sums of the waves' tiles (TILES of 16 x 16 each, lane (g, l16) holding row
// l16, columns 4g..4g+3) and the finished row pieces; tile t covers rows
// 16 (t / NT) and columns 16 (t % NT).
template <int WAVES, int TILES, int NT>
__device__ __forceinline__ void join_waves(const SkinnyArgs& p, float4* part, int64_t m0, int64_t rows, int64_t n0) {
  for (int q = threadIdx.x; q < TILES * 64; q += 64 * WAVES) {
    float4 s = part[q];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) {
      const float4 o = part[w * TILES * 64 + q];
      s.x += o.x;
      s.y += o.y;
      s.z += o.z;
      s.w += o.w;
    }
    const int t = q >> 6, r = 16 * (t / NT) + ((q & 63) >> 2), col = 16 * (t % NT) + 4 * (q & 3);
    if (r < rows) finish4(p, m0 + r, n0 + col, s);
  }
}

// U blocks' fragments and scales of one wave
template <int MT, int NT, int U>
struct SkinnyGroup {
  static constexpr int kBlocks = U;
  v8i b[U][NT], a[U][MT];
  float wb[U], wa[U][MT];
};

template <int MT, int NT, int kU, int WAVES, bool RAGGED>
__global__ __launch_bounds__(64 * WAVES) void skinny_rows_kernel(SkinnyArgs p, uint32_t tiles_n) {
  __shared__ float4 part[WAVES * MT * NT * 64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const uint32_t tm = blockIdx.x / tiles_n;
  const int64_t n0 = (int64_t)(blockIdx.x - tm * tiles_n) * 16 * NT;
  const RaggedTile rt = skinny_tile<MT, RAGGED>(p, (int)tm, lane);
  if (RAGGED && rt.e < 0) return;
  const int64_t K = p.k;
  const int nkb = (int)(K / BK);

  const uint8_t* const wrow = p.qb + ((int64_t)rt.e * p.n + n0 + l16) * K + 32 * g;
  const float* const wsc = p.sb + ((int64_t)rt.e * (p.n / 128) + n0 / 128) * nkb;
  const uint8_t* arow[MT];
  const float* asc[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const int64_t r = rt.m0 + min((int64_t)(16 * j + l16), rt.rows - 1);
    arow[j] = p.qa + r * K + 32 * g;
    asc[j] = p.sa + r * nkb;
  }
  auto load = [&](auto& f, int kb) {
#pragma unroll
    for (int u = 0; u < f.kBlocks; ++u) {
      const int k1 = kb + u * WAVES;
#pragma unroll
      for (int i = 0; i < NT; ++i) f.b[u][i] = load32(wrow + (int64_t)(16 * i) * K + (int64_t)k1 * BK);
      f.wb[u] = wsc[k1];
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        f.a[u][j] = load32(arow[j] + (int64_t)k1 * BK);
        f.wa[u][j] = asc[j][k1];
      }
    }
  };
  const v4f zero = {0.f, 0.f, 0.f, 0.f};
  v4f acc[MT][NT];
#pragma unroll
  for (int j = 0; j < MT; ++j)
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[j][i] = zero;
  auto multiply = [&](const auto& f) {
#pragma unroll
    for (int u = 0; u < f.kBlocks; ++u) {
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const float w = f.wa[u][j] * f.wb[u];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const v4f P = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(f.b[u][i], f.a[u][j], zero, 0, 0, 0, 0, 0, 0);
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[j][i][v] = __builtin_fmaf(w, P[v], acc[j][i][v]);
        }
      }
    }
  };
  constexpr int kStep = kU * WAVES;
  if (wave < nkb) {
    // whole groups, every load on its way before the first use, then block by
    // block (a group's loads past the end would cost as much as real ones)
    int kb = wave;
    for (; kb + (kU - 1) * WAVES < nkb; kb += kStep) {
      SkinnyGroup<MT, NT, kU> f;
      load(f, kb);
      __builtin_amdgcn_sched_barrier(0);
      multiply(f);
    }
    for (; kb < nkb; kb += WAVES) {
      SkinnyGroup<MT, NT, 1> f;
      load(f, kb);
      multiply(f);
    }
  }
#pragma unroll
  for (int j = 0; j < MT; ++j)
#pragma unroll
    for (int i = 0; i < NT; ++i)
      part[((wave * MT + j) * NT + i) * 64 + 4 * l16 + g] =
          make_float4(acc[j][i][0], acc[j][i][1], acc[j][i][2], acc[j][i][3]);
  __syncthreads();
  join_waves<WAVES, MT * NT, NT>(p, part, rt.m0, rt.rows, n0);
}

// b_layout 1.  Each LDS slab its own object, so that the compiler sees that a
// copy into one does not touch the other.
template <int WAVES, int IDX>
__device__ __forceinline__ uint8_t* skinny_slab() {
  __shared__ __attribute__((aligned(16))) uint8_t s[WAVES * 128 * BK];
  return s;
}

template <int MT, int WAVES, bool RAGGED>
__global__ __launch_bounds__(64 * WAVES) void skinny_cols_kernel(SkinnyArgs p, uint32_t tiles_n) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const uint32_t tm = blockIdx.x / tiles_n;
  const int64_t n0 = (int64_t)(blockIdx.x - tm * tiles_n) * 128;
  const RaggedTile rt = skinny_tile<MT, RAGGED>(p, (int)tm, lane);
  if (RAGGED && rt.e < 0) return;
  const int64_t K = p.k, N = p.n;
  const int nkb = (int)(K / BK);

  const __amdgpu_buffer_rsrc_t rb = make_rsrc(p.qb + (int64_t)rt.e * K * N + n0, K * N - n0);
  const float* const wsc = p.sb + (int64_t)rt.e * nkb * (N / 128) + n0 / 128;
  const uint8_t* arow[MT];
  const float* asc[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const int64_t r = rt.m0 + min((int64_t)(16 * j + l16), rt.rows - 1);
    arow[j] = p.qa + r * K + 32 * g;
    asc[j] = p.sa + r * nkb;
  }
  uint8_t* const s0 = skinny_slab<WAVES, 0>() + wave * 128 * BK;
  uint8_t* const s1 = skinny_slab<WAVES, 1>() + wave * 128 * BK;

  struct Side {
    v8i a[MT];
    float wa[MT], wb;
  };
  constexpr int kCopies = 16;                  // of 8 rows each
  auto issue = [&](uint8_t* slab, Side& f, int kb) {
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      const int row = 8 * i + (lane >> 3);
      dma16(rb, slab + i * 1024, (uint32_t)(row * N + (((lane & 7) ^ swz_ht(row)) << 4)), (uint32_t)kb * (uint32_t)(BK * N));
    }
    f.wb = wsc[(int64_t)kb * (N / 128)];
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      f.a[j] = load32(arow[j] + (int64_t)kb * BK);
      f.wa[j] = asc[j][kb];
    }
  };
  const v4f zero = {0.f, 0.f, 0.f, 0.f};
  v4f acc[MT][8];
#pragma unroll
  for (int j = 0; j < MT; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[j][i] = zero;
  auto multiply = [&](const uint8_t* slab, const Side& f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v2i part[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int row = 32 * g + 8 * q + (l16 >> 1);
        part[q] = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
            (__attribute__((address_space(3))) v2i*)(slab + swz_t(row, i) + ((l16 & 1) << 3)));
      }
      const v8i bf = {part[0].x, part[0].y, part[1].x, part[1].y, part[2].x, part[2].y, part[3].x, part[3].y};
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const v4f P = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bf, f.a[j], zero, 0, 0, 0, 0, 0, 0);
        const float w = f.wa[j] * f.wb;
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[j][i][v] = __builtin_fmaf(w, P[v], acc[j][i][v]);
      }
    }
  };
  // a wave waits for its own copies only: those of this slab are older than
  // the kCopies of the next one
  auto step = [&](int kb, uint8_t* slab, Side& f, uint8_t* next_slab, Side& next) {
    if (kb + WAVES < nkb) {
      __builtin_amdgcn_s_waitcnt(0xC07F);      // lgkmcnt(0): next_slab has been read
      asm volatile("" ::: "memory");
      issue(next_slab, next, kb + WAVES);
      wait_vmcnt<kCopies>();
    } else {
      wait_vmcnt<0>();
    }
    asm volatile("" ::: "memory");
    multiply(slab, f);
  };
  if (wave < nkb) {
    Side f0, f1;
    issue(s0, f0, wave);
    for (int kb = wave; kb < nkb; kb += 2 * WAVES) {
      step(kb, s0, f0, s1, f1);
      if (kb + WAVES < nkb) step(kb + WAVES, s1, f1, s0, f0);
    }
  }
  // the partial sums go where the slabs were, once every wave is done with its own
  __syncthreads();
  static_assert(MT * 8 * 1024 <= 128 * BK, "the sums fit where one slab of each wave was");
  float4* const part = reinterpret_cast<float4*>(skinny_slab<WAVES, 0>());
#pragma unroll
  for (int j = 0; j < MT; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      part[((wave * MT + j) * 8 + i) * 64 + 4 * l16 + g] =
          make_float4(acc[j][i][0], acc[j][i][1], acc[j][i][2], acc[j][i][3]);
  __syncthreads();
  join_waves<WAVES, MT * 8, 8>(p, part, rt.m0, rt.rows, n0);
}

// b_layout 0 on 16 MT x 16 NT tiles
template <int MT, int NT, int U, int WAVES, bool RAGGED>
static int launch_rows(const SkinnyArgs& a, hipStream_t s) {
  const int64_t tiles_m = RAGGED ? ragged_tiles(a.m, a.num_experts, 16 * MT) : (a.m + 16 * MT - 1) / (16 * MT);
  const int64_t tiles_n = a.n / (16 * NT);
  if (tiles_m * tiles_n > kMaxGrid) return FP8BS_ERR_SHAPE;
  hipLaunchKernelGGL((skinny_rows_kernel<MT, NT, U, WAVES, RAGGED>), dim3((unsigned)(tiles_m * tiles_n)), dim3(64 * WAVES),
                     0, s, a, (uint32_t)tiles_n);
  return launch_status();
}

// b_layout 1 on 16 MT x 128 tiles
template <int MT, int WAVES, bool RAGGED>
static int launch_cols(const SkinnyArgs& a, hipStream_t s) {
  const int64_t tiles_m = RAGGED ? ragged_tiles(a.m, a.num_experts, 16 * MT) : (a.m + 16 * MT - 1) / (16 * MT);
  const int64_t tiles_n = a.n / 128;
  if (tiles_m * tiles_n > kMaxGrid) return FP8BS_ERR_SHAPE;
  hipLaunchKernelGGL((skinny_cols_kernel<MT, WAVES, RAGGED>), dim3((unsigned)(tiles_m * tiles_n)), dim3(64 * WAVES), 0, s,
                     a, (uint32_t)tiles_n);
  return launch_status();
}

// Shapes, and what a round of one workgroup per CU takes (us over 56 blocks,
// measured, without the 4 us that a launch and its first loads take).  A CU
// sustains about 34 KB per us of requests that miss its L1, whatever number is
// in flight, so a round costs what its tiles load: 2 KB per block and row group
// or (b_layout 0) column group of 16.
struct SkinnyShape {
  int64_t mt, nt, cost;
};
constexpr SkinnyShape kRowShapes[] = {{1, 1, 7}, {1, 2, 11}, {2, 2, 16}, {2, 4, 21}};
constexpr SkinnyShape kColShapes[] = {{1, 8, 14}, {2, 8, 20}};

static int best_shape(const SkinnyArgs& a, int b_layout, int64_t cus, int64_t* cost) {
  const SkinnyShape* const s = b_layout == 0 ? kRowShapes : kColShapes;
  int best = 0;
  for (int i = 0; i < (b_layout == 0 ? 4 : 2); ++i) {
    const int64_t bm = 16 * s[i].mt;
    const int64_t tiles_m = a.seg ? ragged_tiles(a.m, a.num_experts, bm) : (a.m + bm - 1) / bm;
    const int64_t c = (tiles_m * (a.n / (16 * s[i].nt)) + cus - 1) / cus * s[i].cost;
    if (i == 0 || c < *cost) best = i, *cost = c;
  }
  return best;
}

int64_t skinny_cost(const SkinnyArgs& a, int b_layout, int64_t cus) {
  int64_t cost = 0;
  best_shape(a, b_layout, cus, &cost);
  return cost;
}

template <bool RAGGED>
static int launch_shape(const SkinnyArgs& a, int b_layout, int shape, hipStream_t s) {
  if (b_layout == 1) return shape == 0 ? launch_cols<1, 4, RAGGED>(a, s) : launch_cols<2, 4, RAGGED>(a, s);
  switch (shape) {
    case 0: return launch_rows<1, 1, 4, 8, RAGGED>(a, s);
    case 1: return launch_rows<1, 2, 4, 8, RAGGED>(a, s);
    case 2: return launch_rows<2, 2, 2, 8, RAGGED>(a, s);
    default: return launch_rows<2, 4, 2, 8, RAGGED>(a, s);
  }
}

int launch_skinny(const SkinnyArgs& a, int b_layout, int64_t cus, hipStream_t s) {
  int64_t cost = 0;
  const int shape = best_shape(a, b_layout, cus, &cost);
  return a.seg ? launch_shape<true>(a, b_layout, shape, s) : launch_shape<false>(a, b_layout, shape, s);
}

}  // namespace fp8bs
