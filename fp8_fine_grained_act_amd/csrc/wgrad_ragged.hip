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
// kT rows by BM (dy) and BN (x) columns is copied as it lies straight into LDS
// (buffer_load ... lds); the fragments, which need consecutive t per lane, are
// gathered with ds_read_b64_tr_b16: in a group of 16 lanes that each point at 4
// bf16, lane i receives element i mod 4 of the words of lanes 4r + i div 4, r =
// 0..3; lane j therefore points at row t = 8g + j div 4 (+ 4 for the second
// read), columns 4 (j mod 4) of the tile's 16, and lane i ends with column i at
// t = 8g .. 8g + 7.
// LDS rows are units of 32 bytes (one 16-column tile each); unit u of row t is
// stored at u ^ f(t), f = (t & 3) | ((t >> 1) & 4), so the 8 rows that 32 lanes
// read together (t = 0..3 and 8..11 of a half slab) fall on 64 distinct banks.
// Rows past the segment's end read as zeros (buffer range check).
//
// Workgroups are persistent (one per CU, tiles w, w + G, ...) and their waves
// have one role each.  Four copy waves keep a ring of three slabs filled across
// tile boundaries.  The MFMA waves only read LDS, multiply and store: they wait
// for no memory operation.  (With every wave copying, a wave's copies wait behind its
// stores: 32 experts of 4096 x 7168 with 512 rows each took 1.59 ms; 128 x 64 patches
// on four MFMA waves 1.52 ms.)
//
// What bounds it: those 32 experts take 1.39 ms (0.69 PFLOP/s, 3.8 GB written); the
// copies alone 0.61 ms (18 TB/s out of the L2s), LDS reads and MFMAs alone 0.73 ms
// (1.3 PFLOP/s; 1.5 over long segments), the stores alone 0.69 ms (5.4 TB/s into HBM),
// copies and stores without MFMAs 1.23 ms: the two hardly overlap, and that is the
// bound.  Three of a wave's eight pieces of a tile therefore stay in registers and
// leave one per slab under the next tile's MFMAs: 32 experts of 2048 x 2048 with 300
// rows 152 -> 141 us, the sizes above 1.41 -> 1.39 ms.
// Barrier u says that slab u has landed and that slab u - 1 has been read; the
// copy waves then refill the stage of slab u - 1 with slab u + 2, and the MFMA
// waves pass it in the last groups of slab u - 1, reading the first fragments
// of slab u under the MFMAs that are left.

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
  int64_t num_experts, total_rows, m, n;
  float* c;
  int64_t tiles_m, tiles_n;
  int accumulate;
};

constexpr int kT = 64;                         // rows of a slab: two MFMAs' contraction
constexpr int kRing = 3;
constexpr int kHeld = 3;                       // of a tile's 8 pieces per wave, stored under the next tile; 4 would spill
constexpr int kBand = 4;                       // tile rows of a band: tiles walk down it, so the strips of dy
                                               // and x that are read at a time stay few

__device__ __forceinline__ int tswz(int t) { return (t & 3) | ((t >> 1) & 4); }

// SPLIT: each segment's slabs in gridDim.y parts, c holds [gridDim.y][num_experts][m][n].
template <int BM, int BN, bool STREAM, bool SPLIT = false>
__global__ __launch_bounds__(64 * (BM / 64 * (BN / 64) + 4)) void ragged_wgrad_kernel(RaggedWgradArgs p) {
  constexpr int WAVES_N = BN / 64, MW = BM / 64 * WAVES_N, TM = 4, TN = 4;      // 64 x 64 patches
  constexpr int kSlabA = kT * BM * 2, kSlab = kSlabA + kT * BN * 2;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kRing * kSlab];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const uint32_t tiles_m = (uint32_t)p.tiles_m, tiles_n = (uint32_t)p.tiles_n, tiles = tiles_m * tiles_n;
  const uint32_t total = tiles * (uint32_t)p.num_experts, G = gridDim.x;
  const int cap = (int)p.total_rows;
  // Workgroups are dealt to the 8 XCDs in turn; each round of G tiles gives every
  // XCD a run of G / 8 consecutive ones, a block of kBand tile rows whose strips
  // of dy and x its L2 holds.
  const uint32_t first = G % 8 == 0 ? blockIdx.x % 8 * (G / 8) + blockIdx.x / 8 : blockIdx.x;

  struct Tile {
    uint32_t i, e;                             // i >= total: none
    int64_t m0, n0;
    int s0, rows, slabs;
  };
  auto tile_at = [&](uint32_t i) {
    Tile t;
    t.i = i;
    t.e = i / tiles;
    const uint32_t idx = i - t.e * tiles;
    const uint32_t band = idx / (kBand * tiles_n), r = idx - band * kBand * tiles_n;
    const uint32_t height = min((uint32_t)kBand, tiles_m - band * kBand);
    t.m0 = (int64_t)(band * kBand + r % height) * BM;
    t.n0 = (int64_t)(r / height) * BN;
    t.s0 = min(max(p.seg[t.e], 0), cap);
    t.rows = max(0, min(max(p.seg[t.e + 1], 0), cap) - t.s0);
    t.slabs = (t.rows + kT - 1) / kT;
    if (SPLIT) {                               // part blockIdx.y of the segment's slabs
      const uint32_t all = (uint32_t)t.slabs, y = blockIdx.y;
      const int lo = __builtin_amdgcn_readfirstlane((int)(y * all / gridDim.y));
      const int hi = __builtin_amdgcn_readfirstlane((int)((y + 1) * all / gridDim.y));
      t.rows = min(t.rows, hi * kT) - lo * kT;
      t.s0 += lo * kT;
      t.slabs = hi - lo;
    }
    return t;
  };
  // the first tile from i on that has rows
  auto live_tile = [&](uint32_t i) {
    Tile t;
    t.i = i;
    t.slabs = 0;
    for (; i < total; i += G) {
      t = tile_at(i);
      if (t.slabs > 0) return t;
    }
    t.i = total;
    return t;
  };
  auto barrier = [&]() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  if (wave >= MW) {
    // ======================= copy waves ==========================================
    // A copy fills 1 KB: 2 (BM = 256) or 4 rows.  This wave copies q = c + 4i of a
    // slab's; a row's swizzle depends on i only through t's bit 3.
    const int c = wave - MW;
    constexpr int A_CP = kSlabA / 4096, B_CP = kT * BN * 2 / 4096, kCopies = A_CP + B_CP;
    auto lane_off = [&](int width, int64_t ld, int i) -> uint32_t {
      const int chunks = width / 8, t = (c + 4 * i) * (64 / chunks) + lane / chunks, pc = lane % chunks;
      return (uint32_t)((int64_t)(lane / chunks) * ld * 2 + (((((pc >> 1) ^ tswz(t)) << 1) | (pc & 1)) << 4));
    };
    const uint32_t off_a[2] = {lane_off(BM, p.ldy, 0), lane_off(BM, p.ldy, 1)};
    const uint32_t off_b[2] = {lane_off(BN, p.ldx, 0), lane_off(BN, p.ldx, 1)};
    auto issue = [&](const Tile& t, int s, int stage) {
      const int64_t t0 = (int64_t)s * kT, left = t.rows - t0;
      const int64_t mw = min((int64_t)BM, p.m - t.m0), nw = min((int64_t)BN, p.n - t.n0);
      const __amdgpu_buffer_rsrc_t ra = make_rsrc(p.dy + (t.s0 + t0) * p.ldy + t.m0, ((left - 1) * p.ldy + mw) * 2);
      const __amdgpu_buffer_rsrc_t rb = make_rsrc(p.x + (t.s0 + t0) * p.ldx + t.n0, ((left - 1) * p.ldx + nw) * 2);
      uint8_t* const dst = lds + stage * kSlab;
#pragma unroll
      for (int i = 0; i < A_CP; ++i) {
        const int q = c + 4 * i;
        dma16(ra, dst + q * 1024, off_a[i & 1], (uint32_t)(q * (512 / BM)) * (uint32_t)(p.ldy * 2));
      }
#pragma unroll
      for (int i = 0; i < B_CP; ++i) {
        const int q = c + 4 * i;
        dma16(rb, dst + kSlabA + q * 1024, off_b[i & 1], (uint32_t)(q * (512 / BN)) * (uint32_t)(p.ldx * 2));
      }
    };
    Tile t = live_tile(first);
    int s = 0, stage = 0, ahead = 0;           // the next slab to issue; slabs issued and not yet published
    auto issue_next = [&]() {
      if (t.i >= total) return;
      issue(t, s, stage);
      stage = stage == kRing - 1 ? 0 : stage + 1;
      ++ahead;
      if (++s == t.slabs) {
        t = live_tile(t.i + G);
        s = 0;
      }
    };
    issue_next();
    issue_next();
    while (ahead > 0) {
      if (ahead == 2) wait_vmcnt<kCopies>();
      else wait_vmcnt<0>();
      barrier();
      --ahead;
      issue_next();
    }
    return;
  }

  // ========================= MFMA waves ==========================================
  const int wm = wave / WAVES_N, wn = wave % WAVES_N;
  // LDS offsets of the lane's words in slab 0: the first of the wave's four tiles
  // (tile j at ^ (j << 5)), first read of k step 0; the second read lies 4 rows on,
  // k step 1 32 rows on
  const int tl = 8 * g + (l16 >> 2);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_ptr_t*)lds;
  uint32_t at_a = (uint32_t)(tl * BM * 2 + (((TM * wm) ^ tswz(tl)) << 5) + ((l16 & 3) << 3));
  uint32_t at_b = (uint32_t)(kSlabA + tl * BN * 2 + (((TN * wn) ^ tswz(tl)) << 5) + ((l16 & 3) << 3));
  auto frag = [&](uint32_t at, int row_bytes, int step) -> v8bf {
    v4i16 h[2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
      h[u] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (__attribute__((address_space(3))) v4i16*)(uintptr_t)(at + (uint32_t)((32 * step + 4 * u) * row_bytes)));
    typedef short v8i16 __attribute__((ext_vector_type(8)));
    const v8i16 f = {h[0][0], h[0][1], h[0][2], h[0][3], h[1][0], h[1][1], h[1][2], h[1][3]};
    return __builtin_bit_cast(v8bf, f);
  };
  auto frag_a = [&](uint32_t stage, int j, int step) { return frag((at_a ^ (j << 5)) + (stage + lds0), BM * 2, step); };
  auto frag_b = [&](uint32_t stage, int k, int step) { return frag((at_b ^ (k << 5)) + (stage + lds0), BN * 2, step); };

  v4f acc[TN][TM];
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  };
  clear();

  // A patch is stored in 8 pieces of 16 rows by 32 columns (tiles j, k and k + 1):
  // lanes 8 apart swap one tile's values for the other's, so that a store of 8
  // rows writes whole 128-byte lines.
  auto c_rsrc = [&](const Tile& t) {
    return make_rsrc(p.c + (SPLIT ? blockIdx.y * p.num_experts + t.e : (int64_t)t.e) * p.m * p.n + t.m0 * p.n, min((int64_t)BM, p.m - t.m0) * p.n * 4);
  };
  const bool hi = l16 >= 8;
  auto swap = [&](int j, int k, v4f (&o)[2]) {
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const float send = hi ? acc[k][j][v] : acc[k + 1][j][v];
      const float got = __uint_as_float(dpp_shuffle<0x128>(__float_as_uint(send)));
      o[0][v] = hi ? got : acc[k][j][v];
      o[1][v] = hi ? acc[k + 1][j][v] : got;
    }
  };
  // rows past m end behind the range, columns past n are sent there
  auto put = [&](__amdgpu_buffer_rsrc_t rc, int64_t n0, int j, int k, int h, v4f o) {
    const int row = 64 * wm + 16 * j + (l16 & 7) + 8 * h;
    const uint32_t col = (uint32_t)n0 + 64 * wn + 16 * k + (hi ? 16 : 0) + 4 * g;
    const uint32_t off = col < (uint32_t)p.n ? ((uint32_t)row * (uint32_t)p.n + col) * 4u : 0xFFFFFFF0u;
    if (p.accumulate) {
      const v4f old = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(rc, (int)off, 0, 0));
#pragma unroll
      for (int v = 0; v < 4; ++v) o[v] += old[v];
    }
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, o), rc, (int)off, 0, STREAM ? 2 : 0);
  };
  auto store = [&](const Tile& t, int u0) {
    const __amdgpu_buffer_rsrc_t rc = c_rsrc(t);
#pragma unroll
    for (int j = 0; j < TM; ++j) {
#pragma unroll
      for (int k = 0; k < TN; k += 2) {
        if (2 * j + k / 2 < u0) continue;
        v4f o[2];
        swap(j, k, o);
        put(rc, t.n0, j, k, 0, o[0]);
        put(rc, t.n0, j, k, 1, o[1]);
      }
    }
  };
  // The first kHeld pieces of a finished tile wait in registers and are stored one
  // per slab under the next tile's MFMAs.
  v4f held[kHeld][2];
  int pending = 0;
  Tile held_t;
  auto hold = [&](const Tile& t) {
#pragma unroll
    for (int u = 0; u < kHeld; ++u) swap(u / 2, u % 2 * 2, held[u]);
    pending = kHeld;
    held_t = t;
  };
  auto drip = [&]() {
    if (pending == 0) return;
    --pending;
    const __amdgpu_buffer_rsrc_t rc = c_rsrc(held_t);
#pragma unroll
    for (int u = 0; u < kHeld; ++u)
      if (pending == u) {
        put(rc, held_t.n0, u / 2, u % 2 * 2, 0, held[u][0]);
        put(rc, held_t.n0, u / 2, u % 2 * 2, 1, held[u][1]);
      }
  };

  // Groups of one A fragment and its four MFMAs; A fragments are read kAhead
  // groups ahead of them (the other wave of the SIMD covers what that leaves).
  constexpr int kGroups = 2 * TM, kAhead = 1;
  v8bf bf[2][TN], af[kAhead + 1];
  uint32_t stage = 0;                          // byte offset of the current slab's stage
  auto slab = [&](bool more) {
    asm("" : "+v"(at_a), "+v"(at_b));          // the four tiles' offsets are not kept in registers
    const uint32_t next = stage == (kRing - 1) * kSlab ? 0 : stage + kSlab;
#pragma unroll
    for (int q = 0; q < kGroups; ++q) {
      if (q == 5) drip();
      const int step = q / TM, j = q % TM, n = q + kAhead;
      if (q < TN) bf[1][q] = frag_b(stage, q, 1);
      if (n < kGroups) {
        af[n % (kAhead + 1)] = frag_a(stage, n % TM, n / TM);
      } else if (more) {
        if (n == kGroups) {
          __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the slab has been read
          barrier();
#pragma unroll
          for (int k = 0; k < TN; ++k) bf[0][k] = frag_b(next, k, 0);
        }
        af[n % (kAhead + 1)] = frag_a(next, n - kGroups, 0);
      }
#pragma unroll
      for (int k = 0; k < TN; ++k)
        acc[k][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[step][k], af[q % (kAhead + 1)], acc[k][j], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
    stage = next;
  };

  Tile live = live_tile(first);
  if (live.i < total) {
    barrier();                                 // slab 0 landed
#pragma unroll
    for (int k = 0; k < TN; ++k) bf[0][k] = frag_b(0, k, 0);
#pragma unroll
    for (int n = 0; n < kAhead; ++n) af[n] = frag_a(0, n, 0);
  }
  for (uint32_t i = first; i < total; i += G) {
    if (i == live.i) {
      const Tile t = live;
      live = live_tile(i + G);
      for (int s = 0; s < t.slabs; ++s) slab(s + 1 < t.slabs || live.i < total);
      while (pending) drip();
      if (live.i < total && !p.accumulate) {
        hold(t);
        store(t, kHeld);
      } else {
        store(t, 0);
      }
      clear();
    } else if (!p.accumulate) {
      store(tile_at(i), 0);                    // no rows: zeros
    }
  }
}

// c (+)= the parts' sums in order; with accumulate, an empty segment's matrix is not touched.
__global__ __launch_bounds__(256) void wgrad_join_kernel(const float* __restrict__ parts, int64_t splits,
                                                         const int32_t* __restrict__ seg, int64_t num_experts, int cap,
                                                         int64_t mn, float* __restrict__ c, int accumulate) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4, e = blockIdx.y;
  if (i >= mn) return;
  if (accumulate && min(max(seg[e + 1], 0), cap) <= min(max(seg[e], 0), cap)) return;
  const float* src = parts + e * mn + i;
  float4 s = *reinterpret_cast<const float4*>(src);
  for (int64_t k = 1; k < splits; ++k) {
    const float4 o = *reinterpret_cast<const float4*>(src + k * num_experts * mn);
    s.x += o.x;
    s.y += o.y;
    s.z += o.z;
    s.w += o.w;
  }
  float4* const dst = reinterpret_cast<float4*>(c + e * mn + i);
  if (accumulate) {
    const float4 o = *dst;
    s.x += o.x;
    s.y += o.y;
    s.z += o.z;
    s.w += o.w;
  }
  *dst = s;
}

// Parts of the contraction: 1 unless the tiles fill at most half the CUs and the mean
// segment is 48 slabs or more; then as many as fill the CUs, each with 8 slabs or more of
// the mean segment, at most 32.  (The rows' distribution is on the device.)  A slab
// takes 0.7 us there, the stream-ordered workspace and the joining launch about 15: one
// expert of 512 x 512 with 4096 rows 47 -> 27 us, of 256 x 256 with 32768 rows 323 -> 32,
// of 2048 x 2048 with 4096 rows (two parts) 51 either way; shorter ones lose (four
// of 512 x 512 with 2048 rows 27.6 against 27, one of 1536 x 1536 with 1024 rows 19
// against 30).
static int64_t wgrad_splits(const RaggedWgradArgs& a, int64_t tiles, int64_t cus) {
  const int64_t slabs = a.total_rows / (a.num_experts * kT);
  if (2 * tiles > cus || slabs < 48) return 1;
  int64_t s = cus / tiles;
  if (s > slabs / 8) s = slabs / 8;
  return s < 32 ? s : 32;
}

template <int BM, int BN>
static int launch_ragged_wgrad(RaggedWgradArgs a, int64_t cus, hipStream_t s) {
  a.tiles_m = (a.m + BM - 1) / BM;
  a.tiles_n = (a.n + BN - 1) / BN;
  const int64_t total = a.num_experts * a.tiles_m * a.tiles_n;
  if (total > kMaxGrid) return FP8BS_ERR_SHAPE;
  const int64_t splits = wgrad_splits(a, total, cus), mn = a.m * a.n;
  const dim3 b(64 * (BM / 64 * (BN / 64) + 4));
  if (splits > 1) {
    void* ws = nullptr;
    if (hipMallocAsync(&ws, (size_t)(splits * a.num_experts * mn * 4), s) == hipSuccess) {
      RaggedWgradArgs parts = a;
      parts.c = static_cast<float*>(ws);
      parts.accumulate = 0;
      hipLaunchKernelGGL((ragged_wgrad_kernel<BM, BN, false, true>), dim3((unsigned)total, (unsigned)splits), b, 0, s, parts);
      int st = launch_status();
      if (st == FP8BS_OK) {
        hipLaunchKernelGGL(wgrad_join_kernel, dim3((unsigned)((mn / 4 + 255) / 256), (unsigned)a.num_experts), dim3(256), 0,
                           s, parts.c, splits, a.seg, a.num_experts, (int)a.total_rows, mn, a.c, a.accumulate);
        st = launch_status();
      }
      if (hipFreeAsync(ws, s) != hipSuccess && st == FP8BS_OK) st = FP8BS_ERR_LAUNCH;
      return st;
    }
    (void)hipGetLastError();                   // no memory for the parts: unsplit
  }
  const dim3 g((unsigned)(total < cus ? total : cus));
  if (a.num_experts * a.m * a.n * 4 > kStreamBytes)
    hipLaunchKernelGGL((ragged_wgrad_kernel<BM, BN, true>), g, b, 0, s, a);
  else
    hipLaunchKernelGGL((ragged_wgrad_kernel<BM, BN, false>), g, b, 0, s, a);
  return launch_status();
}

}  // namespace fp8bs

using namespace fp8bs;

extern "C" int fp8bs_grouped_wgrad_ragged(const uint16_t* dy, int64_t ldy, const uint16_t* x, int64_t ldx,
                                          const int32_t* seg_offsets, int64_t num_experts, int64_t total_rows,
                                          int64_t m, int64_t n, float* c, int accumulate, void* stream) {
  if (!seg_offsets || !c || (total_rows > 0 && (!dy || !x))) return FP8BS_ERR_NULL;
  if (accumulate != 0 && accumulate != 1) return FP8BS_ERR_FLAG;
  if (num_experts < 1 || num_experts > 65536 || total_rows < 0 || total_rows > 0x3FFFFFFFLL || m <= 0 || n <= 0 ||
      m % 8 || n % 8 || ldy < m || ldx < n || ldy > (1 << 24) || ldx > (1 << 24) || n > (1 << 21))
    return FP8BS_ERR_SHAPE;
  if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(c, 16) || !aligned(seg_offsets, 4) || ldy % 8 || ldx % 8)
    return FP8BS_ERR_ALIGN;
  RaggedWgradArgs a{dy, ldy, x, ldx, seg_offsets, num_experts, total_rows, m, n, c, 0, 0, accumulate};
  return launch_ragged_wgrad<256, 128>(a, cu_count(), (hipStream_t)stream);
}
