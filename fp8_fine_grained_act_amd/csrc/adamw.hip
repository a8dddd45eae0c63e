// One AdamW step over many tensors.
//
//   m = b1 m + (1 - b1) g,   v = b2 v + (1 - b2) g^2          (g = grad * grad_scale)
//   p = p - lr (m / (1 - b1^t) / (sqrt(v / (1 - b2^t)) + eps) + decay p)
//
// The states are FP32, or E4M3 codes in groups of 128 consecutive elements with one FP32
// scale each (amax / 448, the library's tiles): m, and r = sqrt(v), whose range of
// 2^18 in a group is 2^36 of v.  r is rounded at random (upwards with the
// probability that its place between two codes gives): one step moves v by at most 1 - b2
// of itself downwards, less than half the codes' spacing, so rounding to nearest would
// never let r fall.  r > 0 never becomes code 0, which bounds m / sqrt(v).  The update
// of p uses the new m and v before they are rounded.
//
// m is rounded to nearest (half the error of a random rounding) where that lets it fall, and
// at random elsewhere.  Without a gradient a step takes (1 - b1) |m|, and to nearest a code of
// at most 0.5 / (1 - b1) units would stay as it is for ever while sqrt(v) falls: a weight without a gradient would
// move on at up to some lr a step (0.15 lr on average with b1 0.9, hundreds with 0.95 and one live weight in the
// group).  The subnormal codes have 0 to 7 units, all others 8 to 15, so
//   (1 - b1) 8 < 0.5    any code could be held: m is rounded at random everywhere
//   else                only subnormal ones: at random from a subnormal code to a subnormal code
// but for states that are still zero as a whole.  Without a gradient m is then zero after some 40 / (1 - b1) steps.  An
// ordinary code that is rounded to nearest may still rest up to 0.5 / (1 - b1) units beside a gradient that does not
// change at all (5 units of 8 to 15 with b1 0.9).
//
// Random bits: 32-bit mixes of (seed, step), of the tensor's number, of the element's place; 20
// of them stand for the fraction below an E4M3 step of r, 20 of their mix for m's.
//
// Bound by HBM: 30 bytes per element with an FP32 master and FP32 states, 18.1 with
// states in 8 bits.  32 lanes x 4 elements make a group, so FP32 arrays are read in whole
// 16-byte pieces and a group's amax stays in registers.  One quad per lane and many
// waves keep more of the memory busy than several quads per lane: eight 4096 x 7168
// weights with states in 8 bits take 677-688 us (6.2 TB/s) on one, 729 on two, 784 on four (all with the
// non-temporal hint; without it 5.4 TB/s), with FP32 states 1.18 ms (5.9 TB/s), 1.26, 1.31.  The table of tensors travels in
// the kernel's arguments, kPerLaunch tensors each: no device copy of it, nothing to
// keep alive under a captured graph.

#include <math.h>

#include "common.h"
#include "f32_codes.h"
#include "launch.h"

namespace fp8bs {

constexpr int kPerLaunch = 40;                 // tensors per launch: their table stays below 4 KB of arguments
constexpr int kAdamwBlock = 1024;              // elements per workgroup of 256 threads

struct AdamwTensor {
  void* param;
  float* master;
  const void* grad;
  void* avg;
  void* sq;
  float* avg_scales;
  float* root_scales;
  int64_t n;
  float decay;
  uint16_t param_bf16, grad_bf16;
};

struct AdamwArgs {
  AdamwTensor t[kPerLaunch];
  uint32_t block0[kPerLaunch];                 // first workgroup of each tensor
  int count;
  uint32_t number;                             // of the first tensor
  float lr, beta1, beta2, rest1, rest2, eps, grad_scale;   // rest = 1 - beta
  float unbias1, root2;                        // 1 / (1 - beta1^step), sqrt(1 / (1 - beta2^step))
  float log1, log2;                            // ln beta, for a step that is on the device
  float held;                                  // m's codes below this could be held by rounding to nearest
  uint32_t seed, step;
  const float* scalars;                        // lr, grad_scale, step on the device, or null
};
static_assert(sizeof(AdamwArgs) < 4096, "kernel arguments");

__device__ __forceinline__ uint32_t mix32(uint32_t x) {
  x ^= x >> 16;
  x *= 0xBB67AE85u;                            // odd: the leading fraction bits of sqrt(3)
  x ^= x >> 15;
  x *= 0x6A09E667u;                            // of sqrt(2)
  return x ^ (x >> 16);
}

// q in [0, 448] -> the E4M3 value below or above it: 20 random bits added below the last
// kept bit, the rest cut off.  Below 2^-6 the spacing is 2^-9, that of [2^-6, 2^-5), so q is
// moved there and back.
__device__ __forceinline__ float round_at_random(float q, uint32_t bits20) {
  const float move = q < 0x1p-6f ? 0x1p-6f : 0.0f;
  return __uint_as_float((__float_as_uint(q + move) + bits20) & ~0xFFFFFu) - move;
}

// sqrt(v) to nearest: the hardware's (1 ulp) and one correction by its remainder.  A v so
// small that the remainder would be subnormal is scaled by 2^64 first.
__device__ __forceinline__ float sqrt_rn(float v) {
  const bool low = v < 0x1p-64f;
  const float x = low ? v * 0x1p64f : v;
  const float s = __builtin_amdgcn_sqrtf(x);
  const float r = __builtin_fmaf(__builtin_fmaf(-s, s, x), 0.5f * __builtin_amdgcn_rcpf(s), s);
  return (s > 0.0f ? r : 0.0f) * (low ? 0x1p-32f : 1.0f);
}

__device__ __forceinline__ float max32_f32(float v) { return max_xor16_f32(max16_f32(v)); }

struct AdamwStep {
  float lr, grad_scale, unbias1, root2;        // root2 = sqrt(1 / (1 - beta2^step))
  uint32_t key;
};

// 4 consecutive elements per lane.  FULL: all inside the tensor; else elements from n on read as
// zero and are not written.  STREAM: non-temporal accesses (1: but for bf16 parameters' stores).
template <bool FULL, int STREAM>
struct Quad {
  int64_t n;
  template <typename T>
  __device__ __forceinline__ T get(const void* p) const {
    return STREAM ? __builtin_nontemporal_load(static_cast<const T*>(p)) : *static_cast<const T*>(p);
  }
  template <typename T, int FROM = 1>
  __device__ __forceinline__ void put(void* p, T v) const {
    if (STREAM >= FROM) __builtin_nontemporal_store(v, static_cast<T*>(p));
    else *static_cast<T*>(p) = v;
  }
  typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

  __device__ __forceinline__ void load(float (&x)[4], const float* src, int64_t i) const {
    if (FULL || i + 4 <= n) {
      const v4f w = get<v4f>(src + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = w[j];
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = i + j < n ? src[i + j] : 0.0f;
    }
  }
  __device__ __forceinline__ void load(float (&x)[4], const uint16_t* src, int64_t i) const {
    if (FULL || i + 4 <= n) {
      const u32x2 w = get<u32x2>(src + i);
      x[0] = bf16_lo(w.x); x[1] = bf16_hi(w.x); x[2] = bf16_lo(w.y); x[3] = bf16_hi(w.y);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = i + j < n ? __uint_as_float((uint32_t)src[i + j] << 16) : 0.0f;
    }
  }
  __device__ __forceinline__ uint32_t load_codes(const void* codes, int64_t i) const {
    const uint8_t* const src = static_cast<const uint8_t*>(codes);
    if (FULL || i + 4 <= n) return get<uint32_t>(src + i);
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) w |= i + j < n ? (uint32_t)src[i + j] << (8 * j) : 0u;
    return w;
  }
  __device__ __forceinline__ void store(float* dst, const float (&x)[4], int64_t i) const {
    if (FULL || i + 4 <= n) {
      put<v4f>(dst + i, v4f{x[0], x[1], x[2], x[3]});
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < n) dst[i + j] = x[j];
    }
  }
  __device__ __forceinline__ void store(uint16_t* dst, const float (&x)[4], int64_t i) const {
    const u32x2 w = {pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
    if (FULL || i + 4 <= n) {
      put<u32x2, 2>(dst + i, w);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < n) dst[i + j] = (uint16_t)((j < 2 ? w.x : w.y) >> (16 * (j & 1)));
    }
  }
  __device__ __forceinline__ void store_codes(void* codes, uint32_t w, int64_t i) const {
    uint8_t* const dst = static_cast<uint8_t*>(codes);
    if (FULL || i + 4 <= n) {
      put<uint32_t>(dst + i, w);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < n) dst[i + j] = (uint8_t)(w >> (8 * j));
    }
  }
};

// Codes of a group's m (to nearest; at random where the old code `md` and the new one are below `held`) and r (at random).
template <bool SLOW>
__device__ __forceinline__ uint2 state_codes(const float (&m)[4], const float (&r)[4], const F32Scale& mg, const F32Scale& rg,
                                             const float (&md)[4], float held, uint32_t random) {
  float mq[4], rq[4];
  uint32_t bits[4];
  bool some = false;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    bits[j] = mix32(random + (uint32_t)j * 0x9E3779B1u);
    mq[j] = f32_quotient<SLOW>(m[j], mg);
    some = some || (fabsf(md[j]) < held && fabsf(mq[j]) < held);
    // q is rounded to 2^-20 of a step, the random bits' unit, to nearest: no bias on average
    const float q = fminf(f32_quotient<SLOW>(r[j], rg), kE4M3Max);
    rq[j] = fmaxf(round_at_random(q, bits[j] >> 12), r[j] > 0.0f ? 0x1p-9f : 0.0f);
  }
  if (__ballot(some)) {                        // with b1 up to 0.9375 few waves hold such a value
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (fabsf(md[j]) < held && fabsf(mq[j]) < held)      // not a NaN
        mq[j] = copysignf(round_at_random(fminf(fabsf(mq[j]), kE4M3Max), mix32(bits[j] + 0x3C6EF373u) >> 12), mq[j]);
  }
  return make_uint2(code4_f32(mq[0], mq[1], mq[2], mq[3]), code4_f32(rq[0], rq[1], rq[2], rq[3]));
}

template <bool EIGHT, bool FULL, int STREAM>
__device__ __forceinline__ void adamw_block(const AdamwArgs& a, const AdamwTensor& t, const AdamwStep& st, int64_t i) {
  const Quad<FULL, STREAM> io{t.n};
  float p[4], g[4], m[4], v[4], md[4], ms, rs;
  uint32_t mc, rc;
  if (t.grad_bf16) io.load(g, static_cast<const uint16_t*>(t.grad), i);
  else io.load(g, static_cast<const float*>(t.grad), i);
  if (t.master) io.load(p, t.master, i);
  else if (t.param_bf16) io.load(p, static_cast<const uint16_t*>(t.param), i);
  else io.load(p, static_cast<const float*>(t.param), i);
  if (EIGHT) {
    mc = io.load_codes(t.avg, i);
    rc = io.load_codes(t.sq, i);
    ms = FULL || i < t.n ? t.avg_scales[i / kGroup] : 0.0f;
    rs = FULL || i < t.n ? t.root_scales[i / kGroup] : 0.0f;
  } else {
    io.load(m, static_cast<const float*>(t.avg), i);
    io.load(v, static_cast<const float*>(t.sq), i);
  }
  if (EIGHT) {
    typedef float v2f __attribute__((ext_vector_type(2)));
    const v2f m0 = __builtin_amdgcn_cvt_pk_f32_fp8((int)mc, false), m1 = __builtin_amdgcn_cvt_pk_f32_fp8((int)mc, true);
    const v2f r0 = __builtin_amdgcn_cvt_pk_f32_fp8((int)rc, false), r1 = __builtin_amdgcn_cvt_pk_f32_fp8((int)rc, true);
    const float mv[4] = {m0.x, m0.y, m1.x, m1.y}, rd[4] = {r0.x, r0.y, r1.x, r1.y};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      md[j] = mv[j];
      m[j] = md[j] * ms;
      const float r = rd[j] * rs;
      v[j] = r * r;
    }
  }
  float r[4], mt = 0.0f, rt = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float gv = g[j] * st.grad_scale;
    m[j] = m[j] * a.beta1 + gv * a.rest1;
    v[j] = v[j] * a.beta2 + (gv * gv) * a.rest2;
    r[j] = sqrt_rn(v[j]);
    // the quotient by v_rcp_f32: one ulp more than a division, of lr times a number near 1
    const float move = (m[j] * st.unbias1) * __builtin_amdgcn_rcpf(__builtin_fmaf(r[j], st.root2, a.eps));
    p[j] -= st.lr * (move + t.decay * p[j]);
    mt = fmaxf(mt, fabsf(m[j]));
    rt = fmaxf(rt, r[j]);
  }
  if (t.master) io.store(t.master, p, i);
  if (t.param_bf16) io.store(static_cast<uint16_t*>(t.param), p, i);
  else io.store(static_cast<float*>(t.param), p, i);
  if (!EIGHT) {
    io.store(static_cast<float*>(t.avg), m, i);
    io.store(static_cast<float*>(t.sq), v, i);
    return;
  }
  // elements past the end are zero here: their gradient and codes were read as zero
  mt = max32_f32(mt);
  rt = max32_f32(rt);
  // amax times 1 / 448, within 1.5 units of the last place of the quotient: the codes are x / s with this s, and a
  // chain of tensor operations that divides by a number multiplies by its reciprocal too, so that states
  // stay the same over many steps (an s one unit off moves some codes, and those the next step's s)
  const F32Scale mg = f32_scale_as(mt * (1.0f / kE4M3Max), mt), rg = f32_scale_as(rt * (1.0f / kE4M3Max), rt);
  const uint32_t random = st.key + (uint32_t)i * 0x9E3779B1u;
  const bool slow = __ballot(fmaxf(mg.up, rg.up) != 1.0f) != 0;
  const float held = ms > 0.0f ? a.held : 0.0f;     // states that are zero as a whole hold nothing
  const uint2 w = slow ? state_codes<true>(m, r, mg, rg, md, held, random) : state_codes<false>(m, r, mg, rg, md, held, random);
  io.store_codes(t.avg, w.x, i);
  io.store_codes(t.sq, w.y, i);
  if ((threadIdx.x & 31) == 0 && (FULL || i < t.n)) {
    t.avg_scales[i / kGroup] = mg.s;
    t.root_scales[i / kGroup] = rg.s;
  }
}

template <bool EIGHT, int STREAM>
__global__ __launch_bounds__(256) void adamw_kernel(AdamwArgs a) {
  // the workgroup's tensor: the last whose first workgroup is not past this one
  int k = 0;
  for (int hi = a.count; hi - k > 1;) {
    const int mid = (k + hi) >> 1;
    if (a.block0[mid] <= blockIdx.x) k = mid; else hi = mid;
  }
  const AdamwTensor& t = a.t[k];
  AdamwStep st{a.lr, a.grad_scale, a.unbias1, a.root2, 0};
  uint32_t step = a.step;
  if (a.scalars) {
    st.lr = a.scalars[0];
    st.grad_scale = a.scalars[1];
    const float n = a.scalars[2];
    step = (uint32_t)n;
    st.unbias1 = -1.0f / expm1f(n * a.log1);
    st.root2 = __builtin_sqrtf(-1.0f / expm1f(n * a.log2));
  }
  if (EIGHT) st.key = mix32(mix32(a.seed + step * 0x9E3779B1u) + (a.number + (uint32_t)k) * 0x3C6EF373u);
  const int64_t first = (int64_t)(blockIdx.x - a.block0[k]) * kAdamwBlock;
  if (first + kAdamwBlock <= t.n) adamw_block<EIGHT, true, STREAM>(a, t, st, first + 4 * threadIdx.x);
  else adamw_block<EIGHT, false, STREAM>(a, t, st, first + 4 * threadIdx.x);
}

}  // namespace fp8bs

using namespace fp8bs;

extern "C" int fp8bs_adamw_step(const fp8bs_adamw_tensor* tensors, int64_t num_tensors, double lr, double beta1, double beta2,
                                double eps, int64_t step, double grad_scale, const float* scalars, uint32_t seed, void* stream) {
  if (num_tensors < 0 || num_tensors > 0x7FFFFFFFLL) return FP8BS_ERR_SHAPE;
  if (num_tensors > 0 && !tensors) return FP8BS_ERR_NULL;
  // below 2^-126 the reciprocal of eps overflows: a weight that never had a gradient would become 0 times infinity
  if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || !(eps == 0.0 || eps >= 0x1p-126) ||
      (!scalars && step < 1))
    return FP8BS_ERR_FLAG;
  if (!aligned(scalars, 4)) return FP8BS_ERR_ALIGN;
  for (int64_t i = 0; i < num_tensors; ++i) {
    const fp8bs_adamw_tensor& t = tensors[i];
    if (t.param_bf16 < 0 || t.param_bf16 > 1 || t.grad_bf16 < 0 || t.grad_bf16 > 1 || (t.master && !t.param_bf16))
      return FP8BS_ERR_FLAG;
    if ((t.avg_scales == nullptr) != (t.root_scales == nullptr)) return FP8BS_ERR_NULL;
    if (t.n < 0 || t.n > 0xFFFFFFFFLL) return FP8BS_ERR_SHAPE;
    if (t.n > 0 && (!t.param || !t.grad || !t.avg || !t.sq)) return FP8BS_ERR_NULL;
    if (!aligned(t.param, 16) || !aligned(t.master, 16) || !aligned(t.grad, 16) || !aligned(t.avg, 16) || !aligned(t.sq, 16) ||
        !aligned(t.avg_scales, 4) || !aligned(t.root_scales, 4))
      return FP8BS_ERR_ALIGN;
  }
  AdamwArgs a{};
  a.lr = (float)lr;
  a.beta1 = (float)beta1;
  a.beta2 = (float)beta2;
  a.rest1 = (float)(1.0 - beta1);
  a.rest2 = (float)(1.0 - beta2);
  a.eps = (float)eps;
  a.grad_scale = (float)grad_scale;
  a.log1 = (float)log(beta1);
  a.log2 = (float)log(beta2);
  a.held = (1.0 - beta1) * 8.0 < 0.5 ? INFINITY : 0x1p-6f;
  if (!scalars) {
    a.unbias1 = (float)(1.0 / (1.0 - pow(beta1, (double)step)));
    a.root2 = (float)sqrt(1.0 / (1.0 - pow(beta2, (double)step)));
  }
  a.seed = seed;
  a.step = (uint32_t)step;
  a.scalars = scalars;
  // Accesses pass the caches where a launch touches more than half the last-level cache.  New bf16 parameters stay in
  // it, for the forward pass that reads them next, as long as all of the step's fit into that half: three 1536 x 7168
  // (66 MB) with FP32 states 172 -> 164 us, in 8 bits 101 -> 97; eight 4096 x 7168 (470 MB) 677 -> 696, where they do not.
  int64_t params = 0;
  for (int64_t i = 0; i < num_tensors; ++i)
    if (tensors[i].param_bf16) params += 2 * tensors[i].n;
  // launches of up to kPerLaunch tensors of one kind of state, in order
  int64_t i = 0;
  while (i < num_tensors) {
    if (tensors[i].n == 0) {
      ++i;
      continue;
    }
    const bool eight = tensors[i].avg_scales != nullptr;
    int64_t blocks = 0, bytes = 0;
    a.count = 0;
    a.number = (uint32_t)i;
    while (i < num_tensors && a.count < kPerLaunch && tensors[i].n > 0 && (tensors[i].avg_scales != nullptr) == eight) {
      const fp8bs_adamw_tensor& t = tensors[i++];
      const int64_t more = (t.n + kAdamwBlock - 1) / kAdamwBlock;
      if (blocks + more > kMaxGrid) {
        --i;
        break;
      }
      a.t[a.count] = AdamwTensor{t.param, t.master, t.grad, t.avg, t.sq, t.avg_scales, t.root_scales, t.n, t.weight_decay,
                                 (uint16_t)t.param_bf16, (uint16_t)t.grad_bf16};
      a.block0[a.count++] = (uint32_t)blocks;
      blocks += more;
      bytes += t.n * ((t.grad_bf16 ? 2 : 4) + (t.master ? 6 : t.param_bf16 ? 2 : 4) + (eight ? 2 : 8));
    }
    const dim3 grid((unsigned)blocks), block(256);
    hipStream_t s = (hipStream_t)stream;
    const int stream = bytes <= kStreamBytes ? 0 : params <= kStreamBytes ? 1 : 2;
    switch (3 * eight + stream) {
      case 0: hipLaunchKernelGGL((adamw_kernel<false, 0>), grid, block, 0, s, a); break;
      case 1: hipLaunchKernelGGL((adamw_kernel<false, 1>), grid, block, 0, s, a); break;
      case 2: hipLaunchKernelGGL((adamw_kernel<false, 2>), grid, block, 0, s, a); break;
      case 3: hipLaunchKernelGGL((adamw_kernel<true, 0>), grid, block, 0, s, a); break;
      case 4: hipLaunchKernelGGL((adamw_kernel<true, 1>), grid, block, 0, s, a); break;
      default: hipLaunchKernelGGL((adamw_kernel<true, 2>), grid, block, 0, s, a); break;
    }
    const int st = launch_status();
    if (st != FP8BS_OK) return st;
  }
  return FP8BS_OK;
}
