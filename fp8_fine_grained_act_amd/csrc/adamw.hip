// One AdamW step over many tensors.
//
//   m = b1 m + (1 - b1) g,   v = b2 v + (1 - b2) g^2          (g = grad * grad_scale)
//   p = p - lr (m / (1 - b1^t) / (sqrt(v / (1 - b2^t)) + eps) + decay p)
//
// The states are FP32, or E4M3 codes in groups of 128 consecutive elements with one FP32
// scale each (amax / 448, the library's tiles): m, and r = sqrt(v), whose range of
// 2^18 in a group is 2^36 of v.  m is rounded to nearest: a step moves it by (1 - b1)(g -
// m), far more than the codes' spacing.  r is rounded at random (upwards with the
// probability that its place between two codes gives): one step moves v by at most 1 - b2
// of itself downwards, less than half the codes' spacing, so rounding to nearest would
// never let r fall.  r > 0 never becomes code 0, which bounds m / sqrt(v).  The update
// of p uses the new m and v before they are rounded.
//
// Random bits: 32-bit mixes of (seed, step), of the tensor's number, of the element's place; 20
// of them stand for the fraction below an E4M3 step.
//
// Bound by HBM: 30 bytes per element with an FP32 master and FP32 states, 18.1 with
// states in 8 bits.  32 lanes x 4 elements make a group, so FP32 arrays are read in whole
// 16-byte pieces and a group's amax stays in registers.  The table of tensors travels in
// the kernel's arguments, kPerLaunch tensors each: no device copy of it, nothing to
// keep alive under a captured graph.

#include <math.h>

#include "common.h"
#include "launch.h"

namespace fp8bs {

constexpr int kPerLaunch = 40;                 // tensors per launch: their table stays below 4 KB of arguments
constexpr int kAdamwUnroll = 4;
constexpr int kAdamwBlock = 1024 * kAdamwUnroll;   // elements per workgroup of 256 threads

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
  float unbias1, unbias2;                      // 1 / (1 - beta^step)
  float log1, log2;                            // ln beta, for a step that is on the device
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

// q in [0, 448] -> the E4M3 value below or above it: 20 random bits added below the
// last kept bit, the rest cut off; below 2^-6, where the spacing is 2^-9, on the
// fixed-point value.
__device__ __forceinline__ float round_at_random(float q, uint32_t bits20) {
  const float up = __uint_as_float((__float_as_uint(q) + bits20) & ~0xFFFFFu);
  const float low = floorf(q * 512.0f + (float)bits20 * 0x1p-20f) * 0x1p-9f;
  return fminf(q >= 0x1p-6f ? up : low, kE4M3Max);
}

__device__ __forceinline__ float max32_f32(float v) { return max_xor16_f32(max16_f32(v)); }

template <bool EIGHT>
__global__ __launch_bounds__(256) void adamw_kernel(AdamwArgs a) {
  // the workgroup's tensor: the last whose first workgroup is not past this one
  int k = 0;
  for (int hi = a.count; hi - k > 1;) {
    const int mid = (k + hi) >> 1;
    if (a.block0[mid] <= blockIdx.x) k = mid; else hi = mid;
  }
  const AdamwTensor& t = a.t[k];
  float lr = a.lr, gs = a.grad_scale, u1 = a.unbias1, u2 = a.unbias2;
  uint32_t step = a.step;
  if (a.scalars) {
    lr = a.scalars[0];
    gs = a.scalars[1];
    const float n = a.scalars[2];
    step = (uint32_t)n;
    u1 = -1.0f / expm1f(n * a.log1);
    u2 = -1.0f / expm1f(n * a.log2);
  }
  uint32_t key = 0;
  if (EIGHT) key = mix32(mix32(a.seed + step * 0x9E3779B1u) + (a.number + (uint32_t)k) * 0x3C6EF373u);
  const int64_t base = (int64_t)(blockIdx.x - a.block0[k]) * kAdamwBlock + 4 * threadIdx.x;

  float p[kAdamwUnroll][4], g[kAdamwUnroll][4], m[kAdamwUnroll][4], v[kAdamwUnroll][4];
  float ms[kAdamwUnroll], rs[kAdamwUnroll];
  uint32_t mc[kAdamwUnroll], rc[kAdamwUnroll];
  auto load4 = [](float (&x)[4], const float* src, int64_t i, int64_t n) {
    if (i + 4 <= n) {
      const float4 w = *reinterpret_cast<const float4*>(src + i);
      x[0] = w.x; x[1] = w.y; x[2] = w.z; x[3] = w.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = i + j < n ? src[i + j] : 0.0f;
    }
  };
  auto load4_bf16 = [](float (&x)[4], const uint16_t* src, int64_t i, int64_t n) {
    if (i + 4 <= n) {
      const uint2 w = *reinterpret_cast<const uint2*>(src + i);
      x[0] = bf16_lo(w.x); x[1] = bf16_hi(w.x); x[2] = bf16_lo(w.y); x[3] = bf16_hi(w.y);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = i + j < n ? __uint_as_float((uint32_t)src[i + j] << 16) : 0.0f;
    }
  };
  auto load4_code = [](const uint8_t* src, int64_t i, int64_t n) -> uint32_t {
    if (i + 4 <= n) return *reinterpret_cast<const uint32_t*>(src + i);
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) w |= i + j < n ? (uint32_t)src[i + j] << (8 * j) : 0u;
    return w;
  };
#pragma unroll
  for (int u = 0; u < kAdamwUnroll; ++u) {
    const int64_t i = base + 1024 * u;
    if (t.grad_bf16) load4_bf16(g[u], static_cast<const uint16_t*>(t.grad), i, t.n);
    else load4(g[u], static_cast<const float*>(t.grad), i, t.n);
    if (t.master) load4(p[u], t.master, i, t.n);
    else if (t.param_bf16) load4_bf16(p[u], static_cast<const uint16_t*>(t.param), i, t.n);
    else load4(p[u], static_cast<const float*>(t.param), i, t.n);
    if (EIGHT) {
      mc[u] = load4_code(static_cast<const uint8_t*>(t.avg), i, t.n);
      rc[u] = load4_code(static_cast<const uint8_t*>(t.sq), i, t.n);
      ms[u] = i < t.n ? t.avg_scales[i / kGroup] : 0.0f;
      rs[u] = i < t.n ? t.root_scales[i / kGroup] : 0.0f;
    } else {
      load4(m[u], static_cast<const float*>(t.avg), i, t.n);
      load4(v[u], static_cast<const float*>(t.sq), i, t.n);
    }
  }
  auto store4 = [](float* dst, const float (&x)[4], int64_t i, int64_t n) {
    if (i + 4 <= n) {
      *reinterpret_cast<float4*>(dst + i) = make_float4(x[0], x[1], x[2], x[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < n) dst[i + j] = x[j];
    }
  };
#pragma unroll
  for (int u = 0; u < kAdamwUnroll; ++u) {
    const int64_t i = base + 1024 * u;
    if (EIGHT) {
      typedef float v2f __attribute__((ext_vector_type(2)));
      const v2f m0 = __builtin_amdgcn_cvt_pk_f32_fp8((int)mc[u], false), m1 = __builtin_amdgcn_cvt_pk_f32_fp8((int)mc[u], true);
      const v2f r0 = __builtin_amdgcn_cvt_pk_f32_fp8((int)rc[u], false), r1 = __builtin_amdgcn_cvt_pk_f32_fp8((int)rc[u], true);
      const float md[4] = {m0.x, m0.y, m1.x, m1.y}, rd[4] = {r0.x, r0.y, r1.x, r1.y};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        m[u][j] = md[j] * ms[u];
        const float r = rd[j] * rs[u];
        v[u][j] = r * r;
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float gv = g[u][j] * gs;
      m[u][j] = m[u][j] * a.beta1 + gv * a.rest1;
      v[u][j] = v[u][j] * a.beta2 + (gv * gv) * a.rest2;
      const float move = (m[u][j] * u1) / (__builtin_sqrtf(v[u][j] * u2) + a.eps);
      p[u][j] -= lr * (move + t.decay * p[u][j]);
    }
    if (t.master) store4(t.master, p[u], i, t.n);
    if (t.param_bf16) {
      uint16_t* const dst = static_cast<uint16_t*>(t.param) + i;
      const uint2 w = make_uint2(pack_bf16(p[u][0], p[u][1]), pack_bf16(p[u][2], p[u][3]));
      if (i + 4 <= t.n) {
        *reinterpret_cast<uint2*>(dst) = w;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (i + j < t.n) dst[j] = (uint16_t)((j < 2 ? w.x : w.y) >> (16 * (j & 1)));
      }
    } else {
      store4(static_cast<float*>(t.param), p[u], i, t.n);
    }
    if (!EIGHT) {
      store4(static_cast<float*>(t.avg), m[u], i, t.n);
      store4(static_cast<float*>(t.sq), v[u], i, t.n);
      continue;
    }
    // elements past the end are zero here: their gradient and codes were read as zero
    float r[4], mt = 0.0f, rt = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      r[j] = __builtin_sqrtf(v[u][j]);
      mt = fmaxf(mt, fabsf(m[u][j]));
      rt = fmaxf(rt, r[j]);
    }
    const F32Scale mg = f32_scale(max32_f32(mt)), rg = f32_scale(max32_f32(rt));
    float mq[4], rq[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      mq[j] = f32_quotient<true>(m[u][j], mg);
      const uint32_t bits = mix32(key + (uint32_t)(i + j) * 0x9E3779B1u) >> 12;
      const float q = round_at_random(f32_quotient<true>(r[j], rg), bits);
      rq[j] = r[j] > 0.0f ? fmaxf(q, 0x1p-9f) : 0.0f;
    }
    const uint32_t mw = code4_f32(mq[0], mq[1], mq[2], mq[3]), rw = code4_f32(rq[0], rq[1], rq[2], rq[3]);
    uint8_t* const md = static_cast<uint8_t*>(t.avg) + i;
    uint8_t* const rd = static_cast<uint8_t*>(t.sq) + i;
    if (i + 4 <= t.n) {
      *reinterpret_cast<uint32_t*>(md) = mw;
      *reinterpret_cast<uint32_t*>(rd) = rw;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < t.n) {
          md[j] = (uint8_t)(mw >> (8 * j));
          rd[j] = (uint8_t)(rw >> (8 * j));
        }
    }
    if ((threadIdx.x & 31) == 0 && i < t.n) {
      t.avg_scales[i / kGroup] = mg.s;
      t.root_scales[i / kGroup] = rg.s;
    }
  }
}

}  // namespace fp8bs

using namespace fp8bs;

extern "C" int fp8bs_adamw_step(const fp8bs_adamw_tensor* tensors, int64_t num_tensors, double lr, double beta1, double beta2,
                                double eps, int64_t step, double grad_scale, const float* scalars, uint32_t seed, void* stream) {
  if (num_tensors < 0 || num_tensors > 0x7FFFFFFFLL) return FP8BS_ERR_SHAPE;
  if (num_tensors > 0 && !tensors) return FP8BS_ERR_NULL;
  if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || !(eps >= 0.0) || (!scalars && step < 1))
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
  if (!scalars) {
    a.unbias1 = (float)(1.0 / (1.0 - pow(beta1, (double)step)));
    a.unbias2 = (float)(1.0 / (1.0 - pow(beta2, (double)step)));
  }
  a.seed = seed;
  a.step = (uint32_t)step;
  a.scalars = scalars;
  // launches of up to kPerLaunch tensors of one kind of state, in order
  int64_t i = 0;
  while (i < num_tensors) {
    if (tensors[i].n == 0) {
      ++i;
      continue;
    }
    const bool eight = tensors[i].avg_scales != nullptr;
    int64_t blocks = 0;
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
    }
    if (eight) hipLaunchKernelGGL((adamw_kernel<true>), dim3((unsigned)blocks), dim3(256), 0, (hipStream_t)stream, a);
    else hipLaunchKernelGGL((adamw_kernel<false>), dim3((unsigned)blocks), dim3(256), 0, (hipStream_t)stream, a);
    const int st = launch_status();
    if (st != FP8BS_OK) return st;
  }
  return FP8BS_OK;
}
