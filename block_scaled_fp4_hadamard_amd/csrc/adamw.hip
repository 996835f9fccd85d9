// One AdamW step over a list of float32 tensors, with first and second moments
// in 32 bits, or in 8 bits with a float32 scale for each block of 128 values.
// Every float32 operation below is rounded once, in this order:
//
//   g = RN(g * grad_scale)                                  (if one is given)
//   m = RN(RN(b1 m) + RN((1 - b1) g))
//   v = RN(RN(b2 v) + RN(RN((1 - b2) g) g))
//   d = RN(RN(RN(sqrt v) * c2) + eps)                       c2 = 1 / sqrt(1 - b2^t)
//   w = RN(RN(w * (1 - lr wd)) - RN(RN(m / d) * c1))        c1 = lr / (1 - b1^t)
//   copy = bf16 of w, to nearest even
//
// 8-bit moments: m is E4M3, v (never negative) E5M3, that is a float16 without
// its sign and its last 7 mantissa bits, top code 0xF7 (61440).  A block's
// scale is s = max(RN(amax * RN(1 / F)), 2^-126), F = 448 or 61440, and a code rounds
// y = RN(value * RN(1 / s)) by RTNE or stochastically; a v above 0 never
// rounds to code 0, so that a weight whose m is not 0 never meets d = eps.
// The exponent range is why v has a format of its own: a block's v spans twice
// the binades of its gradients.  Stochastic rounding is why the state can
// follow the gradients at all where 1 - b2 is far below half a step of 2^-4:
// round-to-nearest would return the old code forever.
//
// Memory-bound: 28 to 30 bytes per element with 32-bit moments, 16 to 18 with
// 8-bit ones.  218 million weights (a Llama block's linears) take 1208 us with
// 32-bit moments and fp32 gradients (5.4 TB/s) and 713 to 738 us with 8-bit ones,
// rounded either way (5.5).  A lane takes eight consecutive elements, so that 16
// lanes (a DPP row) hold a block of 128 and its maximum needs no LDS.  The tensors'
// addresses ride in the kernel's arguments, 48 to a launch, so a step needs no
// table in device memory; a workgroup takes 4096 elements.
//
// Vector accesses need every array of a tensor at 16 bytes (8-bit moments at 8).
// A tensor that is not so goes element by element, in 2.5 times the time: 2980 and
// 1810 us for the weights above; 100 odd tensors of 13.6 million weights, packed
// without padding, 194 us (32 bits) and 128 (8 bits) against 70 and 57.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include "mx_device.h"
#include "fp8_kernels.h"

// no multiply may be fused with an addition here: each operation rounds once
#pragma clang fp contract(off)

namespace mx {

namespace {

constexpr int kAwThreads = 512;
constexpr int kAwChunk = 8 * kAwThreads;
constexpr unsigned kAwGrid = 1024;         // 4 workgroups on each of the 256 CUs
constexpr unsigned kAwMost = 1u << 22;     // a grid holds fewer than 2^32 threads; further chunks are taken in turn

struct AdamwArgs {
  AdamwTensor t[kAdamwGroup];
  uint32_t end[kAdamwGroup];               // chunks of tensors 0 .. i
  uint8_t flags[kAdamwGroup];              // 1: bf16 gradient, 2: 16-byte vectors may be used
  int count, first;
  AdamwCoef coef;
  AdamwStep step;
};

// beta^t by repeated squaring, the same operations on the host and on the device
__host__ __device__ inline double power(double b, int64_t t) {
  double r = 1.0;
  for (uint64_t e = (uint64_t)t; e != 0; e >>= 1) {
    if (e & 1) r *= b;
    b *= b;
  }
  return r;
}

__host__ __device__ inline AdamwCoef coefficients(const AdamwStep& s, double lr, int64_t t) {
  AdamwCoef c;
  c.beta1 = (float)s.beta1;
  c.one_minus_beta1 = (float)(1.0 - s.beta1);
  c.beta2 = (float)s.beta2;
  c.one_minus_beta2 = (float)(1.0 - s.beta2);
  c.eps = (float)s.eps;
  c.c1 = (float)(lr / (1.0 - power(s.beta1, t)));
  c.c2 = (float)(1.0 / sqrt(1.0 - power(s.beta2, t)));
  c.keep = (float)(1.0 - lr * s.weight_decay);
  return c;
}

// the maximum over the 16 lanes of a DPP row, as unsigned bit patterns
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, false));    // l ^ 1
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, false));    // l ^ 2
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, false));   // 7 - l within 8
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, false));   // 15 - l within 16
  return v;
}

__device__ __forceinline__ float e4m3_value(uint32_t code) {
  return __builtin_amdgcn_cvt_f32_fp8((int)code, 0);
}
__device__ __forceinline__ float e5m3_value(uint32_t code) {
  return (float)__builtin_bit_cast(_Float16, (uint16_t)(code << 7));
}

// Magnitude code with 3 mantissa bits of |y|, least exponent EMIN: with E =
// max(floor(log2 |y|), EMIN), the code is 8 (E - EMIN) + |y| 2^(3 - E) rounded
// (0 .. 16), which carries into the next exponent by itself.  u holds the
// element's 16-bit draw in its top half: the truncated |y| 2^(19 - E) plus the
// draw, without the low 16 bits, rounds up iff floor(frac 2^16) + r >= 2^16.
template <int EMIN, int TOP, int ROUND>
__device__ __forceinline__ uint32_t code3(float y, uint32_t u) {
  const uint32_t bits = __float_as_uint(y) & 0x7FFFFFFFu;
  const int e = max((int)(bits >> 23) - 127, EMIN);
  const float a = __uint_as_float(bits);
  uint32_t k;
  if constexpr (ROUND == MX_ROUND_RTNE) k = (uint32_t)rintf(a * __uint_as_float((uint32_t)(130 - e) << 23));
  else k = ((uint32_t)(a * __uint_as_float((uint32_t)(146 - e) << 23)) + (u >> 16)) >> 16;
  return min(k + 8u * (uint32_t)(e - EMIN), (uint32_t)TOP);
}

// The eight codes of a lane's part of a block and the block's scale.
template <bool FIRST, int ROUND>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], uint64_t group, uint32_t stream, uint64_t seed,
                                         float& s) {
  uint32_t top = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  top = row_max(top);
  const bool bad = top >= 0x7F800000u;
  s = fmaxf(__uint_as_float(top) * (FIRST ? 1.0f / 448.0f : 1.0f / 61440.0f), 0x1p-126f);
  const float r = 1.0f / s;
  if (bad) s = __uint_as_float(0x7FC00000u);
  uint32_t u[8] = {};
  if constexpr (ROUND == MX_ROUND_SR) sr_draws<1>(group, stream, (uint32_t)seed, (uint32_t)(seed >> 32), u);
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float y = x[i] * r;
    uint32_t q;
    if constexpr (FIRST) {
      q = code3<-6, 0x7E, ROUND>(y, u[i]) | ((__float_as_uint(x[i]) >> 24) & 0x80u);
    } else {
      q = code3<-14, 0xF7, ROUND>(y, u[i]);
      if (x[i] > 0.0f) q = max(q, 1u);
    }
    w[i >> 2] |= (bad ? 0u : q) << (8 * (i & 3));
  }
  return uint2{w[0], w[1]};
}

template <int BITS, int ROUND>
__global__ void __launch_bounds__(kAwThreads) adamw_kernel(const AdamwArgs a) {
  AdamwCoef c = a.coef;
  uint64_t seed = a.step.seed;
  if (a.step.step_dev != nullptr || a.step.lr_dev != nullptr) {
    const int64_t step = a.step.step_dev ? *a.step.step_dev : a.step.step;
    c = coefficients(a.step, a.step.lr_dev ? (double)*a.step.lr_dev : a.step.lr, step);
    // the seed is fixed when a graph is captured: the device's step gives every replay draws of its own
    if (a.step.step_dev != nullptr) seed += (uint64_t)step;
  }
  // one value for the whole wave: in scalar registers, as the ten rounds' keys made of it (in vector registers, where the
  // loaded step would put it, 8-bit stochastic steps took 3% longer)
  seed = (uint64_t)__builtin_amdgcn_readfirstlane((uint32_t)(seed >> 32)) << 32 |
         (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)seed);
  const bool scaled = a.step.grad_scale != nullptr;
  const float gs = scaled ? *a.step.grad_scale : 1.0f;
  const uint32_t chunks = a.end[a.count - 1];
  int ti = 0;
  uint32_t base = 0;
  for (uint32_t chunk = blockIdx.x; chunk < chunks; chunk += gridDim.x) {
    while (chunk >= a.end[ti]) base = a.end[ti++];
    const AdamwTensor& t = a.t[ti];
    const int64_t at = (int64_t)(chunk - base) * kAwChunk + 8 * threadIdx.x;
    const int64_t left = t.n - at;                 // elements from here on (may be <= 0: the lane still joins maxima)
    const bool full = left >= 8 && (a.flags[ti] & 2) != 0;
    const int cnt = left >= 8 ? 8 : (left > 0 ? (int)left : 0);
    const bool gbf = (a.flags[ti] & 1) != 0;
    float w[8], g[8], m[8], v[8];
    float sm = 0.0f, sv = 0.0f;
    if constexpr (BITS == 8) {
      if (cnt > 0) {
        sm = t.m_scales[at >> 7];
        sv = t.v_scales[at >> 7];
      }
    }
    if (full) {
      auto load8 = [](const float* src, float (&o)[8]) {
        const float4 x = ((const float4*)src)[0], y = ((const float4*)src)[1];
        o[0] = x.x; o[1] = x.y; o[2] = x.z; o[3] = x.w;
        o[4] = y.x; o[5] = y.y; o[6] = y.z; o[7] = y.w;
      };
      load8(t.w + at, w);
      if (gbf) {
        const uint4 x = *(const uint4*)((const uint16_t*)t.g + at);
        const uint32_t d[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = __uint_as_float((i & 1) ? d[i >> 1] & 0xFFFF0000u : d[i >> 1] << 16);
      } else {
        load8((const float*)t.g + at, g);
      }
      if constexpr (BITS == 32) {
        load8((const float*)t.m + at, m);
        load8((const float*)t.v + at, v);
      } else {
        const uint2 mc = *(const uint2*)((const uint8_t*)t.m + at), vc = *(const uint2*)((const uint8_t*)t.v + at);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          m[i] = e4m3_value(((i < 4 ? mc.x : mc.y) >> (8 * (i & 3))) & 0xFFu) * sm;
          v[i] = e5m3_value(((i < 4 ? vc.x : vc.y) >> (8 * (i & 3))) & 0xFFu) * sv;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        w[i] = g[i] = m[i] = v[i] = 0.0f;
        if (i < cnt) {
          w[i] = t.w[at + i];
          g[i] = gbf ? __uint_as_float((uint32_t)((const uint16_t*)t.g)[at + i] << 16) : ((const float*)t.g)[at + i];
          if constexpr (BITS == 32) {
            m[i] = ((const float*)t.m)[at + i];
            v[i] = ((const float*)t.v)[at + i];
          } else {
            m[i] = e4m3_value(((const uint8_t*)t.m)[at + i]) * sm;
            v[i] = e5m3_value(((const uint8_t*)t.v)[at + i]) * sv;
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (scaled) g[i] *= gs;
      m[i] = m[i] * c.beta1 + g[i] * c.one_minus_beta1;
      v[i] = v[i] * c.beta2 + g[i] * c.one_minus_beta2 * g[i];
      const float d = sqrtf(v[i]) * c.c2 + c.eps;
      w[i] = w[i] * c.keep - m[i] / d * c.c1;
    }
    // a lane past the end must not move its block's maxima (0 / 0 above is NaN where eps is 0)
    if (cnt < 8) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i >= cnt) m[i] = v[i] = 0.0f;
    }
    uint2 mc, vc;
    if constexpr (BITS == 8) {
      const uint64_t group = (uint64_t)at >> 3;
      const uint32_t stream = 4u + 2u * (uint32_t)(a.first + ti);
      mc = encode8<true, ROUND>(m, group, stream, seed, sm);
      vc = encode8<false, ROUND>(v, group, stream + 1u, seed, sv);
      if (cnt > 0 && (threadIdx.x & 15) == 0) {
        t.m_scales[at >> 7] = sm;
        t.v_scales[at >> 7] = sv;
      }
    }
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
      typedef float f32x2_t __attribute__((ext_vector_type(2)));
      h[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t){w[2 * i], w[2 * i + 1]}, bf16x2_t));
    }
    if (full) {
      auto store8 = [](float* dst, const float (&o)[8]) {
        ((float4*)dst)[0] = float4{o[0], o[1], o[2], o[3]};
        ((float4*)dst)[1] = float4{o[4], o[5], o[6], o[7]};
      };
      store8(t.w + at, w);
      if (t.copy) *(uint4*)(t.copy + at) = uint4{h[0], h[1], h[2], h[3]};
      if constexpr (BITS == 32) {
        store8((float*)t.m + at, m);
        store8((float*)t.v + at, v);
      } else {
        *(uint2*)((uint8_t*)t.m + at) = mc;
        *(uint2*)((uint8_t*)t.v + at) = vc;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < cnt) {
          t.w[at + i] = w[i];
          if (t.copy) t.copy[at + i] = (uint16_t)(h[i >> 1] >> (16 * (i & 1)));
          if constexpr (BITS == 32) {
            ((float*)t.m)[at + i] = m[i];
            ((float*)t.v)[at + i] = v[i];
          } else {
            ((uint8_t*)t.m)[at + i] = (uint8_t)((i < 4 ? mc.x : mc.y) >> (8 * (i & 3)));
            ((uint8_t*)t.v)[at + i] = (uint8_t)((i < 4 ? vc.x : vc.y) >> (8 * (i & 3)));
          }
        }
    }
  }
}

// every array of the tensor may be read and written eight elements at a time
bool vectors(const AdamwTensor& t, int bits) {
  const uintptr_t wide = (uintptr_t)t.w | (uintptr_t)t.g | (uintptr_t)t.copy;
  const uintptr_t state = (uintptr_t)t.m | (uintptr_t)t.v;
  return wide % 16 == 0 && state % (bits == 8 ? 8 : 16) == 0;
}

}  // namespace

hipError_t launch_adamw(const AdamwTensor* tensors, const bool* grad_bf16, int count, int first, const AdamwStep& step,
                        int bits, int round, hipStream_t s) {
  AdamwArgs a;
  a.count = count;
  a.first = first;
  a.step = step;
  a.coef = coefficients(step, step.lr, step.step_dev || step.step < 1 ? 1 : step.step);
  uint32_t chunks = 0;
  for (int i = 0; i < kAdamwGroup; ++i) {
    a.t[i] = tensors[i < count ? i : count - 1];
    if (i < count) chunks += (uint32_t)((a.t[i].n + kAwChunk - 1) / kAwChunk);
    a.end[i] = chunks;
    const bool bf = grad_bf16[i < count ? i : count - 1];
    a.flags[i] = (uint8_t)((bf ? 1 : 0) | (vectors(a.t[i], bits) ? 2 : 0));
  }
  if (chunks == 0) return hipSuccess;
  // one workgroup a chunk (5.4 TB/s on a block's weights against 5.0 with a resident grid); where each workgroup forms
  // the coefficients itself, a resident grid, so that the few thousand instructions of it are paid once
  const bool form = step.step_dev != nullptr || step.lr_dev != nullptr;
  const unsigned most = form ? kAwGrid : kAwMost;
  const dim3 g(chunks < most ? chunks : most), b(kAwThreads);
  if (bits == 32) hipLaunchKernelGGL((adamw_kernel<32, MX_ROUND_RTNE>), g, b, 0, s, a);
  else if (round == MX_ROUND_SR) hipLaunchKernelGGL((adamw_kernel<8, MX_ROUND_SR>), g, b, 0, s, a);
  else hipLaunchKernelGGL((adamw_kernel<8, MX_ROUND_RTNE>), g, b, 0, s, a);
  return hipGetLastError();
}

}  // namespace mx
