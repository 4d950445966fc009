// The activations of a linear layer and their slopes (k_linear.cu, k_linear_few.cu), in FP32.
//
//   gelu       z Phi(z), Phi the normal distribution by the rational approximation 7.1.26
//              of Abramowitz and Stegun (off by less than 1.5e-7 in erf): an exponential, a
//              reciprocal and five multiply-adds; relu, silu = z s(z), s(z) = 1 / (1 + e^-z)
//   gelu_tanh  z (1 + tanh u) / 2 = z s(2 u),  u = sqrt(2 / pi) (z + 0.044715 z^3)
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "os2_internal.cuh"

namespace os2act {

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcpf(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kL2e = 1.4426950408889634f;

// 1 / (1 + e^-x)
__device__ __forceinline__ float sigmoid(float x) { return rcpf(1.f + ex2f(-kL2e * x)); }

// Phi(z), and e^(-z^2 / 2)
__device__ __forceinline__ float normal(float z, float &e) {
  const float x = fabsf(z) * 0.70710678118654752f;
  e = ex2f(-0.5f * kL2e * z * z);
  const float t = rcpf(fmaf(0.3275911f, x, 1.f));
  const float p = t * fmaf(t, fmaf(t, fmaf(t, fmaf(t, 1.061405429f, -1.453152027f), 1.421413741f), -0.284496736f), 0.254829592f);
  const float tail = 0.5f * p * e;  // Phi(-|z|)
  return z < 0.f ? tail : 1.f - tail;
}

// z <- act(z).  The choice stands outside the loops: inside, the entries would run one after
// another (a tile of 256 x 256 took 14 us longer).
template <int N>
__device__ __forceinline__ void values(float (&z)[N], int act) {
  float e;
  switch (act) {
    case OS2_ACT_RELU:
#pragma unroll
      for (int i = 0; i < N; i++) z[i] = z[i] < 0.f ? 0.f : z[i];
      break;
    case OS2_ACT_GELU:
#pragma unroll
      for (int i = 0; i < N; i++) z[i] *= normal(z[i], e);
      break;
    case OS2_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < N; i++) z[i] *= sigmoid(1.5957691216057308f * fmaf(0.044715f * z[i] * z[i], z[i], z[i]));
      break;
    case OS2_ACT_SILU:
#pragma unroll
      for (int i = 0; i < N; i++) z[i] *= sigmoid(z[i]);
      break;
  }
}

// z held to [-100, 100], two 16-bit entries at once: a slope is 0 or 1 in FP32 from far less on, and
// beyond it z^3 would overflow, or an infinite z (a rounded one, in FP16 from 65520 on) meet a zero.
// NaN stays.  (In FP32, entry by entry, a gradient of eight tokens took 23.5 us in place of 23.1.)
template <bool BF16>
__device__ __forceinline__ uint32_t near0(uint32_t z) {
  if (BF16) {
    const __nv_bfloat162 far = __bfloat162bfloat162(__float2bfloat16_rn(100.f)), x = reinterpret_cast<const __nv_bfloat162 &>(z),
                         y = __hmax2_nan(__hmin2_nan(x, far), __hneg2(far));
    return reinterpret_cast<const uint32_t &>(y);
  }
  const __half2 far = __half2half2(__float2half_rn(100.f)), x = reinterpret_cast<const __half2 &>(z),
                y = __hmax2_nan(__hmin2_nan(x, far), __hneg2(far));
  return reinterpret_cast<const uint32_t &>(y);
}

// d <- d act'(z), z as near0 gives it.
template <int N>
__device__ __forceinline__ void slopes(float (&d)[N], const float (&z)[N], int act) {
  switch (act) {
    case OS2_ACT_RELU:
#pragma unroll
      for (int i = 0; i < N; i++) d[i] = z[i] > 0.f ? d[i] : 0.f;
      break;
    case OS2_ACT_GELU:
#pragma unroll
      for (int i = 0; i < N; i++) {
        float e;
        const float phi = normal(z[i], e);
        d[i] *= fmaf(z[i] * 0.3989422804014327f, e, phi);
      }
      break;
    case OS2_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < N; i++) {
        const float s = sigmoid(1.5957691216057308f * fmaf(0.044715f * z[i] * z[i], z[i], z[i]));
        d[i] *= fmaf(z[i] * s * (1.f - s), 1.5957691216057308f * fmaf(0.134145f * z[i], z[i], 1.f), s);
      }
      break;
    case OS2_ACT_SILU:
#pragma unroll
      for (int i = 0; i < N; i++) {
        const float s = sigmoid(z[i]);
        d[i] *= s * fmaf(z[i], 1.f - s, 1.f);
      }
      break;
  }
}

}  // namespace os2act
