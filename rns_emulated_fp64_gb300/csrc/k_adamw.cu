// One AdamW step over many tensors in one launch (per kMaxTensors tensors).
//
//   m <- b1 m + (1 - b1) g          v <- b2 v + (1 - b2) g^2
//   p <- p (1 - lr wd) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
//
// The moments are FP32, or 8-bit codes with one FP32 scale a block of 256
// elements (the block's largest magnitude a):
//   m = a sgn(c) (|c| / 127)^2, c int8        v = a (c / 255)^4, c uint8
// Powers, not a line: within a block, moments differ by orders of magnitude.
// The square keeps m down to a / 64516, the fourth power v down to 2.4e-10 a,
// that is sqrt(v), which divides, down to 1.5e-5 of its largest.  A positive v
// never becomes 0 (code 1 at least): the update it divides stays bounded.
//
// Bound by memory: every byte is read or written once, 28 bytes an element
// with FP32 parameters, gradients and moments.  A warp takes 256 elements (one
// 8-bit block), a lane 8 consecutive ones, all loads before the arithmetic:
// 8 (2 e_p + e_g + ...) bytes a lane are in flight, more than 100 KB an SM.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include <algorithm>

#include "os2_internal.cuh"

namespace {

constexpr int kBlock = 256;           // elements of a warp, and of an 8-bit scale
constexpr int kThreads = 256;
constexpr int kChunk = kBlock * kThreads / 32;
constexpr int kMaxTensors = 256;      // of one launch: 20 KB of kernel parameters

struct Tensors {
  int count;
  int vec[kMaxTensors / 32];          // bit: every pointer is aligned to 16 bytes
  unsigned first[kMaxTensors + 1];    // first chunk of each tensor; [count]: all chunks
  long long numel[kMaxTensors];
  void *p[kMaxTensors];
  const void *g[kMaxTensors];
  void *m[kMaxTensors], *v[kMaxTensors];
  float *ms[kMaxTensors], *vs[kMaxTensors];
};
static_assert(sizeof(Tensors) < 32000, "kernel parameter space");

struct Step {
  float b1, one_b1, b2, one_b2, decay, lr_c1, c2, eps;
};

template <int DT>
struct Elem;
template <>
struct Elem<OS2_F32> {
  using T = float;
  static __device__ __forceinline__ float get(T x) { return x; }
  static __device__ __forceinline__ T put(float x) { return x; }
};
template <>
struct Elem<OS2_BF16> {
  using T = __nv_bfloat16;
  static __device__ __forceinline__ float get(T x) { return __bfloat162float(x); }
  static __device__ __forceinline__ T put(float x) { return __float2bfloat16_rn(x); }
};
template <>
struct Elem<OS2_F16> {
  using T = __half;
  static __device__ __forceinline__ float get(T x) { return __half2float(x); }
  static __device__ __forceinline__ T put(float x) { return __float2half_rn(x); }
};

// 8 consecutive elements of which n exist, as vectors where the tensor allows
template <typename T>
__device__ __forceinline__ void load8(const T *src, T (&x)[8], int n, bool vec) {
  constexpr int W = sizeof(T) * 8 < 16 ? sizeof(T) * 8 : 16;  // bytes a load
  if (vec && n == 8) {
    union {
      T e[8];
      uint4 q[sizeof(T) * 8 >= 16 ? sizeof(T) / 2 : 1];
      uint2 d;
    } u;
    if (W == 8)
      u.d = *reinterpret_cast<const uint2 *>(src);
    else
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; i++) u.q[i] = reinterpret_cast<const uint4 *>(src)[i];
#pragma unroll
    for (int i = 0; i < 8; i++) x[i] = u.e[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++) x[i] = i < n ? src[i] : T(0.f);
  }
}
template <typename T>
__device__ __forceinline__ void store8(T *dst, const T (&x)[8], int n, bool vec) {
  if (vec && n == 8) {
    union {
      T e[8];
      uint4 q[sizeof(T) * 8 >= 16 ? sizeof(T) / 2 : 1];
      uint2 d;
    } u;
#pragma unroll
    for (int i = 0; i < 8; i++) u.e[i] = x[i];
    if (sizeof(T) == 1)
      *reinterpret_cast<uint2 *>(dst) = u.d;
    else
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; i++) reinterpret_cast<uint4 *>(dst)[i] = u.q[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++)
      if (i < n) dst[i] = x[i];
  }
}

// The values of codes; the products are rounded one by one, so that every
// reader of a state sees the same FP32 value.
__device__ __forceinline__ float m_value(int c, float a) {
  const float t = __fmul_rn((float)c, 1.0f / 127.0f);
  return __fmul_rn(a, __fmul_rn(t, fabsf(t)));
}
__device__ __forceinline__ float v_value(int c, float a) {
  float t = __fmul_rn((float)c, 1.0f / 255.0f);
  t = __fmul_rn(t, t);
  return __fmul_rn(a, __fmul_rn(t, t));
}
// The nearest code of m / a, of v / a (a > 0).
__device__ __forceinline__ int m_code(float m, float a) {
  const float q = rintf(__fmul_rn(__fsqrt_rn(__fdiv_rn(fabsf(m), a)), 127.0f));
  return (int)copysignf(q, m);
}
__device__ __forceinline__ int v_code(float v, float a) {
  const float q = rintf(__fmul_rn(__fsqrt_rn(__fsqrt_rn(__fdiv_rn(v, a))), 255.0f));
  return v > 0.f ? max((int)q, 1) : (int)q;
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

template <int PT, int GT, bool Q8>
__global__ void __launch_bounds__(kThreads) k_adamw(const __grid_constant__ Tensors ts,
                                                    const Step st) {
  using P = typename Elem<PT>::T;
  using G = typename Elem<GT>::T;
  // the last tensor whose first chunk is not past this one
  int lo = 0, hi = ts.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (ts.first[mid] <= blockIdx.x) lo = mid;
    else hi = mid;
  }
  const bool vec = ts.vec[lo >> 5] >> (lo & 31) & 1;
  const long long numel = ts.numel[lo];
  const int lane = threadIdx.x & 31;
  const long long block = (long long)(blockIdx.x - ts.first[lo]) * (kThreads / 32) + (threadIdx.x >> 5);
  const long long at = block * kBlock + lane * 8;
  if (block * kBlock >= numel) return;  // the whole warp
  const int n = (int)min(8LL, max(0LL, numel - at));

  P p8[8];
  G g8[8];
  P *pp = static_cast<P *>(ts.p[lo]) + at;
  load8(pp, p8, n, vec);
  load8(static_cast<const G *>(ts.g[lo]) + at, g8, n, vec);
  float m[8], v[8];
  if (!Q8) {
    load8(static_cast<const float *>(ts.m[lo]) + at, m, n, vec);
    load8(static_cast<const float *>(ts.v[lo]) + at, v, n, vec);
  } else {
    int8_t cm[8];
    uint8_t cv[8];
    load8(static_cast<const int8_t *>(ts.m[lo]) + at, cm, n, vec);
    load8(static_cast<const uint8_t *>(ts.v[lo]) + at, cv, n, vec);
    const float am = ts.ms[lo][block], av = ts.vs[lo][block];
#pragma unroll
    for (int i = 0; i < 8; i++) {
      m[i] = m_value(cm[i], am);
      v[i] = v_value(cv[i], av);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const float g = Elem<GT>::get(g8[i]);
    m[i] = __fadd_rn(__fmul_rn(m[i], st.b1), __fmul_rn(g, st.one_b1));
    v[i] = __fadd_rn(__fmul_rn(v[i], st.b2), __fmul_rn(__fmul_rn(g, g), st.one_b2));
    const float d = sqrtf(v[i] * st.c2) + st.eps;
    p8[i] = Elem<PT>::put(Elem<PT>::get(p8[i]) * st.decay - __fdividef(m[i] * st.lr_c1, d));
  }
  store8(pp, p8, n, vec);
  if (!Q8) {
    store8(static_cast<float *>(ts.m[lo]) + at, m, n, vec);
    store8(static_cast<float *>(ts.v[lo]) + at, v, n, vec);
  } else {
    float am = 0.f, av = 0.f;
#pragma unroll
    for (int i = 0; i < 8; i++) {
      am = fmaxf(am, i < n ? fabsf(m[i]) : 0.f);
      av = fmaxf(av, i < n ? v[i] : 0.f);
    }
    am = warp_max(am);
    av = warp_max(av);
    int8_t cm[8];
    uint8_t cv[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
      cm[i] = am > 0.f ? (int8_t)m_code(m[i], am) : 0;
      cv[i] = av > 0.f ? (uint8_t)v_code(v[i], av) : 0;
    }
    store8(static_cast<int8_t *>(ts.m[lo]) + at, cm, n, vec);
    store8(static_cast<uint8_t *>(ts.v[lo]) + at, cv, n, vec);
    if (lane == 0) {
      ts.ms[lo][block] = am;
      ts.vs[lo][block] = av;
    }
  }
}

__global__ void __launch_bounds__(kThreads)
    k_moments(long long numel, const int8_t *cm, const float *am, const uint8_t *cv,
              const float *av, float *m, float *v, bool vec) {
  const long long at = ((long long)blockIdx.x * kThreads + threadIdx.x) * 8;
  if (at >= numel) return;
  const int n = (int)min(8LL, numel - at);
  int8_t a[8];
  uint8_t b[8];
  load8(cm + at, a, n, vec);
  load8(cv + at, b, n, vec);
  const float sa = am[at / kBlock], sb = av[at / kBlock];
  float x[8], y[8];
#pragma unroll
  for (int i = 0; i < 8; i++) {
    x[i] = m_value(a[i], sa);
    y[i] = v_value(b[i], sb);
  }
  store8(m + at, x, n, vec);
  store8(v + at, y, n, vec);
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

size_t elem_size(int dt) { return dt == OS2_F32 ? 4 : 2; }

template <int PT, int GT>
void launch_pg(bool q8, const Tensors &t, const Step &st, cudaStream_t s) {
  const unsigned grid = t.first[t.count];
  if (q8) k_adamw<PT, GT, true><<<grid, kThreads, 0, s>>>(t, st);
  else k_adamw<PT, GT, false><<<grid, kThreads, 0, s>>>(t, st);
}
template <int PT>
void launch_p(int gt, bool q8, const Tensors &t, const Step &st, cudaStream_t s) {
  if (gt == OS2_F32) launch_pg<PT, OS2_F32>(q8, t, st, s);
  else if (gt == OS2_F16) launch_pg<PT, OS2_F16>(q8, t, st, s);
  else launch_pg<PT, OS2_BF16>(q8, t, st, s);
}
cudaError_t launch(int pt, int gt, bool q8, const Tensors &t, const Step &st, cudaStream_t s) {
  if (t.count == 0) return cudaSuccess;
  if (pt == OS2_F32) launch_p<OS2_F32>(gt, q8, t, st, s);
  else if (pt == OS2_F16) launch_p<OS2_F16>(gt, q8, t, st, s);
  else launch_p<OS2_BF16>(gt, q8, t, st, s);
  return cudaGetLastError();
}

}  // namespace

extern "C" os2_status os2_adamw(int count, const long long *numel, void *const *params,
                                const void *const *grads, void *const *exp_avg,
                                void *const *exp_avg_sq, float *const *exp_avg_scales,
                                float *const *exp_avg_sq_scales, int param_dtype, int grad_dtype,
                                int state_bits, double lr, double beta1, double beta2, double eps,
                                double weight_decay, long long step, void *stream) {
  if (count < 0 || step < 1 || (state_bits != 8 && state_bits != 32)) return OS2_ERR_INVALID_ARG;
  for (int dt : {param_dtype, grad_dtype})
    if (dt != OS2_F32 && dt != OS2_F16 && dt != OS2_BF16) return OS2_ERR_INVALID_ARG;
  if (!(lr >= 0) || !(beta1 >= 0 && beta1 < 1) || !(beta2 >= 0 && beta2 < 1) || !(eps >= 0) ||
      !isfinite(lr) || !isfinite(eps) || !isfinite(weight_decay))
    return OS2_ERR_INVALID_ARG;
  if (count == 0) return OS2_OK;
  const bool q8 = state_bits == 8;
  if (!numel || !params || !grads || !exp_avg || !exp_avg_sq ||
      (q8 && (!exp_avg_scales || !exp_avg_sq_scales)))
    return OS2_ERR_INVALID_ARG;
  const size_t ep = elem_size(param_dtype), eg = elem_size(grad_dtype), es = q8 ? 1 : 4;
  for (int i = 0; i < count; i++) {
    if (numel[i] < 0) return OS2_ERR_INVALID_ARG;
    if (numel[i] == 0) continue;
    if (!params[i] || !grads[i] || !exp_avg[i] || !exp_avg_sq[i] || !aligned(params[i], ep) ||
        !aligned(grads[i], eg) || !aligned(exp_avg[i], es) || !aligned(exp_avg_sq[i], es))
      return OS2_ERR_INVALID_ARG;
    if (q8 && (!exp_avg_scales[i] || !exp_avg_sq_scales[i] || !aligned(exp_avg_scales[i], 4) ||
               !aligned(exp_avg_sq_scales[i], 4)))
      return OS2_ERR_INVALID_ARG;
    if (numel[i] > (1LL << 40)) return OS2_ERR_UNSUPPORTED;
  }
  Step st;
  st.b1 = (float)beta1;
  st.one_b1 = (float)(1.0 - beta1);
  st.b2 = (float)beta2;
  st.one_b2 = (float)(1.0 - beta2);
  st.decay = (float)(1.0 - lr * weight_decay);
  st.lr_c1 = (float)(lr / (1.0 - pow(beta1, (double)step)));
  st.c2 = (float)(1.0 / (1.0 - pow(beta2, (double)step)));
  st.eps = (float)eps;
  Tensors t;
  t.count = 0;
  std::fill(t.vec, t.vec + kMaxTensors / 32, 0);
  t.first[0] = 0;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto flush = [&]() {
    const cudaError_t e = launch(param_dtype, grad_dtype, q8, t, st, s);
    t.count = 0;
    std::fill(t.vec, t.vec + kMaxTensors / 32, 0);
    return e;
  };
  for (int i = 0; i < count; i++) {
    if (numel[i] == 0) continue;
    const unsigned chunks = (unsigned)((numel[i] + kChunk - 1) / kChunk);  // at most 2^29
    if (t.count == kMaxTensors || (t.count && t.first[t.count] + chunks > (1u << 30)))
      if (flush() != cudaSuccess) return OS2_ERR_CUDA;
    const int c = t.count++;
    t.numel[c] = numel[i];
    t.p[c] = params[i];
    t.g[c] = grads[i];
    t.m[c] = exp_avg[i];
    t.v[c] = exp_avg_sq[i];
    t.ms[c] = q8 ? exp_avg_scales[i] : nullptr;
    t.vs[c] = q8 ? exp_avg_sq_scales[i] : nullptr;
    if (aligned(t.p[c], 16) && aligned(t.g[c], 16) && aligned(t.m[c], 16) && aligned(t.v[c], 16))
      t.vec[c >> 5] |= 1 << (c & 31);
    t.first[c + 1] = t.first[c] + chunks;
  }
  return flush() == cudaSuccess ? OS2_OK : OS2_ERR_CUDA;
}

extern "C" os2_status os2_adamw_moments(long long numel, const int8_t *exp_avg,
                                        const float *exp_avg_scale, const uint8_t *exp_avg_sq,
                                        const float *exp_avg_sq_scale, float *m, float *v,
                                        void *stream) {
  if (numel < 0) return OS2_ERR_INVALID_ARG;
  if (numel == 0) return OS2_OK;
  if (!exp_avg || !exp_avg_scale || !exp_avg_sq || !exp_avg_sq_scale || !m || !v ||
      !aligned(exp_avg_scale, 4) || !aligned(exp_avg_sq_scale, 4) || !aligned(m, 4) ||
      !aligned(v, 4))
    return OS2_ERR_INVALID_ARG;
  if (numel > (1LL << 40)) return OS2_ERR_UNSUPPORTED;
  const bool vec = aligned(exp_avg, 8) && aligned(exp_avg_sq, 8) && aligned(m, 16) && aligned(v, 16);
  const unsigned grid = (unsigned)((numel + kChunk - 1) / kChunk);
  k_moments<<<grid, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      numel, exp_avg, exp_avg_scale, exp_avg_sq, exp_avg_sq_scale, m, v, vec);
  return cudaGetLastError() == cudaSuccess ? OS2_OK : OS2_ERR_CUDA;
}
