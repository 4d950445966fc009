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
// with FP32 parameters, gradients and moments.  A warp takes 256 elements (an 8-bit
// block), a lane 8 consecutive ones, all loads before the arithmetic: more than 100
// KB an SM in flight with FP32 moments.  With 8-bit ones the bytes are fewer and
// the arithmetic (some 75 instructions an element) weighs as much as they do: six
// CTAs an SM rather than five are worth 6 %, conversions are additions of 2^23 and
// 1.5 2^23 instead of I2F and F2I, which run at a quarter of the rate, and the
// exact rounding is taken only where the fast one is in doubt.
// Measured: FP32 moments, FP32 parameters, BF16 gradients, 268 M elements 979 us (7.1
// TB/s); 8-bit moments, BF16 both, 150 M elements 387 us (3.9 TB/s: instruction issue,
// 77 % busy); 24 tensors of 0.3 M in all 3.8 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include <algorithm>

#include "os2_internal.cuh"

namespace {

constexpr int kBlock = 256;           // elements of a warp, and of an 8-bit scale
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = kBlock * kWarps;  // of a CTA
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

// The values of codes c (as FP32); the products are rounded one by one, so that
// every reader of a state sees the same FP32 value.
__device__ __forceinline__ float m_value(float c, float a) {
  const float t = __fmul_rn(c, 1.0f / 127.0f);
  return __fmul_rn(a, __fmul_rn(t, fabsf(t)));
}
// x: 2^23 + c; the product c / 255 in one step, exactly as if c were multiplied
// (2^23 times the constant is a shift of it).
__device__ __forceinline__ float v_value(float x, float a) {
  float t = __fmaf_rn(x, 1.0f / 255.0f, -8388608.0f * (1.0f / 255.0f));
  t = __fmul_rn(t, t);
  return __fmul_rn(a, __fmul_rn(t, t));
}
// Codes of eight moments from their bytes in two words.
__device__ __forceinline__ void m_values(uint32_t lo, uint32_t hi, float a, float (&x)[8]) {
  lo ^= 0x80808080u;  // c + 128
  hi ^= 0x80808080u;
  constexpr float less = 8388608.0f + 128.0f;
#define M4(w, o)                                                                      \
  x[o] = m_value(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440)) - less, a);     \
  x[o + 1] = m_value(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7441)) - less, a); \
  x[o + 2] = m_value(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7442)) - less, a); \
  x[o + 3] = m_value(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7443)) - less, a);
  M4(lo, 0)
  M4(hi, 4)
#undef M4
}
__device__ __forceinline__ void v_values(uint32_t lo, uint32_t hi, float a, float (&x)[8]) {
#define V4(w, o)                                                               \
  x[o] = v_value(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440)), a);     \
  x[o + 1] = v_value(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7441)), a); \
  x[o + 2] = v_value(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7442)), a); \
  x[o + 3] = v_value(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7443)), a);
  V4(lo, 0)
  V4(hi, 4)
#undef V4
}

// The nearest code of m / a, of v / a (a > 0): rint(127 sqrt(|m| / a)) and
// rint(255 sqrt(sqrt(v / a))), every operation correctly rounded.  Those take some
// 60 instructions an element and would bound the kernel, so the approximate
// instructions decide first, with 127^2 / a and 255^4 / a as factors and roots within
// 2^-23: the root is off by less than 2.7e-5 and the fourth root by less than 6.1e-5,
// the correctly rounded ones themselves by less than 2e-5 and 4.2e-5.  Only where one
// lies nearer than 6e-5 or 1.5e-4 to a tie (one element in 2000) both take the exact
// way, asked for once every four elements.  The limits are negative, for every
// element to take it, where the factors or the quotients could leave the normal
// numbers.  A code is the low byte of its FP32 value plus 1.5 2^23.
__device__ __forceinline__ float sqrt_fast(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kRound = 12582912.0f;  // 1.5 * 2^23
struct Encode {
  float am, av;     // the block's largest magnitudes
  float rm, rv;     // 1 / am, 1 / av, or 0
  float dm, dv;     // limits of the distance from the rounded value
};
__device__ __forceinline__ Encode encode_with(float am, float av) {
  Encode e;
  e.am = am;
  e.av = av;
  const bool fm = am > 1e-26f && am < 1e30f, fv = av > 1e-26f && av < 1e30f;
  e.rm = fm ? __fmul_rn(__frcp_rn(am), 127.0f * 127.0f) : 0.f;
  e.rv = fv ? __fmul_rn(__frcp_rn(av), 255.0f * 255.0f * 255.0f * 255.0f) : 0.f;
  // a block of zeros: every code is 0 without a division by 0
  e.dm = fm ? 0.5f - 6e-5f : am > 0.f ? -1.f : 1.f;
  e.dv = fv ? 0.5f - 1.5e-4f : av > 0.f ? -1.f : 1.f;
  return e;
}
// Codes of four moments in the low bytes of cm and cv: the sum of a negative number
// and 1.5 2^23 ends in its two's complement.
__device__ __forceinline__ void codes(const Encode &e, const float *m, const float *v,
                                      uint32_t (&cm)[4], uint32_t (&cv)[4]) {
  float off_m = 0.f, off_v = 0.f;  // furthest from the rounded value
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const float x = copysignf(sqrt_fast(fabsf(m[i]) * e.rm), m[i]);
    const float y = sqrt_fast(sqrt_fast(v[i] * e.rv));
    const float p = x + kRound, q = y + kRound;
    off_m = fmaxf(off_m, fabsf(x - (p - kRound)));
    off_v = fmaxf(off_v, fabsf(y - (q - kRound)));
    cm[i] = __float_as_uint(p);
    cv[i] = __float_as_uint(q);
  }
  // (where the block holds Inf or NaN its limits are negative: whatever its codes, its
  // values are not numbers)
  if (off_m > e.dm || off_v > e.dv) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const float x = sqrt_fast(fabsf(m[i]) * e.rm), y = sqrt_fast(sqrt_fast(v[i] * e.rv));
      if (fabsf(x - rintf(x)) > e.dm || fabsf(y - rintf(y)) > e.dv) {
        if (e.am > 0.f)
          cm[i] = __float_as_uint(
              copysignf(rintf(__fmul_rn(__fsqrt_rn(__fdiv_rn(fabsf(m[i]), e.am)), 127.0f)), m[i]) +
              kRound);
        if (e.av > 0.f)
          cv[i] = __float_as_uint(
              rintf(__fmul_rn(__fsqrt_rn(__fsqrt_rn(__fdiv_rn(v[i], e.av))), 255.0f)) + kRound);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; i++)  // a positive v never becomes 0
    cv[i] = __viaddmax_u32(min(__float_as_uint(v[i]), 1u), 0x4B400000u, cv[i]);
}

template <int PT, int GT, bool Q8>
__global__ void __launch_bounds__(kThreads, Q8 ? 6 : 1) k_adamw(const __grid_constant__ Tensors ts,
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
  const long long block = (long long)(blockIdx.x - ts.first[lo]) * kWarps + (threadIdx.x >> 5);
  const long long at = block * kBlock + lane * 8;
  if (block * kBlock >= numel) return;  // the whole warp
  const int n = (int)min(8LL, max(0LL, numel - at));

  // elements past the end are zeros in, and stay zeros: they change no maximum
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
    union {
      uint8_t b[8];
      uint32_t w[2];
    } cm, cv;
    load8(static_cast<const uint8_t *>(ts.m[lo]) + at, cm.b, n, vec);
    load8(static_cast<const uint8_t *>(ts.v[lo]) + at, cv.b, n, vec);
    m_values(cm.w[0], cm.w[1], ts.ms[lo][block], m);
    v_values(cv.w[0], cv.w[1], ts.vs[lo][block], v);
  }
  uint32_t am = 0, av = 0;  // the block's largest magnitudes
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const float g = Elem<GT>::get(g8[i]);
    m[i] = __fadd_rn(__fmul_rn(m[i], st.b1), __fmul_rn(g, st.one_b1));
    v[i] = __fadd_rn(__fmul_rn(v[i], st.b2), __fmul_rn(__fmul_rn(g, g), st.one_b2));
    const float d = sqrt_fast(v[i] * st.c2) + st.eps;  // 2^-22 of the update
    p8[i] = Elem<PT>::put(Elem<PT>::get(p8[i]) * st.decay - m[i] * st.lr_c1 * rcp_fast(d));
    if (Q8 && (i & 1)) {  // by their bits, which put Inf and NaN above every number (v >= 0)
      am = __vimax3_u32(am, __float_as_uint(m[i - 1]) & 0x7FFFFFFFu, __float_as_uint(m[i]) & 0x7FFFFFFFu);
      av = __vimax3_u32(av, __float_as_uint(v[i - 1]), __float_as_uint(v[i]));
    }
  }
  store8(pp, p8, n, vec);
  if (!Q8) {
    store8(static_cast<float *>(ts.m[lo]) + at, m, n, vec);
    store8(static_cast<float *>(ts.v[lo]) + at, v, n, vec);
  } else {
    const Encode e = encode_with(__uint_as_float(__reduce_max_sync(0xffffffffu, am)),
                                 __uint_as_float(__reduce_max_sync(0xffffffffu, av)));
    union {
      uint8_t b[8];
      uint32_t w[2];
    } cm, cv;
#pragma unroll
    for (int h = 0; h < 2; h++) {
      uint32_t x[4], y[4];
      codes(e, m + 4 * h, v + 4 * h, x, y);
      cm.w[h] = __byte_perm(__byte_perm(x[0], x[1], 0x0040), __byte_perm(x[2], x[3], 0x0040), 0x5410);
      cv.w[h] = __byte_perm(__byte_perm(y[0], y[1], 0x0040), __byte_perm(y[2], y[3], 0x0040), 0x5410);
    }
    store8(static_cast<uint8_t *>(ts.m[lo]) + at, cm.b, n, vec);
    store8(static_cast<uint8_t *>(ts.v[lo]) + at, cv.b, n, vec);
    if (lane == 0) {
      ts.ms[lo][block] = e.am;
      ts.vs[lo][block] = e.av;
    }
  }
}

// Four consecutive elements a lane and run, so that a store instruction covers
// whole lines; four runs in flight.  150 M elements 224 us (6.7 TB/s).
constexpr int kMomentRuns = 4;
__global__ void __launch_bounds__(kThreads)
    k_moments(long long numel, const int8_t *cm, const float *am, const uint8_t *cv,
              const float *av, float *m, float *v, bool vec) {
  const long long base = (long long)blockIdx.x * kThreads * 4 * kMomentRuns + threadIdx.x * 4;
  uint32_t a[kMomentRuns], b[kMomentRuns];
  float sa[kMomentRuns], sb[kMomentRuns];
#pragma unroll
  for (int r = 0; r < kMomentRuns; r++) {
    const long long at = base + (long long)r * kThreads * 4;
    a[r] = b[r] = 0;
    sa[r] = sb[r] = 0.f;
    if (at < numel) {
      sa[r] = am[at / kBlock];
      sb[r] = av[at / kBlock];
      if (vec && at + 4 <= numel) {
        a[r] = *reinterpret_cast<const uint32_t *>(cm + at);
        b[r] = *reinterpret_cast<const uint32_t *>(cv + at);
      } else {
        for (int i = 0; i < 4 && at + i < numel; i++) {
          a[r] |= (uint32_t)(uint8_t)cm[at + i] << (8 * i);
          b[r] |= (uint32_t)cv[at + i] << (8 * i);
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kMomentRuns; r++) {
    const long long at = base + (long long)r * kThreads * 4;
    float x[8], y[8];  // the last four are not used
    m_values(a[r], 0, sa[r], x);
    v_values(b[r], 0, sb[r], y);
    if (vec && at + 4 <= numel) {
      *reinterpret_cast<float4 *>(m + at) = make_float4(x[0], x[1], x[2], x[3]);
      *reinterpret_cast<float4 *>(v + at) = make_float4(y[0], y[1], y[2], y[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; i++)
        if (at + i < numel) {
          m[at + i] = x[i];
          v[at + i] = y[i];
        }
    }
  }
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
  const bool vec = aligned(exp_avg, 4) && aligned(exp_avg_sq, 4) && aligned(m, 16) && aligned(v, 16);
  constexpr long long per = kThreads * 4 * kMomentRuns;
  const unsigned grid = (unsigned)((numel + per - 1) / per);
  k_moments<<<grid, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      numel, exp_avg, exp_avg_scale, exp_avg_sq, exp_avg_sq_scale, m, v, vec);
  return cudaGetLastError() == cudaSuccess ? OS2_OK : OS2_ERR_CUDA;
}
