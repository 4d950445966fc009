// Matrix product in 8-bit integers with a scale for each row of A (token) and
// each row of B (output channel):
//   y_ij = (sum_h qa_ih qb_jh) sa_i sb_j + bias_j,  the sum an exact int32,
// and the quantisation it needs:
//   s_i = max_h |x_ih| / 127,  q_ih = clamp(rint(x_ih / s_i), -127, 127).
//
// Quantisation, layout and dispatch; the products are in k_i8few.cu (few tokens)
// and k_i8tc.cu.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "i8.cuh"

using namespace os2mm;

namespace {

template <int DT>
__device__ __forceinline__ float load_f(const void *p, size_t i) {
  if (DT == OS2_F32) return static_cast<const float *>(p)[i];
  if (DT == OS2_BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
  return __half2float(static_cast<const __half *>(p)[i]);
}

// 8 consecutive entries, of which n exist (vec: base and pitch allow 16-byte loads)
template <int DT>
__device__ __forceinline__ void load8(const void *p, size_t i, int n, bool vec, float (&x)[8]) {
  if (vec && n >= 8) {
    if (DT == OS2_F32) {
      const float4 a = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
      const float4 b = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i + 4);
      x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
      x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    } else {
      const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int q = 0; q < 4; q++) {
        if (DT == OS2_BF16) {
          x[2 * q] = __uint_as_float(w[q] << 16);
          x[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
        } else {
          const float2 f = __half22float2(reinterpret_cast<const __half2 &>(w[q]));
          x[2 * q] = f.x;
          x[2 * q + 1] = f.y;
        }
      }
    }
  } else {
#pragma unroll
    for (int q = 0; q < 8; q++) x[q] = q < n ? load_f<DT>(p, i + q) : 0.f;
  }
}

// Eight times rint(x / s), clamped, as FP32: the quotient is the correctly rounded
// one, so that a plain division gives the same integers.  A division takes some 15
// instructions and would bound the kernel, so x times r = 1 / s decides first: it is
// off by less than 1.6e-5, the rounded quotient itself by less than 8e-6, and only where
// one of the eight lies nearer than 1e-4 to a tie are they divided.  r is 0 where 1 / s
// could leave the normal numbers: all are divided then.
constexpr float kRound = 12582912.0f;  // 1.5 2^23
__device__ __forceinline__ void quant8(const float (&x)[8], float s, float r, float (&c)[8]) {
  float off = 0.f;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const float y = x[i] * r;
    c[i] = (y + kRound) - kRound;
    off = fmaxf(off, fabsf(y - c[i]));
  }
  if (off > 0.4999f || r == 0.f)
#pragma unroll
    for (int i = 0; i < 8; i++)
      c[i] = fminf(fmaxf(rintf(__fdiv_rn(x[i], s)), -127.f), 127.f);
}

constexpr int kQThreads = 256;

// 8 consecutive integers (as FP32) of which n are stored (vec: aligned for one store)
__device__ __forceinline__ void store8(int8_t *dst, const float (&c)[8], int n, bool vec) {
  uint32_t b[8];  // the integer is the low byte
#pragma unroll
  for (int i = 0; i < 8; i++) b[i] = __float_as_uint(c[i] + kRound);
  if (vec && n >= 8) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; i++)
      w[i] = __byte_perm(__byte_perm(b[4 * i], b[4 * i + 1], 0x0040),
                         __byte_perm(b[4 * i + 2], b[4 * i + 3], 0x0040), 0x5410);
    *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++)
      if (i < n) dst[i] = (int8_t)b[i];
  }
}
__device__ __forceinline__ void store8(__half *dst, const float (&c)[8], int n, bool vec) {
  if (vec && n >= 8) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const __half2 h = __floats2half2_rn(c[2 * i], c[2 * i + 1]);
      w[i] = reinterpret_cast<const uint32_t &>(h);
    }
    *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++)
      if (i < n) dst[i] = __float2half_rn(c[i]);
  }
}

// One CTA a row: the row's largest magnitude, then its integers; 4096 entries stay in
// registers between, the second read of the others comes from cache.  The maximum is taken of the bits of |x|, which order
// as the values do and put Inf and NaN above every number.  Q: int8_t, or __half
// for the products' tokens.  Also zeroes the nzero counters of the kernel that
// follows, which may start before this one ends and waits for its end.  8192 x 4096 BF16
// to int8: 33 us (3.0 TB/s), 5 % of the product that follows.
template <int DT, typename Q>
__global__ void __launch_bounds__(kQThreads)
    k_quant(int k, const void *X, long ldx, Q *q, long ldq, float *scale, bool vecx,
            bool vecq, unsigned *zero, int nzero) {
  __shared__ uint32_t s_top[kQThreads / 32];
  const int row = blockIdx.x, tid = threadIdx.x;
  start_call();
  if (row == 0)
    for (int i = tid; i < nzero; i += kQThreads) zero[i] = 0;
  const char *x = static_cast<const char *>(X) + (size_t)row * ldx * (DT == OS2_F32 ? 4 : 2);
  constexpr int STEP = kQThreads * 8, KEPT = 2;
  uint32_t top = 0;
  auto larger = [&](const float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; i++) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  };
  float kept[KEPT][8];
#pragma unroll
  for (int i = 0; i < KEPT; i++) {
    const int h = i * STEP + tid * 8;
    if (h < k) {
      load8<DT>(x, h, k - h, vecx, kept[i]);
      larger(kept[i]);
    }
  }
  for (int h = KEPT * STEP + tid * 8; h < k; h += STEP) {
    float v[8];
    load8<DT>(x, h, k - h, vecx, v);
    larger(v);
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if ((tid & 31) == 0) s_top[tid >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kQThreads / 32; w++) top = max(top, s_top[w]);
  const bool finite = top < 0x7F800000u;
  const float s = __fdiv_rn(__uint_as_float(top), 127.f);
  if (tid == 0) scale[row] = finite ? s : __uint_as_float(0x7FC00000u);
  const float r = s > 1e-30f && finite ? __frcp_rn(s) : 0.f;
  Q *dst = q + (size_t)row * ldq;
  auto put = [&](int h, const float (&v)[8]) {
    float c[8];
    if (finite && s > 0.f) {
      quant8(v, s, r, c);
    } else {
#pragma unroll
      for (int i = 0; i < 8; i++) c[i] = 0.f;
    }
    store8(dst + h, c, k - h, vecq);
  };
#pragma unroll
  for (int i = 0; i < KEPT; i++) {
    const int h = i * STEP + tid * 8;
    if (h < k) put(h, kept[i]);
  }
  for (int h = KEPT * STEP + tid * 8; h < k; h += STEP) {
    float v[8];
    load8<DT>(x, h, k - h, vecx, v);
    put(h, v);
  }
}

// 8-bit tokens as FP16, one CTA a row.
__global__ void __launch_bounds__(kQThreads)
    k_widen_tokens(int k, const int8_t *A, long lda, __half *dst, long pitch, bool vec,
                   unsigned *zero, int nzero) {
  start_call();
  const int row = blockIdx.x, tid = threadIdx.x;
  if (row == 0)
    for (int i = tid; i < nzero; i += kQThreads) zero[i] = 0;
  const int8_t *a = A + (size_t)row * lda;
  for (int h = tid * 8; h < k; h += kQThreads * 8) {
    __half *to = dst + (size_t)row * pitch + h;
    if (vec && h + 8 <= k) {
      const uint2 w = *reinterpret_cast<const uint2 *>(a + h);
      uint4 o;
      os2i8::widen(w.x, o.x, o.y);
      os2i8::widen(w.y, o.z, o.w);
      *reinterpret_cast<uint4 *>(to) = o;
    } else {
      float c[8];
#pragma unroll
      for (int i = 0; i < 8; i++) c[i] = h + i < k ? (float)a[h + i] : 0.f;
      store8(to, c, k - h, true);
    }
  }
}

// Rows of B off the 16-byte boundaries that TMA needs, copied onto them (only
// for such B): 16 bytes a thread, read as words that straddle them.  16384 x 4095: 24 us
// (5.5 TB/s read and written).
__global__ void __launch_bounds__(256)
    k_align_rows(int n, int k, const int8_t *B, long ldb, int8_t *dst, long pitch) {
  // (beside the kernel that quantises the tokens: they share nothing, and B, an input of
  // the call, is complete since that one passed start_call)
  next_may_start();
  const long per = pitch / 16, total = per * n;
  for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < total; i += (long)gridDim.x * 256) {
    const long r = i / per;
    const int h = (int)(i - r * per) * 16;
    const int8_t *src = B + r * ldb + h;
    uint32_t w[4];
    if (h >= 4 && h + 20 <= k) {
      const int o = (int)(reinterpret_cast<uintptr_t>(src) & 3);
      const uint32_t *p = reinterpret_cast<const uint32_t *>(src - o);
      uint32_t x[5];
#pragma unroll
      for (int q = 0; q < 5; q++) x[q] = __ldg(p + q);
#pragma unroll
      for (int q = 0; q < 4; q++) w[q] = __funnelshift_r(x[q], x[q + 1], 8 * o);
    } else {
#pragma unroll
      for (int q = 0; q < 4; q++) w[q] = 0;
#pragma unroll
      for (int q = 0; q < 16; q++)
        if (h + q < k) w[q >> 2] |= (uint32_t)(uint8_t)src[q] << (8 * (q & 3));
    }
    *reinterpret_cast<uint4 *>(dst + r * pitch + h) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  wait_for_previous();  // the next kernel's wait for this one is one for that one too
}

// Without terms, the bias.
__global__ void k_bias(int m, int n, const float *bias, void *y, long ldy, int dtype) {
  const long total = (long)m * n;
  for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < total; i += (long)gridDim.x * 256)
    os2i8::store_y(y, dtype, (size_t)(i / n) * ldy + i % n, bias ? bias[i % n] : 0.f);
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t elem_size(int dt) { return dt == OS2_F32 ? 4 : 2; }
bool is_dtype(int dt) { return dt == OS2_F32 || dt == OS2_F16 || dt == OS2_BF16; }

template <typename Q>
cudaError_t quantize(int m, int k, int dtype, const void *X, long ldx, Q *q, long ldq,
                     float *scale, cudaStream_t s, unsigned *zero = nullptr, int nzero = 0) {
  const bool vecx = aligned(X, 16) && (ldx * elem_size(dtype)) % 16 == 0;
  const bool vecq = aligned(q, 8 * sizeof(Q)) && ldq % 8 == 0;
  auto launch = [&](auto kernel) {
    return launch_after(kernel, m, kQThreads, 0, s, k, X, ldx, q, ldq, scale, vecx, vecq, zero, nzero);
  };
  if (dtype == OS2_F32) return launch(k_quant<OS2_F32, Q>);
  if (dtype == OS2_BF16) return launch(k_quant<OS2_BF16, Q>);
  return launch(k_quant<OS2_F16, Q>);
}

// |sum| <= k 2^14 stays below 2^31
constexpr int kMaxK = (1 << 17) - 1;
constexpr int kMaxDim = 1 << 24;

// Up to 64 tokens go to mma.sync, more to tcgen05: 64 tokens take 16.4 us with the one,
// 65 tokens 21.4 with the other for 4096 x 4096 weights, 32.5 and 32.4 for 14336 x 4096;
// 16 tokens 8.8 and 16.6 us with the first, 22 and 29 with the second.
bool few(int m) { return m <= kI8Few; }

struct Layout {
  long pitch;                               // of the tokens
  long wpitch;                              // of the copied weights, 0: as they lie
  int counters;
  size_t tokens, scale, done, slots, weights, total;
};
Layout layout(int m, int n, int k, const void *B, long ldb) {
  Layout L = {};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += os2_round_up(bytes, 256);
    return o;
  };
  L.pitch = (long)os2_round_up((size_t)k, 8);
  L.tokens = take((size_t)m * L.pitch * 2);
  L.scale = take((size_t)m * 4);
  if (k > 0 && n > 0 && m > 0) {
    if (!few(m)) {
      const I8Sizes z = i8tc_sizes(m, n, k);
      L.counters = z.counters;
      L.done = take((size_t)z.counters * 4);
      L.slots = take(z.slot_ints * 4);
    }
    if (!aligned(B, 16) || ldb % 16) {
      L.wpitch = (long)os2_round_up((size_t)k, 16);
      L.weights = take((size_t)n * L.wpitch);
    }
  }
  L.total = at;
  return L;
}

// After the tokens are in the workspace (k >= 1).
cudaError_t product(int m, int n, int k, const Layout &L, char *ws, const float *sa,
                    const int8_t *B, long ldb, const float *sb, const float *bias, void *C,
                    long ldc, int ot, int *status, cudaStream_t s) {
  const bool overlap = !L.wpitch;
  if (L.wpitch) {
    int8_t *w = reinterpret_cast<int8_t *>(ws + L.weights);
    const long pieces = L.wpitch / 16 * n;
    const cudaError_t e =
        launch_after(k_align_rows, (int)std::min<long>((pieces + 255) / 256, 16L * os2_sm_count()),
                     256, 0, s, n, k, B, ldb, w, L.wpitch);
    if (e != cudaSuccess) return e;
    B = w;
    ldb = L.wpitch;
  }
  I8Args a;
  a.m = m;
  a.n = n;
  a.k = k;
  a.tokens = ws + L.tokens;
  a.pitch = L.pitch;
  a.W = B;
  a.ldw = ldb;
  a.sa = sa;
  a.sb = sb;
  a.bias = bias;
  a.y = C;
  a.ldy = ldc;
  a.out_dtype = ot;
  a.slots = reinterpret_cast<int *>(ws + L.slots);
  a.done = reinterpret_cast<unsigned *>(ws + L.done);
  a.status = status;
  a.overlap = overlap;
  return few(m) ? launch_i8few(a, s) : launch_i8tc(a, s);
}

os2_status check(int m, int n, int k, const void *A, int lda, const void *B, int ldb,
                 const float *sb, const float *bias, const void *C, int ldc, int ot) {
  if (m < 0 || n < 0 || k < 0 || lda < k || ldb < k || ldc < n || !is_dtype(ot))
    return OS2_ERR_INVALID_ARG;
  if (m > 0 && n > 0 && (!C || !aligned(C, elem_size(ot)) || !sb || !aligned(sb, 4) ||
                         (bias && !aligned(bias, 4)) || (k > 0 && (!A || !B))))
    return OS2_ERR_INVALID_ARG;
  if (k > kMaxK || m > kMaxDim || n > kMaxDim || (long long)m * n > (1LL << 40))
    return OS2_ERR_UNSUPPORTED;
  return OS2_OK;
}

}  // namespace

extern "C" os2_status os2_quantize_rows(int m, int k, int dtype, const void *X, int ldx, int8_t *q,
                                        int ldq, float *scale, void *stream) {
  if (m < 0 || k < 0 || ldx < k || ldq < k || !is_dtype(dtype)) return OS2_ERR_INVALID_ARG;
  if (m == 0) return OS2_OK;
  if (k > (1 << 30)) return OS2_ERR_UNSUPPORTED;
  if (!scale || !aligned(scale, 4) || (k > 0 && (!X || !q || !aligned(X, elem_size(dtype)))))
    return OS2_ERR_INVALID_ARG;
  return quantize(m, k, dtype, X, ldx, q, ldq, scale, static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? OS2_OK
             : OS2_ERR_CUDA;
}

extern "C" size_t os2_i8gemm_workspace_size(int m, int n, int k, const void *B, int ldb) {
  if (m < 0 || n < 0 || k < 0 || k > kMaxK || m > kMaxDim || n > kMaxDim || ldb < k ||
      (long long)m * n > (1LL << 40))
    return 0;
  return layout(m, n, k, B, ldb).total;
}

extern "C" os2_status os2_i8gemm(int m, int n, int k, const int8_t *A, int lda,
                                 const float *a_scale, const int8_t *B, int ldb,
                                 const float *b_scale, const float *bias, void *C, int ldc,
                                 int out_dtype, void *workspace, size_t workspace_bytes,
                                 void *stream) {
  const os2_status st = check(m, n, k, A, lda, B, ldb, b_scale, bias, C, ldc, out_dtype);
  if (st) return st;
  if (m == 0 || n == 0) return OS2_OK;
  if (!a_scale || !aligned(a_scale, 4)) return OS2_ERR_INVALID_ARG;
  const Layout L = layout(m, n, k, B, ldb);
  if (!workspace || workspace_bytes < L.total || !aligned(workspace, 256))
    return OS2_ERR_WORKSPACE;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  int *status = os2_status_ptr();
  if (!status) return OS2_ERR_CUDA;
  if (k == 0) {
    k_bias<<<std::min<long>(((long)m * n + 255) / 256, 8L * os2_sm_count()), 256, 0, s>>>(
        m, n, bias, C, ldc, out_dtype);
    return cudaGetLastError() == cudaSuccess ? OS2_OK : OS2_ERR_CUDA;
  }
  char *ws = static_cast<char *>(workspace);
  cudaError_t e = launch_after(k_widen_tokens, m, kQThreads, 0, s, k, A, lda,
                               reinterpret_cast<__half *>(ws + L.tokens), L.pitch,
                               aligned(A, 8) && lda % 8 == 0,
                               reinterpret_cast<unsigned *>(ws + L.done), L.counters);
  if (e != cudaSuccess) return OS2_ERR_CUDA;
  e = product(m, n, k, L, ws, a_scale, B, ldb, b_scale, bias, C, ldc, out_dtype,
                                status, s);
  return e == cudaSuccess ? OS2_OK : OS2_ERR_CUDA;
}

extern "C" os2_status os2_i8linear(int m, int n, int k, int dtype, const void *X, int ldx,
                                   const int8_t *B, int ldb, const float *b_scale,
                                   const float *bias, void *C, int ldc, int out_dtype,
                                   void *workspace, size_t workspace_bytes, void *stream) {
  if (!is_dtype(dtype) || (X && !aligned(X, elem_size(dtype)))) return OS2_ERR_INVALID_ARG;
  const os2_status st = check(m, n, k, X, ldx, B, ldb, b_scale, bias, C, ldc, out_dtype);
  if (st) return st;
  if (m == 0 || n == 0) return OS2_OK;
  const Layout L = layout(m, n, k, B, ldb);
  if (!workspace || workspace_bytes < L.total || !aligned(workspace, 256))
    return OS2_ERR_WORKSPACE;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  int *status = os2_status_ptr();
  if (!status) return OS2_ERR_CUDA;
  if (k == 0) {
    k_bias<<<std::min<long>(((long)m * n + 255) / 256, 8L * os2_sm_count()), 256, 0, s>>>(
        m, n, bias, C, ldc, out_dtype);
    return cudaGetLastError() == cudaSuccess ? OS2_OK : OS2_ERR_CUDA;
  }
  char *ws = static_cast<char *>(workspace);
  float *sa = reinterpret_cast<float *>(ws + L.scale);
  cudaError_t e = quantize(m, k, dtype, X, ldx, reinterpret_cast<__half *>(ws + L.tokens), L.pitch,
                           sa, s, reinterpret_cast<unsigned *>(ws + L.done), L.counters);
  if (e == cudaSuccess)
    e = product(m, n, k, L, ws, sa, B, ldb, b_scale, bias, C, ldc, out_dtype, status, s);
  return e == cudaSuccess ? OS2_OK : OS2_ERR_CUDA;
}
