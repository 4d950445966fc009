// Root-mean-square norm of rows, with the residual's addition in front of it:
//   h = x + r, rounded to the rows' type (the residual stream),
//   rho = (mean h^2 + eps)^(-1/2),   y = h rho w,
// y in the rows' type, or in 8-bit integers with a scale a row:
//   t = h w,  s = max |t| / 127,  q = rint(t / s),  scale = s rho.
// rho is common to a row and cancels in q, so the integers do not depend on the order of
// the sum of squares; t, s and t / s are each rounded once in FP32, sums are FP32.
//
// Every entry is read once and stays in registers between the sum and the result.  With a residual
// memory bounds it: 8192 x 8192 BF16 85 us (6.3 TB/s of what it reads and writes; DRAM 71 % busy, as a
// copy has it).  Without one (47 us, 5.7 TB/s, DRAM 57 % busy) it is the loads that are in flight and the
// waits for a row's sum, in 8 bits (74 us, with a residual 93, DRAM 56 %) the instructions of an entry.  One
// row is bound by latency: 1.8 us at 4096, 2.1 with a residual.
#include "norm.cuh"

using namespace os2norm;

namespace {

struct Args {
  int n, d;
  const void *X, *R;
  void *H;
  const void *w;
  bool w32;
  Lie lie;
  long ldx, ldr, ldh, ldy;
  float eps;
  void *Y;        // the rows' type, or int8
  float *scale;
  int *status;
};

// The integers (in FP32) of a group.
template <int DT, Lie LIE, int E>
__device__ __forceinline__ void store_q(int8_t *row, const Place<DT, LIE> &at, int j, const float (&c)[E]) {
  uint32_t b[E];  // the integer is the low byte
#pragma unroll
  for (int q = 0; q < E; q++) b[q] = __float_as_uint(c[q] + kRound);
  if (LIE != kEntries && at.all(j)) {
    uint32_t w[E / 4];
#pragma unroll
    for (int q = 0; q < E / 4; q++)
      w[q] = __byte_perm(__byte_perm(b[4 * q], b[4 * q + 1], 0x0040), __byte_perm(b[4 * q + 2], b[4 * q + 3], 0x0040),
                         0x5410);
    if constexpr (E == 8) *reinterpret_cast<uint2 *>(row + at.at(j, 0)) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t *>(row + at.at(j, 0)) = w[0];
  } else if (LIE != kGroups) {
#pragma unroll
    for (int q = 0; q < E; q++)
      if (at.in(at.at(j, q))) row[at.at(j, q)] = (int8_t)b[q];
  }
}

// A row's result from its sum of squares: t is h, or h w with its largest magnitude (Q8).
template <int DT, Lie LIE, bool Q8, int NV, int E>
__device__ __forceinline__ void finish_row(const Args &a, const Place<DT, LIE> &at, long row, float sum, float top, float (&t)[NV][E]) {
  const float rho = rsqrtf(sum / (float)a.d + a.eps);
  if constexpr (Q8) {
    const bool finite = __float_as_uint(top) < 0x7F800000u;
    const float s = __fdiv_rn(top, 127.f);
    const float by_s = s > 1e-30f && finite ? __frcp_rn(s) : 0.f;
    if (at.me == 0) a.scale[row] = finite ? s * rho : __uint_as_float(0x7FC00000u);
#pragma unroll
    for (int j = 0; j < NV; j++) {
      float c[E];
#pragma unroll
      for (int q = 0; q < E; q++) c[q] = 0.f;
      if (finite && s > 0.f) quant8<E>(t[j], s, by_s, c);
      store_q(static_cast<int8_t *>(a.Y) + (size_t)row * a.ldy, at, j, c);
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; j++) {
      float w[E];
      at.weights(a.w, a.w32, j, w);
#pragma unroll
      for (int q = 0; q < E; q++) t[j][q] = t[j][q] * rho * w[q];
      Group<DT> y;
      y.set(t[j]);
      at.store(a.Y, (size_t)row * a.ldy, j, y);
    }
  }
}

constexpr int kSmThreads = 1024;  // that an SM holds: at most 64 registers each

template <int DT, Lie LIE, bool Q8, int TEAM, int NV, int MOST>
__global__ void __launch_bounds__(MOST, kSmThreads / MOST) k_norm(const Args a) {
  constexpr bool AHEAD = NV == 2;  // (with four groups the next row's would not fit the registers)
  constexpr int E = kElems<DT>, LANES = TEAM ? TEAM : 1, ROWS = TEAM ? kTeamThreads / LANES : 1;
  __shared__ float s_sum[2][2][32];
  const int tid = (int)threadIdx.x;
  extern __shared__ __align__(16) float s_w[];  // (kShifted: the weights, behind them the rows)
  const int team = TEAM ? TEAM : (int)blockDim.x, step = (int)gridDim.x * ROWS;
  long row = (long)blockIdx.x * ROWS + (TEAM ? tid / LANES : 0);
  const int shift = LIE == kShifted ? shift_of<DT>(a.X, a.ldx, row) : 0, pitch = team * NV * E;
  const Place<DT, LIE> at{TEAM ? tid % LANES : tid, team, a.d, shift, s_w + (TEAM ? shift * pitch : 0), nullptr};
  start_call();
  Group<DT> x[NV], r[NV];
  auto load = [&](long row) {
#pragma unroll
    for (int j = 0; j < NV; j++) {
      if (row < a.n) at.load(a.X, (size_t)row * a.ldx, j, x[j]);
      else x[j].zero();
      if (a.R && row < a.n) at.load(a.R, (size_t)row * a.ldr, j, r[j]);
    }
  };
  if (AHEAD) load(row);
  if (LIE == kShifted) lay_weights<DT, TEAM, false>(s_w, pitch, a.w, a.w32, a.d, shift);
  int turn = 0;
  // (a CTA's teams go round together: the lanes of a warp meet in every sum)
  for (long r0 = (long)blockIdx.x * ROWS; r0 < a.n; r0 += step, row += step) {
    Group<DT> h[NV];
    float sum = 0.f, top = 0.f;
    if (!AHEAD) load(row);
#pragma unroll
    for (int j = 0; j < NV; j++) {
      h[j] = x[j];
      if (a.R && row < a.n) {
        float u[E], v[E];
        x[j].get(u), r[j].get(v);
#pragma unroll
        for (int q = 0; q < E; q++) u[q] += v[q];
        h[j].set(u);
        if (a.H) at.store(a.H, (size_t)row * a.ldh, j, h[j]);
      }
    }
    if (AHEAD) load(row + step);
    uint4 *const groups = reinterpret_cast<uint4 *>(s_w + (TEAM ? E : 1) * pitch) + (TEAM ? tid / LANES * TEAM * NV : 0);
    if constexpr (LIE == kShifted) {
      // (over_team ends the reads of the row before)
#pragma unroll
      for (int j = 0; j < NV; j++) groups[j * team + at.me] = make_uint4(h[j].w[0], h[j].w[1], h[j].w[2], h[j].w[3]);
      if (TEAM) __syncwarp();
      else __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < NV; j++) {
      float u[E], w[E];
      if constexpr (LIE == kShifted) {
        const int next = j * team + at.me + 1;
        straight<DT>(h[j], next < team * NV ? groups[next] : make_uint4(0, 0, 0, 0), shift).get(u);
      } else {
        h[j].get(u);
      }
#pragma unroll
      for (int q = 0; q < E; q++) sum = fmaf(u[q], u[q], sum);
      if (Q8) {
        if (LIE == kShifted) h[j].get(u);
        at.weights(a.w, a.w32, j, w);
#pragma unroll
        for (int q = 0; q < E; q += 2) top = max3_abs(top, u[q] * w[q], u[q + 1] * w[q + 1]);
      }
    }
    over_team<TEAM>(sum, top, std::conditional_t<Q8, Top, None>(), s_sum, turn);
    if (row >= a.n) continue;
    float t[NV][E];
#pragma unroll
    for (int j = 0; j < NV; j++) {
      h[j].get(t[j]);
      if constexpr (Q8) {
        float w[E];
        at.weights(a.w, a.w32, j, w);
#pragma unroll
        for (int q = 0; q < E; q++) t[j][q] *= w[q];
      }
    }
    finish_row<DT, LIE, Q8, NV>(a, at, row, sum, top, t);
  }
}

// The same with the rows from a ring of bulk copies in shared memory (kGroups, a CTA a row
// at a time): `stages` rows of X, each followed by its row of R, are on their way, and a stage is
// filled again once all threads have taken it into registers.  us, walk and ring:
//                      8192 x 4096 BF16   8192 x 8192 BF16   4096 x 16384 BF16   4096 x 8192 FP32
//   residual             49.0   45.5         98.1   85.8         108.9   85.0         98.4   87.4
//   int8                 42.8   39.0         84.6   74.2          86.5   80.1         39.8   54.8
//   both                 64.2   48.4        126.6   93.0         137.8  100.0         81.0   79.7
//   neither              24.6   29.7         47.4   54.8          48.9   60.7         44.8   48.8
// One array with little to do needs no more than the walk has in flight; two, or the longer
// stretch of integers, do.  (The gradient, with a register a column for dw, gained nothing:
// 64.5 and 63.2, 61.2 and 69.3 at 16384 x 2048.)
constexpr int kStages = 8, kRingBytes = 216 * 1024;
struct Ring {
  uint64_t full[kStages];
  int abort;
};
struct RingGrid {
  int ctas, threads, stages;  // no stages: the walk
};
RingGrid ring_grid(int n, int d, int elems, bool q8, bool two) {
  RingGrid g;
  g.threads = (int)os2_round_up((size_t)((d + 2 * elems - 1) / (2 * elems)), 32);
  const int per_sm = std::max(1, kSmThreads / g.threads);
  g.ctas = os2_sm_count() * per_sm;
  g.stages = (int)std::min<size_t>(kStages, (size_t)(kRingBytes / per_sm) / ((size_t)d * (16 / elems) * (two ? 2 : 1)));
  // (a handful of rows a CTA at least, or the ring's start and end weigh more)
  if (!(two || (q8 && elems == 8)) || g.threads < 128 || g.threads > 1024 || g.stages < 2 || n < 4 * g.ctas) g.stages = 0;
  return g;
}

template <int DT, bool Q8, int MOST>
__global__ void __launch_bounds__(MOST, kSmThreads / MOST) k_norm_ring(const Args a, int stages) {
  constexpr int E = kElems<DT>, NV = 2;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_sum[2][2][32];
  __shared__ Ring ring;
  const int tid = (int)threadIdx.x, step = (int)gridDim.x;
  const Place<DT, kGroups> at{tid, (int)blockDim.x, a.d, 0, nullptr, nullptr};
  const uint32_t bytes = (uint32_t)a.d * (16 / E), stage = bytes * (a.R ? 2 : 1);
  if (tid == 0) {
    for (int s = 0; s < stages; s++) mbar_init(&ring.full[s], 1);
    ring.abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  start_call();
  auto fetch = [&](long row, int st) {
    mbar_arrive_expect_tx(&ring.full[st], stage);
    bulk_load(smem + st * stage, static_cast<const char *>(a.X) + (size_t)row * a.ldx * (16 / E), bytes, &ring.full[st]);
    if (a.R)
      bulk_load(smem + st * stage + bytes, static_cast<const char *>(a.R) + (size_t)row * a.ldr * (16 / E), bytes, &ring.full[st]);
  };
  if (tid == 0)
    for (int s = 0; s < stages; s++)
      if (blockIdx.x + (long)s * step < a.n) fetch(blockIdx.x + (long)s * step, s);
  int turn = 0, st = 0;
  uint32_t parity = 0;
  for (long row = blockIdx.x; row < a.n; row += step) {
    // (no thread leaves before the barrier in over_team: all see who gave up)
    if (!mbar_wait_bounded(&ring.full[st], parity, &ring.abort, kWaitLimit)) {
      ring.abort = 1;
      set_status(a.status, OS2_ERR_TIMEOUT);
    }
    float t[NV][E];
    float sum = 0.f, top = 0.f;
#pragma unroll
    for (int j = 0; j < NV; j++) {
      Group<DT> x, r;
      x.zero();
      const bool in = at.at(j, 0) < a.d;
      if (in) x = *reinterpret_cast<const Group<DT> *>(smem + st * stage + at.at(j, 0) * (16 / E));
      x.get(t[j]);
      if (a.R) {
        float v[E];
        r.zero();
        if (in) r = *reinterpret_cast<const Group<DT> *>(smem + st * stage + bytes + at.at(j, 0) * (16 / E));
        r.get(v);
#pragma unroll
        for (int q = 0; q < E; q++) t[j][q] += v[q];
        x.set(t[j]);
        if (a.H) at.store(a.H, (size_t)row * a.ldh, j, x);
        x.get(t[j]);
      }
      float w[E];
      if (Q8) at.weights(a.w, a.w32, j, w);
#pragma unroll
      for (int q = 0; q < E; q += 2) {
        sum = fmaf(t[j][q], t[j][q], sum);
        sum = fmaf(t[j][q + 1], t[j][q + 1], sum);
        if (Q8) {
          t[j][q] *= w[q];
          t[j][q + 1] *= w[q + 1];
          top = max3_abs(top, t[j][q], t[j][q + 1]);
        }
      }
    }
    over_team<0>(sum, top, std::conditional_t<Q8, Top, None>(), s_sum, turn);
    if (*(volatile int *)&ring.abort) break;
    if (tid == 0 && row + (long)stages * step < a.n) fetch(row + (long)stages * step, st);
    if (++st == stages) st = 0, parity ^= 1;
    finish_row<DT, kGroups, Q8, NV>(a, at, row, sum, top, t);
  }
  // (on the way out early: what is still being copied lands first)
  if (tid == 0 && ring.abort)
    for (int s = 0; s < stages; s++) {
      volatile int no_abort = 0;
      mbar_wait_bounded(&ring.full[s], parity ^ (s < st), &no_abort, kWaitLimit);
    }
}

template <int DT, bool Q8, int MOST>
cudaError_t launch_ring(const Args &a, const RingGrid &r, cudaStream_t s) {
  const size_t bytes = (size_t)r.stages * a.d * (16 / kElems<DT>) * (a.R ? 2 : 1);
  static PerDevice ready;
  const cudaError_t e = os2_set_smem(ready, k_norm_ring<DT, Q8, MOST>, kRingBytes);
  return e != cudaSuccess ? e : launch_after(k_norm_ring<DT, Q8, MOST>, r.ctas, r.threads, bytes, s, a, r.stages);
}

// kShifted lays the weights out first, which pays where a CTA has some rows.  us, entry by entry and
// shifted: 8192 x 4095 BF16 104 and 45, with a residual 171 and 68, int8 161 and 64, both 237 and
// 85 (4096: 25, 45, 39, 48); 205 x 1777 FP16 3.8 and 5.0.
template <int DT, Lie LIE, bool Q8>
cudaError_t launch(const Args &a, cudaStream_t s) {
  constexpr int E = kElems<DT>;
  if constexpr (LIE == kGroups) {
    const RingGrid r = ring_grid(a.n, a.d, E, Q8, a.R != nullptr);
    if (r.stages) return r.threads <= 512 ? launch_ring<DT, Q8, 512>(a, r, s) : launch_ring<DT, Q8, 1024>(a, r, s);
  }
  return for_shape<E>(span(a.d, E, LIE), [&](auto team, auto nv, auto most) {
    constexpr int T = decltype(team)::value, NV = decltype(nv)::value, MOST = decltype(most)::value;
    const Grid g = grid_for(a.n, span(a.d, E, LIE), T, NV, E, kSmThreads);
    size_t bytes = 0;
    if constexpr (LIE == kShifted) {
      if (a.n <= 2L * g.ctas * (T ? kTeamThreads / T : 1)) return launch<DT, kEntries, Q8>(a, s);
      bytes = shifted_bytes(T, NV, E, g.threads, 1);
      static PerDevice ready;
      const cudaError_t e = os2_set_smem(ready, k_norm<DT, LIE, Q8, T, NV, MOST>, shifted_bytes(T, NV, E, MOST, 1));
      if (e != cudaSuccess) return e;
    }
    return launch_after(k_norm<DT, LIE, Q8, T, NV, MOST>, g.ctas, g.threads, bytes, s, a);
  });
}

// Of the arguments that both entry points have.
os2_status check(int n, int d, int dtype, const void *X, int ldx, const void *R, int ldr, const void *H, int ldh,
                 const void *w, int wt, double eps, int ldy) {
  if (n < 0 || d < 1 || ldx < d || ldy < d || (R && ldr < d) || (H && ldh < d) || !is_dtype(dtype)) return OS2_ERR_INVALID_ARG;
  if ((wt != OS2_F32 && wt != dtype) || !(eps >= 0) || !(eps < 1e30)) return OS2_ERR_INVALID_ARG;
  if (!w || !aligned(w, elem_size(wt)) || (H && !R)) return OS2_ERR_INVALID_ARG;
  const size_t e = elem_size(dtype);
  if (n > 0 && (!X || !aligned(X, e) || !aligned(R, e) || !aligned(H, e))) return OS2_ERR_INVALID_ARG;
  return d > kMaxD ? OS2_ERR_UNSUPPORTED : OS2_OK;
}

Args args(int n, int d, int dtype, const void *X, int ldx, const void *R, int ldr, void *H, int ldh, const void *w, int wt,
          double eps) {
  const size_t e = elem_size(dtype);
  Args a = {};
  a.n = n, a.d = d;
  a.X = X, a.ldx = ldx, a.R = R, a.ldr = ldr, a.H = H, a.ldh = ldh;
  a.w = w, a.w32 = wt == OS2_F32;
  a.eps = (float)eps;
  a.status = os2_status_ptr();
  const bool groups = on16(X, ldx, e) && (!R || on16(R, ldr, e)) && (!H || on16(H, ldh, e)) && aligned(w, 16) && d % (16 / e) == 0;
  const bool shifted = (!R || same16(R, ldr, X, ldx, e)) && (!H || same16(H, ldh, X, ldx, e)) && d + 7 <= kMaxD;
  a.lie = groups ? kGroups : shifted ? kShifted : kEntries;
  return a;
}

template <Lie LIE, bool Q8>
cudaError_t launch_t(const Args &a, int dtype, cudaStream_t s) {
  if (dtype == OS2_F32) return launch<OS2_F32, LIE, Q8>(a, s);
  if (dtype == OS2_BF16) return launch<OS2_BF16, LIE, Q8>(a, s);
  return launch<OS2_F16, LIE, Q8>(a, s);
}
template <bool Q8>
os2_status run(const Args &a, int dtype, void *stream) {
  if (!a.status) return OS2_ERR_CUDA;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a.lie == kGroups    ? launch_t<kGroups, Q8>(a, dtype, s)
                        : a.lie == kShifted ? launch_t<kShifted, Q8>(a, dtype, s)
                                            : launch_t<kEntries, Q8>(a, dtype, s);
  return e == cudaSuccess ? OS2_OK : OS2_ERR_CUDA;
}

}  // namespace

extern "C" os2_status os2_rmsnorm(int n, int d, int dtype, const void *X, int ldx, const void *R, int ldr, void *H,
                                  int ldh, const void *weight, int weight_dtype, double eps, void *Y, int ldy,
                                  void *stream) {
  const os2_status st = check(n, d, dtype, X, ldx, R, ldr, H, ldh, weight, weight_dtype, eps, ldy);
  if (st) return st;
  if (n == 0) return OS2_OK;
  if (!Y || !aligned(Y, elem_size(dtype))) return OS2_ERR_INVALID_ARG;
  Args a = args(n, d, dtype, X, ldx, R, ldr, H, ldh, weight, weight_dtype, eps);
  a.Y = Y, a.ldy = ldy;
  const size_t e = elem_size(dtype);
  if (a.lie == kGroups && !on16(Y, ldy, e)) a.lie = kEntries;
  if (a.lie == kShifted && !same16(Y, ldy, X, ldx, e)) a.lie = kEntries;
  return run<false>(a, dtype, stream);
}

extern "C" os2_status os2_rmsnorm_quantize(int n, int d, int dtype, const void *X, int ldx, const void *R, int ldr,
                                           void *H, int ldh, const void *weight, int weight_dtype, double eps, int8_t *q,
                                           int ldq, float *scale, void *stream) {
  const os2_status st = check(n, d, dtype, X, ldx, R, ldr, H, ldh, weight, weight_dtype, eps, ldq);
  if (st) return st;
  if (n == 0) return OS2_OK;
  if (!q || !scale || !aligned(scale, 4)) return OS2_ERR_INVALID_ARG;
  Args a = args(n, d, dtype, X, ldx, R, ldr, H, ldh, weight, weight_dtype, eps);
  a.Y = q, a.ldy = ldq, a.scale = scale;
  // (the integers of a group are stored at once: as many bytes as it has entries)
  const uintptr_t e = elem_size(dtype), E = 16 / e;
  if (a.lie == kGroups && !(aligned(q, E) && ldq % E == 0)) a.lie = kEntries;
  if (a.lie == kShifted && ((reinterpret_cast<uintptr_t>(q) - reinterpret_cast<uintptr_t>(X) / e) % E || (long)(ldq - ldx) % (long)E))
    a.lie = kEntries;
  return run<true>(a, dtype, stream);
}
