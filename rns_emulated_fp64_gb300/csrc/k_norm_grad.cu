// The gradient of the norm (k_norm.cu): with xn = h rho and a = dy w,
//   dx = rho (a - xn mean(a xn)) + dh,    dw = sum over the rows of dy xn,
// where dh is what comes back along the residual stream; dx is the gradient of x and of r.
//
// h, dy and dh are read once and dx written once.  In 16 bits the waits of a row bound it (its loads, two
// sums over the CTA): 8192 x 8192 BF16 120 us, 4.5 TB/s of what it reads and writes, DRAM 42 % busy; in
// FP32 memory does (6.1 TB/s).  rho is computed again
// from the row that is read anyway.  CTAs walk the rows and keep their part of dw in
// registers; the parts are joined in the CTAs' order by a second kernel, so that dw is the
// same from run to run.
#include "norm.cuh"

using namespace os2norm;

namespace {

struct Args {
  int n, d;
  const void *H, *dY, *dH;
  const void *w;
  bool w32;
  long ldh, lddy, lddh, lddx;
  float eps;
  void *dX;       // or null
  float *part;    // [CTAs][d], or null
};

// Threads that an SM holds: 128 registers each, or 64.
constexpr int sm_threads(int most) { return most > 512 ? 1024 : 512; }
// As for_shape; the wider rows in 16-byte groups with one group a thread, which leaves room for
// twice the threads: what a row waits for (its loads, sums over lanes, the barrier) weighs
// more than their number.  us with one and two: 8192 x 4096 BF16 60.0 64.3, 8192 x 8192 119.8
// 122.2, 16384 x 2048 59.4 63.4; 8192 x 4095 (entry by entry) 208 186.
template <int E, Lie LIE, class F>
auto grad_shape(int d, F &&f) {
  using std::integral_constant;
  const int g = (span(d, E, LIE) + E - 1) / E;
  if (LIE != kEntries && g > 64 && g <= 1024) return f(integral_constant<int, 0>(), integral_constant<int, 1>(), integral_constant<int, 1024>());
  return for_shape<E>(span(d, E, LIE), f);
}

// (fma and mul in pairs: 122 us for 8192 x 8192 BF16, one by one 130)
template <int DT, Lie LIE, int TEAM, int NV, int MOST>
__global__ void __launch_bounds__(MOST, sm_threads(MOST) / MOST) k_norm_grad(const Args a) {
  constexpr bool AHEAD = NV == 1 || MOST <= 512;  // (else 64 registers do not hold the next row too)
  constexpr int E = kElems<DT>, LANES = TEAM ? TEAM : 1, ROWS = TEAM ? kTeamThreads / LANES : 1;
  __shared__ float s_sum[2][2][32];
  __shared__ float s_dw[TEAM ? ROWS * TEAM * NV * E : 1];
  const int tid = (int)threadIdx.x;
  extern __shared__ __align__(16) float s_w[];  // (kShifted: the weights, behind them the rows)
  const int team = TEAM ? TEAM : (int)blockDim.x, pitch = team * NV * E;
  const int mine = TEAM ? tid / LANES : 0, step = (int)gridDim.x * ROWS;
  long row = (long)blockIdx.x * ROWS + mine;
  const int shift = LIE == kShifted ? shift_of<DT>(a.H, a.ldh, row) : 0;
  const Place<DT, LIE> at{TEAM ? tid % LANES : tid, team, a.d, shift, s_w + (TEAM ? shift * pitch : 0), s_w + (TEAM ? 0 : pitch)};
  start_call();
  Two dw2[NV][E / 2];
#pragma unroll
  for (int j = 0; j < NV; j++)
#pragma unroll
    for (int q = 0; q < E / 2; q++) dw2[j][q] = Two(0.f, 0.f);
  const float by_d = 1.f / (float)a.d;
  const bool along = a.dX && a.dH;
  Group<DT> nh[NV], ng[NV];
  auto load = [&](long row) {
#pragma unroll
    for (int j = 0; j < NV; j++) {
      if (row < a.n) {
        at.load(a.H, (size_t)row * a.ldh, j, nh[j]);
        at.load(a.dY, (size_t)row * a.lddy, j, ng[j]);
      } else {
        nh[j].zero();
        ng[j].zero();
      }
    }
  };
  if (AHEAD) load(row);
  if (LIE == kShifted) lay_weights<DT, TEAM, true>(s_w, pitch, a.w, a.w32, a.d, shift);
  int turn = 0;
  for (long r0 = (long)blockIdx.x * ROWS; r0 < a.n; r0 += step, row += step) {
    Group<DT> h[NV], g[NV], s[NV];
    if (!AHEAD) load(row);
#pragma unroll
    for (int j = 0; j < NV; j++) {
      h[j] = nh[j], g[j] = ng[j];
      s[j].zero();
      // (a row ahead as well: 140 us in place of 120 for 8192 x 8192)
      if (along && row < a.n) at.load(a.dH, (size_t)row * a.lddh, j, s[j]);
    }
    if (AHEAD) load(row + step);
    Two sums(0.f, 0.f), dots(0.f, 0.f);
    uint4 *const groups = reinterpret_cast<uint4 *>(s_w + (TEAM ? E : 2) * pitch) + mine * 2 * team * NV;
    if constexpr (LIE == kShifted) {
      // (over_team ends the reads of the row before)
#pragma unroll
      for (int j = 0; j < NV; j++) {
        groups[j * team + at.me] = make_uint4(h[j].w[0], h[j].w[1], h[j].w[2], h[j].w[3]);
        groups[(NV + j) * team + at.me] = make_uint4(g[j].w[0], g[j].w[1], g[j].w[2], g[j].w[3]);
      }
      if (TEAM) __syncwarp();
      else __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < NV; j++) {
      float x[E], y[E], w[E];
      if constexpr (LIE == kShifted) {
        const int next = j * team + at.me + 1;
        const bool is = next < team * NV;
        straight<DT>(h[j], is ? groups[next] : make_uint4(0, 0, 0, 0), shift).get(x);
        straight<DT>(g[j], is ? groups[NV * team + next] : make_uint4(0, 0, 0, 0), shift).get(y);
#pragma unroll
        for (int q = 0; q < E; q++) w[q] = at.w0[(j * team + at.me) * E + q];
      } else {
        h[j].get(x), g[j].get(y);
        at.weights(a.w, a.w32, j, w);
      }
#pragma unroll
      for (int q = 0; q < E; q += 2) {
        const Two x2(x[q], x[q + 1]);
        sums = fma2(x2, x2, sums);
        dots = fma2(Two(y[q], y[q + 1]) * Two(w[q], w[q + 1]), x2, dots);
      }
    }
    float sum = sums.get().x + sums.get().y, dot = dots.get().x + dots.get().y;
    over_team<TEAM>(sum, dot, Plus(), s_sum, turn);
    if (row >= a.n) continue;
    const float rho = rsqrtf(sum * by_d + a.eps);
    const float c = rho * dot * by_d;   // mean(a xn)
    const Two rho2(rho, rho), c2(-c, -c);
#pragma unroll
    for (int j = 0; j < NV; j++) {
      float x[E], y[E], w[E], v[E];
      h[j].get(x), g[j].get(y), s[j].get(v);
      at.weights(a.w, a.w32, j, w);
#pragma unroll
      for (int q = 0; q < E; q += 2) {
        const Two xn = Two(x[q], x[q + 1]) * rho2, y2(y[q], y[q + 1]);
        dw2[j][q / 2] = fma2(y2, xn, dw2[j][q / 2]);
        const float2 f = fma2(fma2(xn, c2, y2 * Two(w[q], w[q + 1])), rho2, Two(v[q], v[q + 1])).get();
        x[q] = f.x, x[q + 1] = f.y;
      }
      if (a.dX) {
        h[j].set(x);
        at.store(a.dX, (size_t)row * a.lddx, j, h[j]);
      }
    }
  }
  float dw[NV][E];
#pragma unroll
  for (int j = 0; j < NV; j++)
#pragma unroll
    for (int q = 0; q < E; q += 2) {
      const float2 f = dw2[j][q / 2].get();
      dw[j][q] = f.x, dw[j][q + 1] = f.y;
    }
  if (!a.part) return;
  float *const part = a.part + (size_t)blockIdx.x * a.d;
  if (TEAM) {
    constexpr int PITCH = LANES * NV * E;
#pragma unroll
    for (int j = 0; j < NV; j++)
#pragma unroll
      for (int q = 0; q < E; q++) s_dw[mine * PITCH + at.at(j, q) + shift] = dw[j][q];
    __syncthreads();
    for (int i = tid; i < a.d; i += kTeamThreads) {
      float x = 0.f;
      for (int t = 0; t < ROWS; t++)
        x += s_dw[t * PITCH + i + (LIE == kShifted ? shift_of<DT>(a.H, a.ldh, (long)blockIdx.x * ROWS + t) : 0)];
      part[i] = x;
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; j++)
#pragma unroll
      for (int q = 0; q < E; q++) {
        const int i = at.at(j, q);
        if (at.in(i)) part[i] = dw[j][q];
      }
  }
}

// dw from the CTAs' parts: 32 columns a CTA, 16 threads a column, in a fixed order.
constexpr int kJoin = 16;
__global__ void __launch_bounds__(32 * kJoin) k_norm_join(const float *part, int parts, int d, void *dW, int dtype) {
  __shared__ float s[kJoin][32];
  next_may_start();
  wait_for_previous();
  const int c = threadIdx.x & 31, g = threadIdx.x >> 5, i = blockIdx.x * 32 + c;
  float x = 0.f;
  if (i < d)
#pragma unroll 4
    for (int p = g; p < parts; p += kJoin) x += part[(size_t)p * d + i];
  s[g][c] = x;
  __syncthreads();
  if (g || i >= d) return;
#pragma unroll
  for (int t = 1; t < kJoin; t++) x += s[t][c];
  if (dtype == OS2_F32) static_cast<float *>(dW)[i] = x;
  else if (dtype == OS2_BF16) static_cast<__nv_bfloat16 *>(dW)[i] = __float2bfloat16_rn(x);
  else static_cast<__half *>(dW)[i] = __float2half_rn(x);
}

// CTAs of the gradient.
template <int E, Lie LIE>
Grid grad_grid(int n, int d) {
  return grad_shape<E, LIE>(d, [&](auto team, auto nv, auto most) {
    return grid_for(n, span(d, E, LIE), decltype(team)::value, decltype(nv)::value, E, sm_threads(decltype(most)::value));
  });
}
int ctas(int n, int d, int dtype, Lie lie) {
  if (dtype == OS2_F32)
    return lie == kGroups ? grad_grid<4, kGroups>(n, d).ctas : lie == kShifted ? grad_grid<4, kShifted>(n, d).ctas : grad_grid<4, kEntries>(n, d).ctas;
  return lie == kGroups ? grad_grid<8, kGroups>(n, d).ctas : lie == kShifted ? grad_grid<8, kShifted>(n, d).ctas : grad_grid<8, kEntries>(n, d).ctas;
}

template <int DT, Lie LIE>
cudaError_t launch(const Args &a, cudaStream_t s) {
  constexpr int E = kElems<DT>;
  return grad_shape<E, LIE>(a.d, [&](auto team, auto nv, auto most) {
    constexpr int T = decltype(team)::value, NV = decltype(nv)::value, MOST = decltype(most)::value;
    const Grid g = grid_for(a.n, span(a.d, E, LIE), T, NV, E, sm_threads(MOST));
    size_t bytes = 0;
    if constexpr (LIE == kShifted && NV == 4) return cudaErrorInvalidValue;  // (not asked for: many)
    else if constexpr (LIE == kShifted) {
      bytes = shifted_bytes(T, NV, E, g.threads, 2);
      static PerDevice ready;
      const cudaError_t e = os2_set_smem(ready, k_norm_grad<DT, LIE, T, NV, MOST>, shifted_bytes(T, NV, E, MOST, 2));
      if (e != cudaSuccess) return e;
    }
    return launch_after(k_norm_grad<DT, LIE, T, NV, MOST>, g.ctas, g.threads, bytes, s, a);
  });
}

template <Lie LIE>
cudaError_t launch_t(const Args &a, int dtype, cudaStream_t s) {
  if (dtype == OS2_F32) return launch<OS2_F32, LIE>(a, s);
  if (dtype == OS2_BF16) return launch<OS2_BF16, LIE>(a, s);
  return launch<OS2_F16, LIE>(a, s);
}

// Whether kShifted pays, as in k_norm.cu: some rows a CTA.  us, entry by entry and shifted: 8192 x 3701
// BF16 174 and 93, 8192 x 1777 85 and 51, 20000 x 401 FP16 72 and 37; 8192 x 4095, whose 513 groups
// leave an SM one CTA, 185 and 155.
bool many(int n, int d, int dtype) {
  if (d + 7 > (dtype == OS2_F32 ? kMaxD / 2 : kMaxD)) return false;  // (shared memory)
  return n > 4L * ctas(1 << 30, d, dtype, kShifted) * (d + 7 <= 64 * (dtype == OS2_F32 ? 4 : 8) ? 8 : 1);
}

}  // namespace

extern "C" size_t os2_rmsnorm_workspace_size(int n, int d) {
  if (n < 0 || d < 1 || d > kMaxD) return 0;
  int most = 0;
  for (const int dtype : {OS2_F32, OS2_BF16})
    for (const Lie lie : {kEntries, kGroups, kShifted})
      if (lie != kShifted || d + 7 <= kMaxD) most = std::max(most, ctas(n, d, dtype, lie));
  return n == 0 ? 256 : os2_round_up((size_t)most * d * 4, 256);
}

extern "C" os2_status os2_rmsnorm_backward(int n, int d, int dtype, const void *H, int ldh, const void *weight,
                                           int weight_dtype, const void *dY, int lddy, const void *dH, int lddh, double eps,
                                           void *dX, int lddx, void *dW, void *workspace, size_t workspace_bytes,
                                           void *stream) {
  if (n < 0 || d < 1 || ldh < d || lddy < d || (dH && lddh < d) || (dX && lddx < d) || !is_dtype(dtype))
    return OS2_ERR_INVALID_ARG;
  if ((weight_dtype != OS2_F32 && weight_dtype != dtype) || !(eps >= 0) || !(eps < 1e30)) return OS2_ERR_INVALID_ARG;
  const size_t e = elem_size(dtype), we = elem_size(weight_dtype);
  if (!weight || !aligned(weight, we) || !aligned(dW, we)) return OS2_ERR_INVALID_ARG;
  if (n > 0 && (!H || !dY || !aligned(H, e) || !aligned(dY, e) || !aligned(dH, e) || !aligned(dX, e)))
    return OS2_ERR_INVALID_ARG;
  if (d > kMaxD) return OS2_ERR_UNSUPPORTED;
  if (!dX && !dW) return OS2_OK;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (n == 0) {
    if (!dW) return OS2_OK;
    return cudaMemsetAsync(dW, 0, (size_t)d * we, s) == cudaSuccess ? OS2_OK : OS2_ERR_CUDA;
  }
  Args a = {};
  a.n = n, a.d = d;
  a.H = H, a.ldh = ldh, a.dY = dY, a.lddy = lddy, a.dH = dH, a.lddh = lddh, a.dX = dX, a.lddx = lddx;
  a.w = weight, a.w32 = weight_dtype == OS2_F32;
  a.eps = (float)eps;
  const bool groups = on16(H, ldh, e) && on16(dY, lddy, e) && (!dH || on16(dH, lddh, e)) && (!dX || on16(dX, lddx, e)) && aligned(weight, 16) &&
                      d % (16 / e) == 0;
  const bool shifted = same16(dY, lddy, H, ldh, e) && (!dH || same16(dH, lddh, H, ldh, e)) &&
                       (!dX || same16(dX, lddx, H, ldh, e)) && many(n, d, dtype);
  const Lie lie = groups ? kGroups : shifted ? kShifted : kEntries;
  a.part = dW ? static_cast<float *>(workspace) : nullptr;
  const int grid = ctas(n, d, dtype, lie);
  if (dW && (!workspace || workspace_bytes < os2_rmsnorm_workspace_size(n, d) || !aligned(workspace, 256)))
    return OS2_ERR_WORKSPACE;
  cudaError_t err = lie == kGroups    ? launch_t<kGroups>(a, dtype, s)
                    : lie == kShifted ? launch_t<kShifted>(a, dtype, s)
                                      : launch_t<kEntries>(a, dtype, s);
  if (err == cudaSuccess && dW)
    err = launch_after(k_norm_join, (d + 31) / 32, 32 * kJoin, 0, s, a.part, grid, d, dW, weight_dtype);
  return err == cudaSuccess ? OS2_OK : OS2_ERR_CUDA;
}
