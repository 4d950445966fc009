// What the cross entropy's kernels share (k_xent.cu, k_xent_few.cu).
#pragma once
#include "mm2.cuh"

namespace os2xent {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// (top, sum) stands for sum 2^top; (x, y) is added to it.
__device__ __forceinline__ void add_exp(float &top, float &sum, float x, float y) {
  const float t = fmaxf(top, x);
  // nothing but -inf so far: exponents against 0 (every term is 0)
  const float t0 = t == -INFINITY ? 0.f : t;
  sum = sum * ex2(top - t0) + y * ex2(x - t0);
  top = t;
}

}  // namespace os2xent

struct XentFewArgs {
  int n, k, v;
  bool bf16;
  const void *Hc;              // packed rows [n][hpitch]
  long hpitch;
  const void *W;
  long ldw;
  bool overlap;                // W is the caller's: it may be read before the kernel in front ends
  const int *count, *label;
  float *zlabel;
  float2 *part;                // [n][parts]
  int *status;
};
// Up to this many rows of H, the forward pass is k_xent_few: 28 us for one or 8 rows and 31
// for 16 (k = 2048, v = 32000), against 37 to 39 with the tiles of k_xent.cu for 17 to 64.
constexpr int kXentFew = 16;
// At most one pair a row and SM; *parts receives the pairs of a row.
cudaError_t launch_xent_few(const XentFewArgs &a, int *parts, cudaStream_t s);
