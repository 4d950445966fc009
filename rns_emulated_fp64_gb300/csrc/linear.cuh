// What the linear layer's kernels share (k_linear.cu, k_linear_few.cu).
#pragma once
#include "act.cuh"
#include "mm2_epi.cuh"

struct LinearArgs {
  int m, n, k;             // tokens, outputs, terms (>= 1 each)
  bool bf16;
  const uint16_t *X, *W;   // rows that TMA takes
  long ldx, ldw;
  const void *bias;        // of FP32 (b32) or of the operands' type, or null
  bool b32;
  int act;
  const uint16_t *R;       // residual, or null
  long ldr;
  uint16_t *Y, *pre;       // pre may be null
  long ldy, ldp;
  float by;                // dx in FP16: the sums times this
  int *status;
};

// A tile's columns are outputs and its rows tokens in k_linear.cu; k_linear_few.cu turns that
// round for few tokens.  How it would go about it, and its estimate of the time.
struct LinearPlan {
  int nt, cluster;   // tokens of a tile, CTAs that share its terms
  double us;
};
LinearPlan linear_few_plan(int m, int n, int k, bool more);  // (more: an activation, or pre)
// w_mn: W is k x n (dx = D W with D as X), else n x k.
cudaError_t launch_linear_few(const LinearArgs &a, bool w_mn, cudaStream_t s);

namespace os2lin {

template <bool BF16>
__device__ __forceinline__ float widen16(uint16_t b) {
  return BF16 ? __uint_as_float((uint32_t)b << 16) : __half2float(__ushort_as_half(b));
}
template <bool BF16>
__device__ __forceinline__ float bias_at(const void *bias, bool b32, int i) {
  return b32 ? __ldg(static_cast<const float *>(bias) + i) : widen16<BF16>(__ldg(static_cast<const uint16_t *>(bias) + i));
}

// Four neighbouring entries of a row, of which `left` exist; whole: in one access.
__device__ __forceinline__ uint2 load4(const uint16_t *p, int left, bool whole) {
  if (whole && left >= 4) return *reinterpret_cast<const uint2 *>(p);
  uint32_t w[2] = {};
#pragma unroll
  for (int i = 0; i < 4; i++)
    if (i < left) w[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
  return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void store4(uint16_t *p, uint2 v, int left, bool whole) {
  if (whole && left >= 4) {
    *reinterpret_cast<uint2 *>(p) = v;
    return;
  }
  const uint32_t w[2] = {v.x, v.y};
#pragma unroll
  for (int i = 0; i < 4; i++)
    if (i < left) p[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
}

}  // namespace os2lin
