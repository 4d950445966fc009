// What the 8-bit product's kernels share (k_i8.cu, k_i8few.cu, k_i8tc.cu).
#pragma once
#include "mm2.cuh"

struct I8Args {
  int m, n, k;                 // tokens, channels, terms (k >= 1)
  const void *tokens;          // FP16 integers [m][pitch], pitch a multiple of 8, 16-byte aligned
  long pitch;
  const void *W;               // int8 [n][ldw], ldw a multiple of 16, 16-byte aligned
  long ldw;
  const float *sa, *sb, *bias; // bias may be null
  void *y;
  long ldy;
  int out_dtype;
  bool overlap;                // W is the caller's: it may be read before the kernel in front ends
  int *slots;                  // I8Sizes
  unsigned *done;              // zero before the launch
  int *status;
};
struct I8Sizes {
  int counters;                // of `done`
  size_t slot_ints;
};
// k_i8few: m <= kI8Few tokens, mma.sync, no slots or counters; k_i8tc: tcgen05.
constexpr int kI8Few = 64;
cudaError_t launch_i8few(const I8Args &a, cudaStream_t s);
I8Sizes i8tc_sizes(int m, int n, int k);
cudaError_t launch_i8tc(const I8Args &a, cudaStream_t s);

namespace os2i8 {

using namespace os2mm;

// The work: tiles of CH channels x NT tokens over stages of 128 terms.  Whole
// tiles go round the workers; those that are left over after the last whole wave
// are cut along k into `parts` for as many workers.
struct I8Job {
  int m, n;            // tokens, channels
  int tiles_c, tiles_t, stages;  // tiles of channels and tokens, stages of 128 terms
  int workers;         // pairs of CTAs
  int waves;           // whole tiles of each worker
  int rest, parts;     // tiles left over, parts of each (rest * parts <= workers)
  int out_dtype;
  const float *sa, *sb, *bias;
  void *y;
  long ldy;
  int *slots;          // [workers][2 CTAs][NT / 4][128][4] partial sums
  unsigned *done;      // [rest][2] stages finished, zero before the launch
};

__device__ __forceinline__ uint32_t add2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ void widen(uint32_t w, uint32_t &lo, uint32_t &hi) {
  const uint32_t x = w ^ 0x80808080u;
  lo = add2(__byte_perm(x, 0x64646464u, 0x4140), 0xE480E480u);  // - 1152
  hi = add2(__byte_perm(x, 0x64646464u, 0x4342), 0xE480E480u);
}

// The segments of a worker, in order: f(tile, first stage, end stage, index of the
// cut tile or -1 for a whole one).  Every role walks the same.
template <class F>
__device__ __forceinline__ void for_segments(const I8Job &j, int worker, F &&f) {
  const int last = worker < j.rest * j.parts ? 1 : 0;
  for (int w = 0; w < j.waves + last; w++) {
    int t = w * j.workers + worker, s0 = 0, s1 = j.stages, cut = -1;
    if (w == j.waves) {
      const int r = worker / j.parts, part = worker - r * j.parts;
      t = j.waves * j.workers + r;
      s0 = part * j.stages / j.parts;
      s1 = (part + 1) * j.stages / j.parts;
      if (j.parts > 1) cut = r;
    }
    if (!f(t, s0, s1, cut)) return;
  }
}

__device__ __forceinline__ void store_y(void *y, int dtype, size_t i, float v) {
  if (dtype == OS2_F32) static_cast<float *>(y)[i] = v;
  else if (dtype == OS2_BF16) static_cast<__nv_bfloat16 *>(y)[i] = __float2bfloat16_rn(v);
  else static_cast<__half *>(y)[i] = __float2half_rn(v);
}

// How the eight warps of a CTA that hold a part of a cut tile learn whether it
// was the last one: two barriers of shared memory (a: 8 arrivals, b: 1), waited
// for with a limit like every other.
struct I8Join {
  uint64_t *a, *b;
  volatile unsigned *last;
  uint32_t parity;
};
// After the part (`mine` stages of a tile's `stages`) is in its slot; every lane
// of the eight warps calls it, `elected` is true for one thread.  0: not the
// last, 1: the last, -1: gave up.
__device__ __forceinline__ int last_part(I8Join &jn, unsigned *counter, int mine, int stages,
                                         bool elected, volatile int *s_abort) {
  __threadfence();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(jn.a);
  if (elected) {
    if (!mbar_wait_bounded(jn.a, jn.parity, s_abort, kWaitLimit)) *s_abort = 1;
    else {
      const unsigned before = atomicAdd(counter, (unsigned)mine);
      *jn.last = before + (unsigned)mine == (unsigned)stages;
      __threadfence();
      mbar_arrive(jn.b);
    }
  }
  __syncwarp();
  const bool ok = mbar_wait_bounded(jn.b, jn.parity, s_abort, kWaitLimit);
  jn.parity ^= 1;
  if (!__all_sync(0xffffffffu, ok)) return -1;
  return *jn.last ? 1 : 0;  // (the parts are read past L1, after the elected thread's fence)
}

inline void i8_fill(I8Job &j, const I8Args &a) {
  j.out_dtype = a.out_dtype;
  j.sa = a.sa;
  j.sb = a.sb;
  j.bias = a.bias;
  j.y = a.y;
  j.ldy = a.ldy;
  j.slots = a.slots;
  j.done = a.done;
}

// 8-bit rows: box 128 terms x 128 rows, 128-byte swizzle.
inline bool map_w(CUtensorMap *map, const void *base, long k, long rows, long pitch) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)k, (cuuint64_t)rows, 1};
  cuuint64_t strides[2] = {(cuuint64_t)pitch, (cuuint64_t)pitch * (cuuint64_t)rows};
  cuuint32_t box[3] = {(cuuint32_t)kStageK, (cuuint32_t)kHalf, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ------------------------------------------------ streams in clusters (host)
// The cluster size of a streaming kernel (k_i8few.cu, k_xent_few.cu) for `tiles`
// tiles of `stages` 16 KB stages, by an estimate in microseconds: a stage takes a
// CTA 0.19 (what its SM can take in), or 0.0026 for each CTA that streams at the same
// time (memory); a tile's end takes 0.3, and 1.0 more where parts are joined.
void few_clusters(const void *kernel, int threads, size_t smem, int tiles, int stages,
                  int *cluster, int *clusters);

// Launches a kernel in clusters of `cluster` CTAs; overlap: before the kernel in
// front of it on the stream has ended (it waits for that itself).
template <class... P, class... A>
cudaError_t launch_cluster(void (*kernel)(P...), int cluster, int grid, int block, size_t smem,
                           bool overlap, cudaStream_t s, const A &...args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)cluster, 1, 1};
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = overlap ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}

}  // namespace os2i8
