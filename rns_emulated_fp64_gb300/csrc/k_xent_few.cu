// The forward pass of k_xent.cu for few rows, where W's bytes bound it: a token
// scored, a few streams decoded.  The same stream as k_i8few.cu: a ring of TMA
// copies (some 200 KB an SM in flight) brings 128 rows of W x 64 terms a stage
// with the matching terms of the packed rows of H; eight warps take 16 rows of W
// each (mma.sync.m16n8k16, whose 16 terms may be any as long as both operands'
// are the same, so fragments are 16-byte reads); a cluster of C CTAs shares out the
// terms of a tile and joins its sums, in the order of the CTAs, through distributed
// shared memory.
//
// A thread keeps the running maximum and sum of exponentials of its columns over
// all tiles of its CTA, so that a row leaves one pair a CTA for k_xent_join.
// Sums are taken out of the accumulators every 1024 terms, as in k_xent.cu.
// Measured with packing and joining: one row 17 us for 32000 x 1024 (3.8 TB/s), 28 for
// 32000 x 2048 and 88 for 128256 x 2048 (6.0 TB/s; the copy rate is 6.8): a start of 4 us and
// an end of 2 do not shrink with W.  Two groups of warps, as in k_i8few.cu, gain nothing
// here (17.6 us), where nothing is widened.
#include "i8.cuh"
#include "xent.cuh"

using namespace os2i8;
using namespace os2xent;

namespace {

constexpr int kWarps = 8, kThreadsFew = 32 * kWarps + 32;
constexpr uint32_t kW = 128 * kBK * 2;   // a stage's rows of W: 64 terms

template <int NG>
struct Shape {
  static constexpr uint32_t stage = kW + NG * 8 * kBK * 2;
  static constexpr uint32_t part = kWarps * NG * 32 * 16;  // a tile's sums, one side
  static constexpr uint32_t stats = kWarps * NG * 8 * 8;      // a pair of each warp and row
  static constexpr int stages = (int)((227 * 1024 - 1024 - 512 - stats - 2 * part) / stage);
  static constexpr size_t smem = 1024 + (size_t)stages * stage + 2 * part + stats + 512;
};

template <bool BF16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  if (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct Job {
  int v, tiles, stages;
  int cluster, clusters;
  const int *count, *label;
  float *zlabel;
  float2 *part;     // [rows][parts], this grid's CTAs the parts
  int parts;
};

template <bool BF16, int NG>
__global__ void __launch_bounds__(kThreadsFew, 1)
    k_xent_few(const __grid_constant__ CUtensorMap mapW, const __grid_constant__ CUtensorMap mapH,
               const Job j, int *status) {
  using S = Shape<NG>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~uintptr_t(1023));
  uint8_t *sPart = smem + S::stages * S::stage;
  float2 *stats = reinterpret_cast<float2 *>(sPart + 2 * S::part);  // [kWarps][NG * 8]
  uint64_t *full = reinterpret_cast<uint64_t *>(sPart + 2 * S::part + S::stats);
  uint64_t *empty = full + S::stages, *part = empty + S::stages;  // part: [2][kWarps]
  volatile int *s_abort = reinterpret_cast<volatile int *>(part + 2 * kWarps);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank(), first = (int)blockIdx.x / j.cluster;
  const int s0 = rank * j.stages / j.cluster, s1 = (rank + 1) * j.stages / j.cluster;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::stages; s++) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kWarps);
    }
    for (int s = 0; s < 2 * kWarps; s++) mbar_init(&part[s], 1);
    *s_abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&mapW);
    tma_prefetch_desc(&mapH);
  }
  next_may_start();
  __syncthreads();
  cluster_arrive();  // waited for before anything is sent to another CTA

  auto gave_up = [&]() {
    *s_abort = 1;
    set_status(status, OS2_ERR_TIMEOUT);
    return false;
  };

  if (warp == kWarps) {
    // ------------------------------------------------------------ TMA
    if (lane == 0) {
      auto weights = [&](int st, int t, int ks) {
        mbar_arrive_expect_tx(&full[st], S::stage);
        tma_load_3d(smem + st * S::stage, &mapW, &full[st], ks * kBK, t * 128, 0);
      };
      // the first turn of the ring: W, an input of the call (complete since the kernel in
      // front passed start_call; a copy of W is waited for: overlap is off); then, once the
      // kernel in front has packed them, H's rows
      int i = 0;
      for (int t = first; t < j.tiles && i < S::stages; t += j.clusters)
        for (int ks = s0; ks < s1 && i < S::stages; ks++) weights(i++, t, ks);
      wait_for_previous();
      int st = 0;
      uint32_t ph = 0, used = 0, last_par = 0;
      bool ok = true;
      i = 0;
      for (int t = first; ok && t < j.tiles; t += j.clusters)
        for (int ks = s0; ks < s1; ks++, i++) {
          if (i >= S::stages) {
            if (!mbar_wait_bounded(&empty[st], ph ^ 1, s_abort, kWaitLimit)) {
              ok = gave_up();
              break;
            }
            weights(st, t, ks);
          }
          tma_load_3d(smem + st * S::stage + kW, &mapH, &full[st], ks * kBK, 0, 0);
          used |= 1u << st;
          last_par = (last_par & ~(1u << st)) | (ph << st);
          if (++st == S::stages) {
            st = 0;
            ph ^= 1;
          }
        }
      for (int s = 0; s < S::stages; s++)
        if (used >> s & 1) {
          volatile int no_abort = 0;
          mbar_wait_bounded(&full[s], (last_par >> s) & 1, &no_abort, kWaitLimit);
        }
    }
    __syncwarp();
    cluster_wait();
  } else {
    // ------------------------------------------------------------ products
    const int g = lane >> 2, t4 = lane & 3;
    // Lane row g takes row gw of eight, of W and of H: no bank conflicts (k_i8few.cu).
    const int gw = g >> 1 | (g & 1) << 2;
    const uint32_t w0 = (uint32_t)(warp * 16 + gw) * 128, w1 = w0 + 8 * 128;
    // Entry (q, e): row ch + 8 (e / 2) of W, packed row 8 q + t4 + 4 (e % 2) of H.  Rows of
    // lane row g meet in CTA g C / 8; two sides are enough (k_i8few.cu).
    const int owner = g * j.cluster / 8;
    const bool mine = owner == rank;
    wait_for_previous();
    cluster_wait();
    const int m = *j.count;
    int label[NG][2];
    float top[NG][2], total[NG][2];
#pragma unroll
    for (int q = 0; q < NG; q++)
#pragma unroll
      for (int e = 0; e < 2; e++) {
        const int r = q * 8 + t4 + 4 * e;
        label[q][e] = r < m ? j.label[r] : -1;
        top[q][e] = -INFINITY;
        total[q][e] = 0.f;
      }
    int st = 0, side = 0;
    uint32_t ph = 0, pph = 0;
    bool ok = true;
    for (int t = first; ok && t < j.tiles; t += j.clusters) {
      float acc[NG][4], sum[NG][4];
#pragma unroll
      for (int q = 0; q < NG; q++)
#pragma unroll
        for (int e = 0; e < 4; e++) acc[q][e] = 0.f, sum[q][e] = 0.f;
      for (int ks = s0; ks < s1; ks++) {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&full[st], ph, s_abort, kWaitLimit));
        if (!ok) break;
        const uint32_t base = smem_u32(smem + st * S::stage);
#pragma unroll
        for (int h = 0; h < 2; h++) {
          const uint32_t at = (uint32_t)((4 * h + t4) ^ gw) << 4;  // 8 terms
          const uint4 a = lds16(base + w0 + at), b = lds16(base + w1 + at);
#pragma unroll
          for (int q = 0; q < NG; q++) {
            const uint4 x = lds16(base + kW + (uint32_t)(q * 8 + gw) * 128 + at);
            mma<BF16>(acc[q], a.x, b.x, a.y, b.y, x.x, x.y);
            mma<BF16>(acc[q], a.z, b.z, a.w, b.w, x.z, x.w);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
        if (++st == S::stages) {
          st = 0;
          ph ^= 1;
        }
        if ((ks - s0) % 16 == 15 || ks == s1 - 1) {
#pragma unroll
          for (int q = 0; q < NG; q++)
#pragma unroll
            for (int e = 0; e < 4; e++) sum[q][e] += acc[q][e], acc[q][e] = 0.f;
        }
      }
      if (!ok) break;
      if (j.cluster > 1) {
        const uint32_t bar = smem_u32(&part[side * kWarps + warp]);
        const uint32_t buf = smem_u32(sPart + side * S::part);
        const int per = 32 / j.cluster;  // lanes of a part
        const uint32_t to = mapa_shared(buf, owner) + (uint32_t)warp * NG * 512 +
                            (uint32_t)(rank * per + (lane & (per - 1))) * 16;
        const uint32_t to_bar = mapa_shared(bar, owner);
        if (lane == 0) mbar_arrive_expect_tx(&part[side * kWarps + warp], NG * 512);
#pragma unroll
        for (int q = 0; q < NG; q++)
          st_async16(to + q * 512, to_bar, __float_as_int(sum[q][0]), __float_as_int(sum[q][1]),
                     __float_as_int(sum[q][2]), __float_as_int(sum[q][3]));
        ok = __all_sync(0xffffffffu,
                        mbar_wait_bounded(&part[side * kWarps + warp], pph, s_abort, kWaitLimit));
        if (!ok) break;
        const uint32_t from = buf + (uint32_t)warp * NG * 512 + (uint32_t)(lane & (per - 1)) * 16;
#pragma unroll
        for (int q = 0; q < NG; q++) {
#pragma unroll
          for (int e = 0; e < 4; e++) sum[q][e] = 0.f;
          for (int p = 0; p < j.cluster; p++) {
            const uint4 x = lds16(from + q * 512 + (uint32_t)(p * per) * 16);
            sum[q][0] += __uint_as_float(x.x);
            sum[q][1] += __uint_as_float(x.y);
            sum[q][2] += __uint_as_float(x.z);
            sum[q][3] += __uint_as_float(x.w);
          }
        }
        side ^= 1;
        if (side == 0) pph ^= 1;
      }
      if (mine)
#pragma unroll
        for (int e = 0; e < 2; e++) {
          const int ch = t * 128 + warp * 16 + gw;
#pragma unroll
          for (int q = 0; q < NG; q++)
#pragma unroll
            for (int h = 0; h < 2; h++) {
              const float z = sum[q][2 * h + e];
              if (ch + 8 * h < j.v) {
                add_exp(top[q][e], total[q][e], z * kLog2e, 1.f);
                if (ch + 8 * h == label[q][e]) j.zlabel[q * 8 + t4 + 4 * e] = z;
              }
            }
        }
      __syncwarp();
    }
    if (!ok) gave_up();
    // the CTA's pair of each row: over the lanes of a column, then over the warps
#pragma unroll
    for (int q = 0; q < NG; q++)
#pragma unroll
      for (int e = 0; e < 2; e++) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          const float x = __shfl_xor_sync(0xffffffffu, top[q][e], o);
          const float y = __shfl_xor_sync(0xffffffffu, total[q][e], o);
          add_exp(top[q][e], total[q][e], x, y);
        }
        if (g == 0) stats[warp * NG * 8 + q * 8 + t4 + 4 * e] = make_float2(top[q][e], total[q][e]);
      }
  }
  // the pairs are written; and no CTA leaves while another may still send to it
  __syncwarp();
  cluster_sync();
  if ((int)threadIdx.x < NG * 8 && (int)threadIdx.x < *j.count) {
    float top = -INFINITY, total = 0.f;
    for (int w = 0; w < kWarps; w++) {
      const float2 p = stats[w * NG * 8 + threadIdx.x];
      add_exp(top, total, p.x, p.y);
    }
    j.part[(size_t)threadIdx.x * j.parts + blockIdx.x] = make_float2(top, total);
  }
}

template <bool BF16, int NG>
cudaError_t launch(const XentFewArgs &a, int *parts, cudaStream_t s) {
  using S = Shape<NG>;
  static PerDevice ready;
  const cudaError_t attr_err = os2_set_smem(ready, k_xent_few<BF16, NG>, S::smem);
  if (attr_err != cudaSuccess) return attr_err;
  Job j;
  j.v = a.v;
  j.tiles = (a.v + 127) / 128;
  j.stages = (a.k + kBK - 1) / kBK;
  few_clusters(reinterpret_cast<const void *>(k_xent_few<BF16, NG>), kThreadsFew, S::smem, j.tiles,
               j.stages, &j.cluster, &j.clusters);
  CUtensorMap mw, mh;
  if (!make_map(&mw, a.W, BF16, a.k, a.v, a.ldw, false) ||
      !make_map(&mh, a.Hc, BF16, a.k, a.n, a.hpitch, false, NG * 8))
    return cudaErrorInvalidValue;
  j.count = a.count;
  j.label = a.label;
  j.zlabel = a.zlabel;
  j.part = a.part;
  *parts = j.parts = j.cluster * j.clusters;
  return launch_cluster(k_xent_few<BF16, NG>, j.cluster, j.parts, kThreadsFew, S::smem, a.overlap, s,
                        mw, mh, j, a.status);
}

template <bool BF16>
cudaError_t launch_t(const XentFewArgs &a, int *parts, cudaStream_t s) {
  return a.n <= 8 ? launch<BF16, 1>(a, parts, s) : launch<BF16, 2>(a, parts, s);
}

}  // namespace

cudaError_t launch_xent_few(const XentFewArgs &a, int *parts, cudaStream_t s) {
  return a.bf16 ? launch_t<true>(a, parts, s) : launch_t<false>(a, parts, s);
}
