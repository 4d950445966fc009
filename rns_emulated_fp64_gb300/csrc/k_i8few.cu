// The 8-bit product of k_i8.cu for few tokens, where the weights' bytes bound it.
//
// A CTA streams its share of the weights through a ring of TMA copies (up to 200
// KB an SM in flight, whatever the registers hold) with the tokens' matching
// terms beside them.  Eight warps take 16 channels each of a stage of 128 channels
// x 128 terms (up to 16 tokens, two groups of eight take the stages in turn: one reads
// shared memory while the other multiplies).  A lane reads 16 bytes of two channels
// at a time, widens them to FP16 in registers (exact) and multiplies with
// mma.sync.m16n8k16, whose fragments are the lanes' own bytes: the 16 terms of an
// instruction may be any, as long as the tokens' are the same, so lane t's 16
// consecutive bytes serve four
// instructions.  tcgen05 would need the FP16 weights back in shared memory
// (k_i8tc.cu: half the rate for 16 tokens).  FP32 accumulators are exact for 1024
// terms (2^24); they are emptied into int32 after those.
//
// A cluster of C CTAs takes a tile of 128 channels, each CTA its C-th of the terms,
// so that a few thousand channels already use every SM.  The int32 sums of a
// channel meet in the CTA that stores it, sent there through distributed shared
// memory by stores whose bytes the receiving warp waits for.  (Parts joined
// through global memory, with stages dealt out evenly over single CTAs, took 3 us
// longer: 12.5 us instead of 8 for 4096 x 4096 and one token.)
//
// Warps: 8 or 16 as above, one more for TMA.  The first weights are asked for, and the
// channels' scales and bias read, before the kernel waits for the one in front of it on the
// stream, which quantises the tokens: they are inputs of the call, and nothing in front
// of that kernel can be writing them still (start_call).  Every wait is bounded, as in
// mm2.cuh.
//
// Measured with the quantising launch: one token 7.6 us for 4096 x 4096 weights, 16.4
// for 14336 x 4096 and 16.8 for 32000 x 2048 (3.9 TB/s; a kernel that only reads takes 6.2,
// 12.4 and 13.6); 12 tokens 8.8, 17.9 and 18.7; 64 tokens 16.4, 33.4 and 35.7.  The rest is the start of the ring, 500 cycles
// of shared memory a stage (weights in and out, tokens) against 740 of DRAM, and tiles
// that do not divide by the SMs.
#include "i8.cuh"
#include "i8_ring.h"

using namespace os2i8;

namespace {

static_assert(kFewW == 128 * kStageK && Few<1>::block == 8 * kBK * 2, "a stage of the ring");

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
struct FewJob {
  int m, n, tiles, stages;
  int cluster, clusters;     // CTAs of a cluster (1, 2, 4 or 8), clusters of the grid
  int out_dtype;
  const float *sa, *sb, *bias;
  void *y;
  long ldy;
};

template <int NG>
__global__ void __launch_bounds__(Few<NG>::threads, 1)
    k_i8few(const __grid_constant__ CUtensorMap mapW, const __grid_constant__ CUtensorMap mapT,
            const FewJob j, int *status) {
  using F = Few<NG>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~uintptr_t(1023));
  uint8_t *sPart = smem + F::stages * F::stage;
  uint64_t *full = reinterpret_cast<uint64_t *>(sPart + 2 * F::part);
  uint64_t *empty = full + F::stages, *part = empty + F::stages;  // part: [2][kFewWarps]
  volatile int *s_abort = reinterpret_cast<volatile int *>(part + 2 * kFewWarps);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank(), first = (int)blockIdx.x / j.cluster;
  // this CTA's stages of every tile
  const int s0 = rank * j.stages / j.cluster, s1 = (rank + 1) * j.stages / j.cluster;

  if (threadIdx.x == 0) {
    for (int s = 0; s < F::stages; s++) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kFewWarps);  // of the group that takes it
    }
    for (int s = 0; s < 2 * kFewWarps; s++) mbar_init(&part[s], 1);
    *s_abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&mapW);
    tma_prefetch_desc(&mapT);
  }
  next_may_start();
  __syncthreads();
  cluster_arrive();  // waited for before anything is sent to another CTA

  auto gave_up = [&]() {
    *s_abort = 1;
    set_status(status, OS2_ERR_TIMEOUT);
    return false;
  };

  if (warp == F::all) {
    // ------------------------------------------------------------ TMA
    if (lane == 0) {
      auto weights = [&](int st, int tc, int ks) {
        mbar_arrive_expect_tx(&full[st], F::stage);
        tma_load_3d(smem + st * F::stage, &mapW, &full[st], ks * kStageK, tc * 128, 0);
      };
      auto tokens = [&](int st, int ks) {
#pragma unroll
        for (int h = 0; h < 2; h++)
          tma_load_3d(smem + st * F::stage + kFewW + h * F::block, &mapT, &full[st],
                      ks * kStageK + h * kBK, 0, 0);
      };
      // The first weights; then, once they are there, the tokens with the rest.  A long
      // stream does not ask for the whole ring at first: memory serves all that is asked for
      // side by side, so the first stage would be there as late as the last, and the
      // tokens behind it (32000 x 2048, one token: 18.0 us with the whole ring, 16.7 with
      // 6 stages; 4096 x 4096, whose 8 stages a CTA fit in the ring: 8.5 with all, 8.8 with 6).
      const int share = (j.tiles - first + j.clusters - 1) / j.clusters * (s1 - s0);
      const int ahead = share <= F::stages ? F::stages : min(6, F::stages);
      int i = 0;
      for (int t = first; t < j.tiles && i < ahead; t += j.clusters)
        for (int ks = s0; ks < s1 && i < ahead; ks++) weights(i++, t, ks);
      wait_for_previous();
      int st = 0;
      uint32_t ph = 0, used = 0, last_par = 0;
      bool ok = true;
      i = 0;
      for (int t = first; ok && t < j.tiles; t += j.clusters)
        for (int ks = s0; ks < s1; ks++, i++) {
          if (i >= ahead) {
            if (i >= F::stages &&
                !mbar_wait_bounded(&empty[st], ph ^ 1, s_abort, kWaitLimit)) {
              ok = gave_up();
              break;
            }
            weights(st, t, ks);
          }
          tokens(st, ks);
          used |= 1u << st;
          last_par = (last_par & ~(1u << st)) | (ph << st);
          if (++st == F::stages) {
            st = 0;
            ph ^= 1;
          }
        }
      for (int s = 0; s < F::stages; s++)
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
    // 16-byte piece c of a 128-byte row r of a swizzled block: c ^ (r & 7).  Lane row g
    // takes row gw of the eight: then eight lanes that read at once have two rows four
    // apart, whose pieces are in different banks (two neighbours' are in the same).
    const int gw = g >> 1 | (g & 1) << 2;
    const int group = warp / kFewWarps, cw = warp % kFewWarps;
    const uint32_t w0 = (uint32_t)(cw * 16 + gw) * 128, w1 = w0 + 8 * 128;
    int st = 0, turn = 0;
    uint32_t ph = 0;
    // Entry (q, e) of a thread: channel ch + 8 (e / 2), token 8 q + 2 t4 + e % 2.  The
    // channels of lane row g meet in CTA g C / 8 of the cluster, in group 0.  A warp
    // sends the sums of tile i + 2 after it has had everyone's of tile i + 1, which their warps
    // sent after they had read tile i: two sides are enough.
    const int owner = g * j.cluster / 8;
    const bool mine = owner == rank && group == 0;
    bool waited = false;  // for the kernel in front, and for the cluster
    bool ok = true;
    int side = 0;
    uint32_t pph = 0;
    for (int t = first; ok && t < j.tiles; t += j.clusters) {
      float acc[NG][4];
      int sum[NG][4];
#pragma unroll
      for (int q = 0; q < NG; q++)
#pragma unroll
        for (int e = 0; e < 4; e++) acc[q][e] = 0.f, sum[q][e] = 0;
      const int ch = t * 128 + cw * 16 + gw;
      float sb[2], bias[2];
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const bool in = ch + 8 * h < j.n;
        sb[h] = in ? j.sb[ch + 8 * h] : 0.f;
        bias[h] = in && j.bias ? j.bias[ch + 8 * h] : 0.f;
      }
      int held = 0;  // stages in acc
      for (int ks = s0; ks < s1; ks++) {
        if (turn != group) {
          turn = (turn + 1) % F::groups;
          if (++st == F::stages) {
            st = 0;
            ph ^= 1;
          }
          continue;
        }
        turn = (turn + 1) % F::groups;
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&full[st], ph, s_abort, kWaitLimit));
        if (!ok) break;
        const uint32_t base = smem_u32(smem + st * F::stage);
#pragma unroll
        for (int h = 0; h < 2; h++) {
          const uint32_t at = (uint32_t)((4 * h + t4) ^ gw) << 4;
          const uint4 a = lds16(base + w0 + at), b = lds16(base + w1 + at);
          uint4 x[NG][2];
#pragma unroll
          for (int q = 0; q < NG; q++)
#pragma unroll
            for (int e = 0; e < 2; e++)  // the same 16 terms of token q * 8 + g
              x[q][e] = lds16(base + kFewW + h * F::block + (uint32_t)(q * 8 + g) * 128 +
                              ((uint32_t)((2 * t4 + e) ^ g) << 4));
          const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int e = 0; e < 4; e++) {
            uint32_t a0, a1, a2, a3;
            widen(wa[e], a0, a2);
            widen(wb[e], a1, a3);
#pragma unroll
            for (int q = 0; q < NG; q++) {
              const uint4 xx = x[q][e >> 1];
              mma16816(acc[q], a0, a1, a2, a3, e & 1 ? xx.z : xx.x, e & 1 ? xx.w : xx.y);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
        if (++st == F::stages) {
          st = 0;
          ph ^= 1;
        }
        if (++held == 8) {
          held = 0;
#pragma unroll
          for (int q = 0; q < NG; q++)
#pragma unroll
            for (int e = 0; e < 4; e++) sum[q][e] += __float2int_rn(acc[q][e]), acc[q][e] = 0.f;
        }
      }
#pragma unroll
      for (int q = 0; q < NG; q++)
#pragma unroll
        for (int e = 0; e < 4; e++) sum[q][e] += __float2int_rn(acc[q][e]);
      if (!ok) break;
      if (!waited) {  // the tokens' scales and the output; the other CTAs' barriers
        wait_for_previous();
        cluster_wait();
        waited = true;
      }
      if (j.cluster * F::groups > 1) {
        // the parts of a channel's C CTAs and their groups lie side by side:
        // [C][groups][8 / C lane rows] lanes
        const uint32_t bar = smem_u32(&part[side * kFewWarps + cw]);
        const uint32_t buf = smem_u32(sPart + side * F::part) + (uint32_t)cw * NG * 512 * F::groups;
        const int per = 32 / j.cluster;  // lanes of a part
        const uint32_t to = mapa_shared(buf, owner) +
                            (uint32_t)((rank * F::groups + group) * per + (lane & (per - 1))) * 16;
        const uint32_t to_bar = mapa_shared(bar, owner);
        if (lane == 0 && group == 0)
          mbar_arrive_expect_tx(&part[side * kFewWarps + cw], NG * 512 * F::groups);
#pragma unroll
        for (int q = 0; q < NG; q++)
          st_async16(to + q * 512 * F::groups, to_bar, sum[q][0], sum[q][1], sum[q][2], sum[q][3]);
        ok = __all_sync(0xffffffffu,
                        mbar_wait_bounded(&part[side * kFewWarps + cw], pph, s_abort, kWaitLimit));
        if (!ok) break;
        if (mine) {
          const uint32_t from = buf + (uint32_t)(lane & (per - 1)) * 16;
#pragma unroll
          for (int q = 0; q < NG; q++) {
            int4 v = make_int4(0, 0, 0, 0);
            for (int p = 0; p < j.cluster * F::groups; p++) {
              const uint4 x = lds16(from + q * 512 * F::groups + (uint32_t)(p * per) * 16);
              v.x += (int)x.x;
              v.y += (int)x.y;
              v.z += (int)x.z;
              v.w += (int)x.w;
            }
            sum[q][0] = v.x;
            sum[q][1] = v.y;
            sum[q][2] = v.z;
            sum[q][3] = v.w;
          }
        }
        side ^= 1;
        if (side == 0) pph ^= 1;
      }
      if (mine)
#pragma unroll
        for (int q = 0; q < NG; q++)
#pragma unroll
          for (int e = 0; e < 4; e++) {
            const int c = ch + 8 * (e >> 1), to = q * 8 + 2 * t4 + (e & 1);
            if (c < j.n && to < j.m && OS2_DBG_GUARD(c >= 0 && j.ldy >= j.n, status))
              store_y(j.y, j.out_dtype, (size_t)to * j.ldy + c,
                      (float)sum[q][e] * j.sa[to] * sb[e >> 1] + bias[e >> 1]);
          }
      __syncwarp();
    }
    if (!ok) gave_up();
    if (!waited) cluster_wait();
  }
  // no CTA leaves while another may still send to it
  __syncwarp();
  cluster_sync();
}

template <int NG>
cudaError_t launch(const I8Args &a, cudaStream_t s) {
  using F = Few<NG>;
  static PerDevice ready;
  const cudaError_t attr_err = os2_set_smem(ready, k_i8few<NG>, F::smem);
  if (attr_err != cudaSuccess) return attr_err;
  FewJob j;
  j.m = a.m;
  j.n = a.n;
  j.tiles = (a.n + 127) / 128;
  j.stages = (a.k + kStageK - 1) / kStageK;
  few_clusters(reinterpret_cast<const void *>(k_i8few<NG>), F::threads, F::smem, j.tiles, j.stages,
               &j.cluster, &j.clusters);
  CUtensorMap mw, mt;
  if (!map_w(&mw, a.W, a.k, a.n, a.ldw) ||
      !make_map(&mt, a.tokens, false, a.k, a.m, a.pitch, false, NG * 8))
    return cudaErrorInvalidValue;
  j.out_dtype = a.out_dtype;
  j.sa = a.sa;
  j.sb = a.sb;
  j.bias = a.bias;
  j.y = a.y;
  j.ldy = a.ldy;
  return launch_cluster(k_i8few<NG>, j.cluster, j.cluster * j.clusters, F::threads, F::smem,
                        a.overlap, s, mw, mt, j, a.status);
}

int groups(int m) { return m <= 8 ? 1 : m <= 16 ? 2 : m <= 32 ? 4 : 8; }

}  // namespace

cudaError_t launch_i8few(const I8Args &a, cudaStream_t s) {
  const int g = groups(a.m);
  return g == 1   ? launch<1>(a, s)
         : g == 2 ? launch<2>(a, s)
         : g == 4 ? launch<4>(a, s)
                  : launch<8>(a, s);
}

// ------------------------------------------------------------- cluster sizes
namespace {

// Clusters of c CTAs of a kernel that run at once on the device (asked once for
// each kernel and device; a handful of kernels).
int resident_clusters(const void *kernel, int threads, size_t smem, int c) {
  static std::mutex mu;
  static struct {
    const void *kernel;
    int device;
    int n[9];
  } known[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  std::lock_guard<std::mutex> g(mu);
  int i = 0;
  while (i < 63 && known[i].kernel && !(known[i].kernel == kernel && known[i].device == dev)) i++;
  if (known[i].kernel != kernel || known[i].device != dev) known[i] = {kernel, dev, {}};
  int &n = known[i].n[c];
  if (!n) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim = {(unsigned)c, 1, 1};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(os2_sm_count() / c * c));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int v = 0;
    if (cudaOccupancyMaxActiveClusters(&v, kernel, &cfg) != cudaSuccess) v = 0;
    n = std::max(1, std::min(v, os2_sm_count() / c));
  }
  return n;
}

}  // namespace

void os2i8::few_clusters(const void *kernel, int threads, size_t smem, int tiles, int stages,
                         int *cluster, int *clusters) {
  double least = 1e30;
  for (const int c : {1, 2, 4, 8}) {
    if (c > stages) break;
    const int most = std::min(resident_clusters(kernel, threads, smem, c), tiles);
    const int per = (stages + c - 1) / c, rest = tiles % most;
    auto wave = [&](int n) {
      return per * std::max(0.19, 0.0026 * n * c) + (c > 1 ? 1.3 : 0.3);
    };
    const double t = (tiles / most) * wave(most) + (rest ? wave(rest) : 0.);
    if (t < least) {
      least = t;
      *cluster = c;
      *clusters = most;
    }
  }
}
