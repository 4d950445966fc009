// The linear layer for few tokens, y = r + act(x W^T + b), and its dx = D W: W's bytes bound them.
//
// W's rows (dx: its columns) are the M of the MMAs and the tokens the N, in multiples of 16, so
// that a tile is as large as the tokens are: a CTA takes 128 outputs and up to 128 tokens
// (tcgen05.mma cta_group::1, kind::f16, the accumulator in tensor memory), and a cluster shares
// out the terms of a tile.  A ring of TMA copies keeps some 200 KB an SM in flight, of two CTAs.
// The parts meet in shared memory: each CTA of the cluster adds up its share of the tokens, in the
// CTAs' order, and finishes them (bias, activation, residual).  Every wait is bounded; on expiry the
// CTA records OS2_ERR_TIMEOUT and goes on to the end.
//
// 4096 x 4096 BF16: one token 8.6 us (a kernel that only reads W takes 8.7), 32 tokens 9.1, 128
// 14.9; 256 take 17.2 as tiles of k_linear.cu.  dx of one token 10.8 with D, as tiles 20.6.  One
// token, 16384 x 4096: 26 us (5.1 TB/s).
#include "i8.cuh"
#include "linear.cuh"

using namespace os2mm;
using namespace os2lin;

namespace {

constexpr int kThreadsF = 256;
constexpr int kM = 128;                             // outputs of a CTA
constexpr uint32_t kWStage = kM * kBK * 2;          // 64 terms
constexpr int kMaxStages = 12;
constexpr int kTokens = 128;                        // of a tile, at most

struct Job {
  LinearArgs a;
  int nt;           // tokens of a tile, a multiple of 16
  int tiles_c, stages, ring;  // tiles of outputs, stages of 64 terms, stages of the ring
  int cluster;
  uint32_t cols;    // tensor memory columns
  bool rwhole, ywhole, pwhole;  // four entries on a boundary of their own
};

// W_MN: the terms run along W's rows (dX = D W), else along its columns.
template <bool BF16, bool W_MN>
__global__ void __launch_bounds__(kThreadsF)
    k_linear_few(const __grid_constant__ CUtensorMap mapW, const __grid_constant__ CUtensorMap mapX, const Job j) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], done;
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  const LinearArgs &a = j.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank(), tile = (int)blockIdx.x / j.cluster;
  const int ch0 = tile % j.tiles_c * kM, t0 = tile / j.tiles_c * j.nt;
  const int s0 = (int)((long)rank * j.stages / j.cluster), s1 = (int)((long)(rank + 1) * j.stages / j.cluster);
  const uint32_t stage_bytes = kWStage + (uint32_t)j.nt * kBK * 2;

  if (threadIdx.x == 0) {
    for (int s = 0; s < j.ring; s++) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&done, 1);
    s_abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&mapW);
    tma_prefetch_desc(&mapX);
  }
  if (warp == 1) {
    tmem_alloc(&s_tmem, j.cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  // (after the allocation: no kernel behind this one takes tensor memory before all its CTAs have it)
  start_call();

  auto gave_up = [&]() {
    s_abort = 1;
    set_status(a.status, OS2_ERR_TIMEOUT);
    return false;
  };
  if (warp == 0 && lane == 0) {
    // ------------------------------------------------------------ TMA
    int st = 0;
    uint32_t ph = 0, used = 0, last = 0;
    for (int ks = s0; ks < s1; ks++) {
      if (!mbar_wait_bounded(&empty[st], ph ^ 1, &s_abort, kWaitLimit)) {
        gave_up();
        break;
      }
      mbar_arrive_expect_tx(&full[st], stage_bytes);
      uint8_t *to = smem + st * stage_bytes;
      if (W_MN) {  // two boxes of 64 outputs x 64 terms
        tma_load_3d(to, &mapW, &full[st], ch0, ks * kBK, 0);
        tma_load_3d(to + kWStage / 2, &mapW, &full[st], ch0 + 64, ks * kBK, 0);
      } else {
        tma_load_3d(to, &mapW, &full[st], ks * kBK, ch0, 0);
      }
      tma_load_3d(to + kWStage, &mapX, &full[st], ks * kBK, t0, 0);
      used |= 1u << st;
      last = (last & ~(1u << st)) | (ph << st);
      if (++st == j.ring) st = 0, ph ^= 1;
    }
    // (the copies have landed before the ring is used for other things or the CTA ends)
    for (int s = 0; s < j.ring; s++)
      if (used >> s & 1) {
        volatile int no_abort = 0;
        mbar_wait_bounded(&full[s], (last >> s) & 1, &no_abort, kWaitLimit);
      }
  } else if (warp == 1 && lane == 0) {
    // ------------------------------------------------------------ MMA
    const uint32_t idesc = idesc_f16_f32(kM, j.nt) | (BF16 ? (1u << 7) | (1u << 10) : 0u) | (W_MN ? 1u << 15 : 0u);
    int st = 0;
    uint32_t ph = 0;
    for (int ks = s0; ks < s1; ks++) {
      if (!mbar_wait_bounded(&full[st], ph, &s_abort, kWaitLimit)) {
        gave_up();
        break;
      }
      tc_fence_after();
      const uint32_t at = smem_u32(smem + st * stage_bytes);
      const uint64_t ad = W_MN ? sdesc_mn128(at, kWStage / 2, 1024) : sdesc_k128(at), bd = sdesc_k128(at + kWStage);
      constexpr uint64_t step = (W_MN ? 16 * 128 : 32) >> 4;
#pragma unroll
      for (int kk = 0; kk < kBK / 16; kk++) umma_f16(tmem, ad + step * kk, bd + 2 * kk, idesc, ks > s0 || kk > 0);
      umma_commit(&empty[st]);
      if (++st == j.ring) st = 0, ph ^= 1;
    }
    umma_commit(&done);
  }
  __syncwarp();
  // what the first of this warp's tokens takes besides, on its way before the sums are there
  const int ch = ch0 + lane * 4, left = a.n - ch;
  float bias[4] = {};
  if (a.bias)
#pragma unroll
    for (int i = 0; i < 4; i++)
      if (i < left) bias[i] = bias_at<BF16>(a.bias, a.b32, ch + i);
  const int t_first = t0 + rank * (j.nt / j.cluster) + warp;
  uint2 r_first = make_uint2(0, 0);
  if (a.R && t_first < a.m && left > 0) r_first = load4(a.R + (size_t)t_first * a.ldr + ch, left, j.rwhole);
  // ------------------------------------------------------------ the sums
  // (the MMAs that were issued, all of them, have ended; bounded like every wait)
  {
    volatile int no_abort = 0;
    if (!mbar_wait_bounded(&done, 0, &no_abort, 2 * kWaitLimit)) gave_up();
  }
  __syncthreads();
  tc_fence_after();
  // Through shared memory, [tokens][128 outputs], so that a lane finishes four neighbouring
  // outputs of a token; two warps for each lane quarter of the tensor memory.
  const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
  float *const part = reinterpret_cast<float *>(smem);
  {
    for (int g = (warp >> 2) * 16; g < j.nt; g += 32) {
      uint32_t r[16];
      tmem_ld16(lanes + g, r);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 16; i++) part[(g + i) * kM + (warp & 3) * 32 + lane] = __uint_as_float(r[i]);
    }
    cluster_sync();
    // this CTA's tokens: a warp one at a time (nt is a multiple of 16, the CTAs are at most 8)
    const int per = j.nt / j.cluster;
#pragma unroll 2
    for (int i = warp; i < per; i += kThreadsF / 32) {
      const int mine = rank * per + i, t = t0 + mine;
      const bool in = t < a.m && left > 0;
      const uint32_t from = smem_u32(part + mine * kM + lane * 4);
      uint4 x[8];
#pragma unroll
      for (int c = 0; c < 8; c++)
        if (c < j.cluster)
          asm volatile("ld.shared::cluster.v4.u32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(x[c].x), "=r"(x[c].y), "=r"(x[c].z), "=r"(x[c].w)
                       : "r"(mapa_shared(from, c)));
        else
          x[c] = make_uint4(0, 0, 0, 0);
      const uint2 r = i == warp ? r_first : a.R && in ? load4(a.R + (size_t)t * a.ldr + ch, left, j.rwhole) : make_uint2(0, 0);
      float z[4] = {};
#pragma unroll
      for (int c = 0; c < 8; c++) {
        z[0] += __uint_as_float(x[c].x), z[1] += __uint_as_float(x[c].y);
        z[2] += __uint_as_float(x[c].z), z[3] += __uint_as_float(x[c].w);
      }
#pragma unroll
      for (int q = 0; q < 4; q++) z[q] = W_MN && !BF16 ? z[q] * a.by : z[q] + bias[q];
      if (a.pre && in)
        store4(a.pre + (size_t)t * a.ldp + ch, make_uint2(pack2<BF16>(z[0], z[1]), pack2<BF16>(z[2], z[3])), left, j.pwhole);
      os2act::values(z, a.act);
      if (a.R) {
        const uint32_t w[2] = {r.x, r.y};
#pragma unroll
        for (int q = 0; q < 4; q++) z[q] += widen16<BF16>((uint16_t)(w[q >> 1] >> (16 * (q & 1))));
      }
      if (in) store4(a.Y + (size_t)t * a.ldy + ch, make_uint2(pack2<BF16>(z[0], z[1]), pack2<BF16>(z[2], z[3])), left, j.ywhole);
    }
    cluster_sync();  // (read before its CTA ends)
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, j.cols);
  }
}

template <bool BF16, bool W_MN>
cudaError_t launch(const LinearArgs &a, cudaStream_t s) {
  Job j;
  j.a = a;
  const LinearPlan plan = linear_few_plan(a.m, a.n, a.k, a.act != OS2_ACT_NONE || a.pre);
  j.nt = plan.nt;
  j.tiles_c = (a.n + kM - 1) / kM;
  j.stages = (a.k + kBK - 1) / kBK;
  const size_t stage = kWStage + (size_t)j.nt * kBK * 2, room = 110 * 1024;
  j.ring = (int)std::min<size_t>(kMaxStages, room / stage);
  auto whole = [](const void *p, long ld) { return reinterpret_cast<uintptr_t>(p) % 8 == 0 && ld % 4 == 0; };
  j.rwhole = whole(a.R, a.ldr), j.ywhole = whole(a.Y, a.ldy), j.pwhole = whole(a.pre, a.ldp);
  j.cols = 32;
  while (j.cols < (uint32_t)j.nt) j.cols *= 2;
  const long tiles = (long)j.tiles_c * ((a.m + j.nt - 1) / j.nt);
  j.cluster = plan.cluster;
  const size_t smem = 1024 + j.ring * stage;
  static_assert(110 * 1024 / (kWStage + 16 * kBK * 2) * (kWStage + 16 * kBK * 2) >= 16 * kM * 4, "a part fits the ring");
  static PerDevice ready;
  const cudaError_t e = os2_set_smem(ready, k_linear_few<BF16, W_MN>, 1024 + 110 * 1024);
  if (e != cudaSuccess) return e;
  CUtensorMap mw, mx;
  if (!(W_MN ? make_map(&mw, a.W, BF16, a.n, a.k, a.ldw, true) : make_map(&mw, a.W, BF16, a.k, a.n, a.ldw, false)) || !make_map(&mx, a.X, BF16, a.k, a.m, a.ldx, false, j.nt))
    return cudaErrorInvalidValue;
  return os2i8::launch_cluster(k_linear_few<BF16, W_MN>, j.cluster, (int)(tiles * j.cluster), kThreadsF, smem, true, s, mw, mx, j);
}

}  // namespace

// By an estimate in microseconds, fitted at 512 x 512 to 5000 x 2048, 88 x 7168 and 8192 x 256 and 48 to
// 8000 tokens: a start of 2.3, joining parts 1.2; a wave of CTAs its stages, a CTA's bytes at 75 a
// ns (64 where a stage is large) or those of all that run at once at 13000, and for each token
// 0.01 and, shared out over the cluster, 0.055 (0.075 with an activation or pre); all of W at 6300.
// With it and tiles_us, 243 cases there take 1 % longer than by the better way each.
LinearPlan linear_few_plan(int m, int n, int k, bool more) {
  const int sms = os2_sm_count(), stages = (k + kBK - 1) / kBK, tiles_c = (n + kM - 1) / kM;
  LinearPlan best = {16, 1, 1e30};
  const int whole = (int)os2_round_up((size_t)m, 16);
  for (const int most : {64, kTokens}) {
    const int tiles_t = (m + most - 1) / most;
    const int nt = std::min(whole, (int)os2_round_up((size_t)((m + tiles_t - 1) / tiles_t), 16));
    const long tiles = (long)tiles_c * ((m + nt - 1) / nt);
    for (const int c : {1, 2, 4, 8}) {
      if (c > stages) break;
      const long ctas = tiles * c, waves = (ctas + 2L * sms - 1) / (2 * sms);
      if (c > 1 && 10 * ctas > 17L * sms) break;  // clusters in a second wave wait for one another's SMs
      // (and those of eight leave some unused: 48 tokens of 4096 x 1024 take 6.7 us by 256 CTAs, 5.5 by 128)
      const double late = c == 8 && 10 * ctas > 15L * sms ? nt > 64 ? 2.6 : 1.3 : 0.;
      const double bytes = kWStage + nt * kBK * 2., at_once = (double)std::min(ctas, 2L * sms);
      const double stage = std::max(bytes / (nt > 64 ? 64e3 : 75e3), bytes * at_once / 13e6);
      const double wave = ((stages + c - 1) / c) * stage + (more ? 0.075 : 0.055) * nt / c + 0.01 * nt;
      const double t = 2.3 + late + (c > 1 ? 1.2 : 0.) + std::max(waves * wave, 2. * n * k / 6.3e6 + 0.01 * nt);
      if (t < best.us) best = {nt, c, t};
    }
    if (whole <= most) break;
  }
  return best;
}

cudaError_t launch_linear_few(const LinearArgs &a, bool w_mn, cudaStream_t s) {
  if (w_mn) return a.bf16 ? launch<true, true>(a, s) : launch<false, true>(a, s);
  return a.bf16 ? launch<true, false>(a, s) : launch<false, false>(a, s);
}
