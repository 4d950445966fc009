// The 8-bit product of k_i8.cu on the tensor cores, for more than a few tokens.
//
// sm_103a has no tcgen05 MMA for integers, and its mma.sync s8 path runs at a
// fifteenth of the FP16 rate, so the integers are multiplied as FP16, which holds
// them exactly: 1024 products of at most 2^14 sum to at most 2^24, where FP32 is
// exact, so the accumulator is emptied into an int32 sum in registers every
// 1024 terms, while the next 1024 go to a second accumulator.
//
// The weights stay 8-bit up to the SM: they are the A operand (output channels
// on M), which tcgen05.mma takes from tensor memory.  Eight warps widen a stage
// of them in registers (1024 + (b + 128) is the FP16 of bit pattern 0x64, b ^
// 0x80; one packed add of -1152 leaves b) and write it there.  So shared memory
// carries a weight once as a byte in and out, where FP16 weights through shared
// memory would add two bytes in and two out for the MMA.  The tokens, quantised
// or widened before, come as FP16 (B operand, NT tokens a tile).
//
// A CTA pair computes 256 channels x NT tokens, a stage holds 128 terms.  Whole
// tiles go round the pairs; the last one or two per pair are cut along k as well,
// so that all pairs end together and few tiles still use all SMs.  A pair that
// has part of a tile writes its int32 sums to its own slot, and the CTA that
// ends a tile last adds the slots up: integers, so in any order the same result.
//
// Warps (19): 0 weights by TMA, 1 MMA, 2-9 epilogue, 10-17 widening, 18 tokens by
// TMA.  Every wait is bounded, as in mm2.cuh.
#include "i8.cuh"
#include "mm2.cuh"

using namespace os2mm;

namespace {

constexpr int kRawStages = 6;                    // 128 rows x 128 bytes of weights
constexpr uint32_t kRawBytes = kHalf * kStageK;
constexpr int kTc = 4;                           // stages of widened weights and tokens
constexpr int kTcThreads = 19 * 32;
constexpr int kChunk = 8;                        // stages between emptyings: 1024 terms
constexpr int kConvWarps = 8;

template <int NT>
constexpr uint32_t tok_block() { return NT / 2 * kBK * 2; }   // one k-block of this CTA's tokens
template <int NT>
constexpr size_t smem_tc() {
  return 1024 + (size_t)kRawStages * kRawBytes + (size_t)kTc * 2 * tok_block<NT>() + 256;
}

struct I8Job {
  int m, n;            // tokens, channels
  int tiles_c, tiles_t, stages;
  int waves;           // whole tiles of each pair
  int rest;            // tiles cut along k
  int pairs;
  int out_dtype;
  const float *sa, *sb, *bias;
  void *y;
  long ldy;
  int *slots;          // [pairs][2][2 CTAs][NT][128] partial sums
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

// First unit (stage of a cut tile) of pair p.
__device__ __forceinline__ int unit_begin(const I8Job &j, int p) {
  return (int)((long long)p * j.rest * j.stages / j.pairs);
}

// The segments of a pair, in order: f(tile, first stage, end stage, index of the
// cut tile or -1 for a whole one).  Every role walks the same.
template <class F>
__device__ __forceinline__ void for_segments(const I8Job &j, int pair, F &&f) {
  for (int w = 0; w < j.waves; w++)
    if (!f(w * j.pairs + pair, 0, j.stages, -1)) return;
  const int u1 = unit_begin(j, pair + 1);
  for (int u = unit_begin(j, pair); u < u1;) {
    const int r = u / j.stages, s0 = u - r * j.stages, s1 = min(j.stages, s0 + u1 - u);
    const bool whole = s0 == 0 && s1 == j.stages;
    if (!f(j.waves * j.pairs + r, s0, s1, whole ? -1 : r)) return;
    u += s1 - s0;
  }
}

// The part of pair p in cut tile r is its first segment there (slot 0) unless
// its range began in an earlier tile (slot 1).
__device__ __forceinline__ int slot_of(const I8Job &j, int p, int r) {
  return unit_begin(j, p) >= r * j.stages ? 0 : 1;
}

template <int NT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kTcThreads, 1)
    k_i8tc(const __grid_constant__ CUtensorMap mapW, const __grid_constant__ CUtensorMap mapT,
           const I8Job j, int *status) {
  constexpr uint32_t IDESC = idesc_f16_f32(2 * kHalf, NT);
  constexpr uint32_t TOK = 2 * tok_block<NT>();
  constexpr uint32_t A_COL = 2 * NT;              // widened weights after the accumulators
  constexpr int COLS = NT / 2;                    // columns of an epilogue thread

  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~uintptr_t(1023));
  uint8_t *sRaw = smem, *sTok = smem + kRawStages * kRawBytes;
  uint64_t *rfull = reinterpret_cast<uint64_t *>(sTok + kTc * TOK);
  uint64_t *rempty = rfull + kRawStages;
  uint64_t *full = rempty + kRawStages, *tfull = full + kTc, *empty = tfull + kTc;
  uint64_t *acc_full = empty + kTc, *acc_empty = acc_full + 2, *mma_done = acc_empty + 2;
  uint32_t *s_tmem = reinterpret_cast<uint32_t *>(mma_done + 1);
  volatile int *s_abort = reinterpret_cast<volatile int *>(s_tmem + 1);
  volatile unsigned *s_last = reinterpret_cast<volatile unsigned *>(s_tmem + 2);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = (int)(blockIdx.x >> 1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kRawStages; s++) {
      mbar_init(&rfull[s], 1);
      mbar_init(&rempty[s], kConvWarps);
    }
    for (int s = 0; s < kTc; s++) {
      mbar_init(&full[s], 2 * kConvWarps);  // both CTAs' widening warps
      mbar_init(&tfull[s], 1);              // both CTAs' tokens
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; b++) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * kEpiThreads);
    }
    mbar_init(mma_done, 1);
    *s_abort = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&mapW);
    tma_prefetch_desc(&mapT);
  }
  if (warp == 1) {
    tmem_alloc2(s_tmem, 512);
    tmem_relinquish2();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the peer's barriers are initialised before any remote arrive / copy
  tc_fence_after();
  const uint32_t tmem_base = *s_tmem;

  auto gave_up = [&]() {
    *s_abort = 1;
    set_status(status, OS2_ERR_TIMEOUT);
    return false;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ weights
    if (lane == 0) {
      int rs = 0;
      uint32_t ph = 0, used = 0, last_par = 0;
      for_segments(j, pair, [&](int t, int s0, int s1, int) -> bool {
        int tc, tt;
        tile_coords(t, j.tiles_c, j.tiles_t, tc, tt);
        for (int ks = s0; ks < s1; ks++) {
          if (!mbar_wait_bounded(&rempty[rs], ph ^ 1, s_abort, kWaitLimit)) return gave_up();
          mbar_arrive_expect_tx(&rfull[rs], kRawBytes);
          tma_load_3d(sRaw + rs * kRawBytes, &mapW, &rfull[rs], ks * kStageK,
                      tc * 2 * kHalf + (int)rank * kHalf, 0);
          used |= 1u << rs;
          last_par = (last_par & ~(1u << rs)) | (ph << rs);
          if (++rs == kRawStages) {
            rs = 0;
            ph ^= 1;
          }
        }
        return true;
      });
      for (int s = 0; s < kRawStages; s++)
        if (used >> s & 1) {
          volatile int no_abort = 0;
          mbar_wait_bounded(&rfull[s], (last_par >> s) & 1, &no_abort, kWaitLimit);
        }
    }
  } else if (warp == 18) {
    // ------------------------------------------------------------ tokens
    if (lane == 0) {
      int st = 0;
      uint32_t ph = 0, used = 0, last_par = 0;
      for_segments(j, pair, [&](int t, int s0, int s1, int) -> bool {
        int tc, tt;
        tile_coords(t, j.tiles_c, j.tiles_t, tc, tt);
        for (int ks = s0; ks < s1; ks++) {
          if (!mbar_wait_cluster_bounded(&empty[st], ph ^ 1, s_abort, kWaitLimit)) return gave_up();
          const uint32_t fbar = mapa_shared(smem_u32(&tfull[st]), 0);
          if (leader) mbar_arrive_expect_tx(&tfull[st], 2 * TOK);
#pragma unroll
          for (int h = 0; h < 2; h++)
            tma_load_3d_pair(sTok + st * TOK + h * tok_block<NT>(), &mapT, fbar,
                             ks * kStageK + h * kBK, tt * NT + (int)rank * (NT / 2), 0);
          used |= 1u << st;
          last_par = (last_par & ~(1u << st)) | (ph << st);
          if (++st == kTc) {
            st = 0;
            ph ^= 1;
          }
        }
        return true;
      });
      // the pair's copies complete on the leader's barriers: it waits for the last of each stage
      if (leader)
        for (int s = 0; s < kTc; s++)
          if (used >> s & 1) {
            volatile int no_abort = 0;
            mbar_wait_cluster_bounded(&tfull[s], (last_par >> s) & 1, &no_abort, kWaitLimit);
          }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (leader && lane == 0) {
      int st = 0, unit = 0;
      uint32_t ph = 0, aph[2] = {0, 0};
      for_segments(j, pair, [&](int, int s0, int s1, int) -> bool {
        for (int c0 = s0; c0 < s1; c0 += kChunk, unit++) {
          const int buf = unit & 1, c1 = min(s1, c0 + kChunk);
          if (!mbar_wait_cluster_bounded(&acc_empty[buf], aph[buf] ^ 1, s_abort, kWaitLimit))
            return gave_up();
          aph[buf] ^= 1;
          tc_fence_after();
          const uint32_t d = tmem_base + (uint32_t)(buf * NT);
          for (int ks = c0; ks < c1; ks++) {
            if (!mbar_wait_cluster_bounded(&tfull[st], ph, s_abort, kWaitLimit) ||
                !mbar_wait_cluster_bounded(&full[st], ph, s_abort, kWaitLimit))
              return gave_up();
            tc_fence_after();
            const uint32_t a = tmem_base + A_COL + (uint32_t)(st * 64);
#pragma unroll
            for (int h = 0; h < 2; h++) {
              const uint64_t bd = sdesc_k128(smem_u32(sTok + st * TOK + h * tok_block<NT>()));
#pragma unroll
              for (int kk = 0; kk < kBK / 16; kk++)
                umma2_f16_ta(d, a + h * 32 + kk * 8, bd + 2 * kk, IDESC,
                             (ks > c0 || h > 0 || kk > 0) ? 1u : 0u);
            }
            umma2_commit_mc(&empty[st], 0x3);
            if (++st == kTc) {
              st = 0;
              ph ^= 1;
            }
          }
          umma2_commit_mc(&acc_full[buf], 0x3);
        }
        return true;
      });
      umma2_commit_mc(mma_done, 0x1);
      volatile int no_abort = 0;
      mbar_wait_bounded(mma_done, 0, &no_abort, kWaitLimit);
    }
  } else if (warp >= 10) {
    // ------------------------------------------------------------ widening
    // a thread takes 64 terms of its lane's channel: four 16-byte pieces of a
    // 128-byte-swizzled row (no bank conflicts), 32 columns of tensor memory
    const int quarter = warp & 3, khalf = (warp - 10) >> 2;
    const int row = quarter * 32 + lane;
    uint32_t full_leader[kTc];
#pragma unroll
    for (int s = 0; s < kTc; s++) full_leader[s] = mapa_shared(smem_u32(&full[s]), 0);
    const uint32_t dst0 = tmem_base + ((uint32_t)(quarter * 32) << 16) + A_COL + khalf * 32;
    int rs = 0, st = 0;
    uint32_t rph = 0, ph = 0;
    for_segments(j, pair, [&](int, int s0, int s1, int) -> bool {
      for (int ks = s0; ks < s1; ks++) {
        bool ok = mbar_wait_bounded(&rfull[rs], rph, s_abort, kWaitLimit);
        uint32_t v[32];
        if (__all_sync(0xffffffffu, ok)) {
          const uint32_t src = smem_u32(sRaw + rs * kRawBytes) + row * 128;
#pragma unroll
          for (int q = 0; q < 4; q++) {
            uint32_t w0, w1, w2, w3;
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(w0), "=r"(w1), "=r"(w2), "=r"(w3)
                         : "r"(src + (((khalf * 4 + q) ^ (row & 7)) << 4)));
            widen(w0, v[8 * q], v[8 * q + 1]);
            widen(w1, v[8 * q + 2], v[8 * q + 3]);
            widen(w2, v[8 * q + 4], v[8 * q + 5]);
            widen(w3, v[8 * q + 6], v[8 * q + 7]);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&rempty[rs]);
          ok = mbar_wait_cluster_bounded(&empty[st], ph ^ 1, s_abort, kWaitLimit);
        }
        if (!__all_sync(0xffffffffu, ok)) return gave_up();
        tc_fence_after();
        tmem_st32(dst0 + (uint32_t)(st * 64), v);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(full_leader[st]);
        if (++rs == kRawStages) {
          rs = 0;
          rph ^= 1;
        }
        if (++st == kTc) {
          st = 0;
          ph ^= 1;
        }
      }
      return true;
    });
  } else {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const uint32_t lane_base = tmem_base + ((uint32_t)(quarter * 32) << 16) + half * COLS;
    const uint32_t empty_leader[2] = {mapa_shared(smem_u32(&acc_empty[0]), 0),
                                      mapa_shared(smem_u32(&acc_empty[1]), 0)};
    const int r_cta = quarter * 32 + lane;
    uint32_t aph[2] = {0, 0};
    int unit = 0;
    for_segments(j, pair, [&](int t, int s0, int s1, int cut) -> bool {
      int sum[COLS];
#pragma unroll
      for (int i = 0; i < COLS; i++) sum[i] = 0;
      for (int c0 = s0; c0 < s1; c0 += kChunk, unit++) {
        const int buf = unit & 1;
        const bool ok = __all_sync(
            0xffffffffu, mbar_wait_cluster_bounded(&acc_full[buf], aph[buf], s_abort, kWaitLimit));
        if (!ok) return gave_up();
        aph[buf] ^= 1;
        tc_fence_after();
#pragma unroll
        for (int g = 0; g < COLS / 16; g++) {
          uint32_t r[16];
          tmem_ld16(lane_base + (uint32_t)(buf * NT) + g * 16, r);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; i++) sum[g * 16 + i] += __float2int_rn(__uint_as_float(r[i]));
        }
        tc_fence_before();
        mbar_arrive_cluster(empty_leader[buf]);
      }
      if (cut >= 0) {
        // this CTA's part to its slot; the last CTA of a tile (its rank's rows)
        // adds up the others'
        int *mine = j.slots + (((size_t)pair * 2 + slot_of(j, pair, cut)) * 2 + rank) * NT * 128;
#pragma unroll
        for (int i = 0; i < COLS; i++) __stcg(mine + (half * COLS + i) * 128 + r_cta, sum[i]);
        __threadfence();
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (threadIdx.x == 64) {
          const unsigned before = atomicAdd(&j.done[cut * 2 + rank], (unsigned)(s1 - s0));
          *s_last = before + (unsigned)(s1 - s0) == (unsigned)j.stages;
          __threadfence();
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
        const bool last = *s_last != 0;
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (!last) return true;
        const int u0 = cut * j.stages, u1 = u0 + j.stages;
        // pairs whose range meets [u0, u1): a little either side of the proportion
        const long long units = (long long)j.rest * j.stages;
        int p = max(0, (int)((long long)u0 * j.pairs / units) - 1);
        for (; p < j.pairs && unit_begin(j, p) < u1; p++) {
          if (p == pair || unit_begin(j, p + 1) <= u0 || unit_begin(j, p) == unit_begin(j, p + 1))
            continue;
          const int *o = j.slots + (((size_t)p * 2 + slot_of(j, p, cut)) * 2 + rank) * NT * 128;
#pragma unroll
          for (int i = 0; i < COLS; i++) sum[i] += __ldcg(o + (half * COLS + i) * 128 + r_cta);
        }
      }
      int tc, tt;
      tile_coords(t, j.tiles_c, j.tiles_t, tc, tt);
      const int ch = tc * 2 * kHalf + (int)rank * kHalf + r_cta;
      const int tok0 = tt * NT + half * COLS;
      if (ch < j.n) {
        const float sb = j.sb[ch], b = j.bias ? j.bias[ch] : 0.f;
        const size_t at = (size_t)tok0 * j.ldy + ch;
#pragma unroll
        for (int i = 0; i < COLS; i++)
          if (tok0 + i < j.m) {
            const float y = (float)sum[i] * j.sa[tok0 + i] * sb + b;
            const size_t o = at + (size_t)i * j.ldy;
            if (j.out_dtype == OS2_F32) static_cast<float *>(j.y)[o] = y;
            else if (j.out_dtype == OS2_BF16) static_cast<__nv_bfloat16 *>(j.y)[o] = __float2bfloat16_rn(y);
            else static_cast<__half *>(j.y)[o] = __float2half_rn(y);
          }
      }
      __syncwarp();
      return true;
    });
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no CTA leaves while its peer may still touch its shared memory or TMEM
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc2(tmem_base, 512);
  }
}

int pairs_of(long units) {
  return (int)std::max<long>(1, std::min<long>(std::max(os2_sm_count() / 2, 1), units));
}

template <int NT>
I8Job plan(int m, int n, int k) {
  I8Job j = {};
  j.m = m;
  j.n = n;
  j.tiles_c = (n + 2 * kHalf - 1) / (2 * kHalf);
  j.tiles_t = (m + NT - 1) / NT;
  j.stages = std::max((k + kStageK - 1) / kStageK, 1);
  const long tiles = (long)j.tiles_c * j.tiles_t;
  j.pairs = pairs_of(tiles * j.stages);
  // a remainder of tiles takes the last whole wave with it, so that a cut tile
  // has few parts
  j.waves = (int)(tiles / j.pairs) - (tiles % j.pairs && tiles >= j.pairs ? 1 : 0);
  j.rest = (int)(tiles - (long)j.waves * j.pairs);
  return j;
}

bool map_w(CUtensorMap *map, const void *base, long k, long rows, long pitch) {
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

template <int NT>
cudaError_t launch(const I8TcArgs &a, cudaStream_t s) {
  static std::once_flag once;
  static cudaError_t attr_err = cudaSuccess;
  std::call_once(once, [] {
    attr_err = cudaFuncSetAttribute(k_i8tc<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)smem_tc<NT>());
  });
  if (attr_err != cudaSuccess) return attr_err;
  I8Job j = plan<NT>(a.m, a.n, a.k);
  CUtensorMap mw, mt;
  if (!map_w(&mw, a.W, a.k, a.n, a.ldw) ||
      !make_map(&mt, a.tokens, false, a.k, a.m, a.pitch, false, NT / 2))
    return cudaErrorInvalidValue;
  j.out_dtype = a.out_dtype;
  j.sa = a.sa;
  j.sb = a.sb;
  j.bias = a.bias;
  j.y = a.y;
  j.ldy = a.ldy;
  j.slots = a.slots;
  j.done = a.done;
  k_i8tc<NT><<<2 * j.pairs, kTcThreads, smem_tc<NT>(), s>>>(mw, mt, j, a.status);
  return cudaGetLastError();
}

// Tokens a tile: as many as there are, up to 128.
int tile_tokens(int m) { return m <= 32 ? 32 : m <= 64 ? 64 : 128; }

}  // namespace

I8TcSizes i8tc_sizes(int m, int n, int k) {
  const int nt = tile_tokens(m);
  const I8Job j = nt == 32 ? plan<32>(m, n, k) : nt == 64 ? plan<64>(m, n, k) : plan<128>(m, n, k);
  I8TcSizes z;
  z.counters = 2 * j.rest;
  z.slot_ints = j.rest ? (size_t)j.pairs * 4 * nt * 128 : 0;
  return z;
}

cudaError_t launch_i8tc(const I8TcArgs &a, cudaStream_t s) {
  const int nt = tile_tokens(a.m);
  return nt == 32 ? launch<32>(a, s) : nt == 64 ? launch<64>(a, s) : launch<128>(a, s);
}
