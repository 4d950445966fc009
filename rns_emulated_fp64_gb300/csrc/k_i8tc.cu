// The 8-bit product of k_i8.cu on the tensor cores, for more than a few tokens.
//
// sm_103a has no tcgen05 MMA for integers, and its mma.sync s8 path runs at a
// fifteenth of the FP16 rate, so the integers are multiplied as FP16, which holds
// them exactly: 1024 products of at most 2^14 sum to at most 2^24, where FP32 is
// exact, so the accumulator is emptied into an int32 sum in registers every
// 1024 terms, while the next 1024 go to a second accumulator.
//
// The weights stay 8-bit up to the SM: they are the A operand (output channels
// on M), and eight warps widen a stage of them from the bytes that TMA brings to
// the swizzled FP16 tile that the MMAs read (1024 + (b + 128) is the FP16 of bit
// pattern 0x64, b ^ 0x80; one packed add of -1152 leaves b).  The tokens, quantised
// or widened before, come as FP16 (B operand, NT tokens a tile).  Shared memory
// then moves 96 KB + 256 NT bytes a stage of 128 terms (the weights' bytes in and
// out, their FP16 in and out, the tokens in and out), 768 + 2 NT cycles at 128
// bytes a cycle, against 4 NT cycles of MMA: shared memory bounds up to 256 tokens
// a tile (1280 against 1024).  Tried before: the widened weights in tensor memory
// as A, with less traffic; but such an MMA took 125 cycles or more whatever its N.
//
// A CTA pair computes 256 channels x NT tokens.  Whole tiles go round the pairs;
// those left over may be cut along k, where the time saved is more than the 4 to
// 10 us of joining them (plan): a pair then writes its int32 sums to its slot, and
// the CTA that ends a tile last adds the slots up: integers, so in any order the
// same result.  (Dealing all stages out evenly, with up to two cut tiles a pair, took 30.5
// us instead of 25 for 256 x 4096 x 4096, and 47 instead of 33 for 1024 tokens.)
//
// Warps: 0 weights by TMA, 1 MMA, 2 tokens by TMA, 4-11 epilogue (its int32 sums
// take up to 128 registers a thread), 12 and up widening; each role has the registers
// it needs.  Every wait is bounded, as in mm2.cuh.  Between the CTAs of
// a pair go arrivals without a release at cluster scope (ptx.cuh); with it, every
// stage waited for its fence: 1985 us instead of 1075 for 8192 x 4096 x 16384.
// Measured with quantising: 684 us for that (1.6 PFLOP/s, 0.84 of cuBLAS's BF16 burst), 21 us
// for 65 tokens and 4096 x 4096 weights, 22.9 for 205, 5003 x 1777 and rows that are copied first.
#include "i8.cuh"

using namespace os2i8;

namespace {

constexpr uint32_t kRawBytes = kHalf * kStageK;  // a stage of weights: 128 rows x 128 bytes
constexpr int kTc = 3;                           // stages of widened weights and tokens
constexpr int kChunk = 8;                        // stages between emptyings: 1024 terms
constexpr int kConvWarps = 8;                    // that widen one stage

// Warps and registers: 256 tokens take 128 sums a thread and leave registers for
// one widening group; with fewer tokens the MMAs are short and two groups keep up
// better (a stage takes a group about 1300 cycles).
template <int NT>
struct Threads {
  static constexpr int groups = NT == 256 ? 1 : 2;
  static constexpr int conv = groups * kConvWarps * 32;
  static constexpr int all = 128 + 256 + conv;
  static constexpr int launch = 65536 / all / 8 * 8;  // registers a thread
  static constexpr int r_misc = 48, r_epi = NT == 256 ? 160 : 112, r_conv = 56;
  static_assert(128 * r_misc + 256 * r_epi + conv * r_conv <= all * launch, "registers");
};

template <int NT>
constexpr uint32_t tok_block() { return NT / 2 * kBK * 2; }   // one k-block of this CTA's tokens
// What shared memory is left holds weights in flight.
template <int NT>
constexpr int raw_stages() {
  return (int)((227 * 1024 - 1280 - kTc * (kOpBytes + 2 * tok_block<NT>())) / kRawBytes);
}
template <int NT>
constexpr size_t smem_tc() {
  return 1280 + (size_t)raw_stages<NT>() * kRawBytes + (size_t)kTc * (kOpBytes + 2 * tok_block<NT>());
}

template <int NT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Threads<NT>::all, 1)
    k_i8tc(const __grid_constant__ CUtensorMap mapW, const __grid_constant__ CUtensorMap mapT,
           const I8Job j, int *status) {
  using T = Threads<NT>;
  constexpr int RAW = raw_stages<NT>();
  // Two groups take the stages in turn, so that with an odd number of slots a group meets
  // every second phase of a slot's barrier only, and these have the same parity.  No wait
  // passes on an old one all the same: MMAs end in order, and a group that comes to stage j has
  // seen that of stage j - 2 - kTc end, so that the stages up to it were there and read.  The
  // phase between is among them in both rings:
  static_assert(T::groups == 1 || (RAW >= kTc + T::groups && kTc >= T::groups), "rings");
  constexpr uint32_t IDESC = idesc_f16_f32(2 * kHalf, NT);
  constexpr uint32_t TOK = 2 * tok_block<NT>();
  constexpr int COLS = NT / 2;                    // columns of an epilogue thread

  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~uintptr_t(1023));
  uint8_t *sW = smem, *sTok = sW + kTc * kOpBytes, *sRaw = sTok + kTc * TOK;
  uint64_t *rfull = reinterpret_cast<uint64_t *>(sRaw + RAW * kRawBytes);
  uint64_t *rempty = rfull + RAW;
  uint64_t *full = rempty + RAW, *tfull = full + kTc, *empty = tfull + kTc;
  uint64_t *acc_full = empty + kTc, *acc_empty = acc_full + 2, *mma_done = acc_empty + 2;
  uint64_t *join = mma_done + 1;
  uint32_t *s_tmem = reinterpret_cast<uint32_t *>(join + 2);
  volatile int *s_abort = reinterpret_cast<volatile int *>(s_tmem + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = (int)(blockIdx.x >> 1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < RAW; s++) {
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
      mbar_init(&acc_empty[b], 16);  // both CTAs' epilogue warps
    }
    mbar_init(mma_done, 1);
    mbar_init(&join[0], 8);
    mbar_init(&join[1], 1);
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
  next_may_start();
  wait_for_previous();  // the tokens, their scales, the counters, copied weights

  auto gave_up = [&]() {
    *s_abort = 1;
    set_status(status, OS2_ERR_TIMEOUT);
    return false;
  };

  if (warp < 4) {
    regs_fewer<T::r_misc>();
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
            if (++rs == RAW) {
              rs = 0;
              ph ^= 1;
            }
          }
          return true;
        });
        for (int s = 0; s < RAW; s++)
          if (used >> s & 1) {
            volatile int no_abort = 0;
            mbar_wait_bounded(&rfull[s], (last_par >> s) & 1, &no_abort, kWaitLimit);
          }
      }
    } else if (warp == 2) {
      // ------------------------------------------------------------ tokens
      if (lane == 0) {
        int st = 0;
        uint32_t ph = 0, used = 0, last_par = 0;
        for_segments(j, pair, [&](int t, int s0, int s1, int) -> bool {
          int tc, tt;
          tile_coords(t, j.tiles_c, j.tiles_t, tc, tt);
          for (int ks = s0; ks < s1; ks++) {
            if (!mbar_wait_bounded(&empty[st], ph ^ 1, s_abort, kWaitLimit)) return gave_up();
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
              mbar_wait_bounded(&tfull[s], (last_par >> s) & 1, &no_abort, kWaitLimit);
            }
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer
      if (leader && lane == 0) {
        int st = 0, unit = 0;
        uint32_t ph = 0, aph[2] = {0, 0};
        for_segments(j, pair, [&](int, int s0, int s1, int) -> bool {
          for (int ks = s0; ks < s1; ks++) {
            const int buf = unit & 1, rel = (ks - s0) % kChunk;
            if (rel == 0) {
              if (!mbar_wait_bounded(&acc_empty[buf], aph[buf] ^ 1, s_abort, kWaitLimit))
                return gave_up();
              aph[buf] ^= 1;
            }
            if (!mbar_wait_bounded(&tfull[st], ph, s_abort, kWaitLimit) ||
                !mbar_wait_bounded(&full[st], ph, s_abort, kWaitLimit))
              return gave_up();
            tc_fence_after();
            const uint32_t d = tmem_base + (uint32_t)(buf * NT);
#pragma unroll
            for (int h = 0; h < 2; h++) {
              const uint64_t ad = sdesc_k128(smem_u32(sW + st * kOpBytes + h * kBlockBytes));
              const uint64_t bd = sdesc_k128(smem_u32(sTok + st * TOK + h * tok_block<NT>()));
#pragma unroll
              for (int kk = 0; kk < kBK / 16; kk++)
                umma2_f16(d, ad + 2 * kk, bd + 2 * kk, IDESC,
                          (rel > 0 || h > 0 || kk > 0) ? 1u : 0u);
            }
            umma2_commit_mc(&empty[st], 0x3);
            if (rel == kChunk - 1 || ks == s1 - 1) {
              umma2_commit_mc(&acc_full[buf], 0x3);
              unit++;
            }
            if (++st == kTc) {
              st = 0;
              ph ^= 1;
            }
          }
          return true;
        });
        umma2_commit_mc(mma_done, 0x1);
        volatile int no_abort = 0;
        mbar_wait_bounded(mma_done, 0, &no_abort, kWaitLimit);
      }
    }
  } else if (warp >= 12) {
    regs_fewer<T::r_conv>();
    // ------------------------------------------------------------ widening
    // A group of eight warps takes a stage, two groups the stages in turn.  A thread
    // takes 64 terms (one k-block) of its channel: four 16-byte pieces of a
    // 128-byte-swizzled row in, eight out; no bank conflicts either way.
    const int group = (warp - 12) / kConvWarps, half = ((warp - 12) >> 2) & 1;
    const int row = ((warp - 12) & 3) * 32 + lane;
    uint32_t full_leader[kTc];
#pragma unroll
    for (int s = 0; s < kTc; s++) full_leader[s] = mapa_shared(smem_u32(&full[s]), 0);
    int rs = 0, st = 0, turn = 0;
    uint32_t rph = 0, ph = 0;
    for_segments(j, pair, [&](int, int s0, int s1, int) -> bool {
      for (int ks = s0; ks < s1; ks++) {
        if (turn == group) {
          bool ok = mbar_wait_bounded(&rfull[rs], rph, s_abort, kWaitLimit);
          if (!__all_sync(0xffffffffu, ok)) return gave_up();
          uint32_t v[32];
          const uint32_t src = smem_u32(sRaw + rs * kRawBytes) + row * 128;
#pragma unroll
          for (int q = 0; q < 4; q++) {
            uint32_t w0, w1, w2, w3;
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(w0), "=r"(w1), "=r"(w2), "=r"(w3)
                         : "r"(src + (((half * 4 + q) ^ (row & 7)) << 4)));
            widen(w0, v[8 * q], v[8 * q + 1]);
            widen(w1, v[8 * q + 2], v[8 * q + 3]);
            widen(w2, v[8 * q + 4], v[8 * q + 5]);
            widen(w3, v[8 * q + 6], v[8 * q + 7]);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&rempty[rs]);
          ok = mbar_wait_bounded(&empty[st], ph ^ 1, s_abort, kWaitLimit);
          if (!__all_sync(0xffffffffu, ok)) return gave_up();
          const uint32_t dst = smem_u32(sW + st * kOpBytes + half * kBlockBytes) + row * 128;
#pragma unroll
          for (int q = 0; q < 8; q++)
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(dst + ((q ^ (row & 7)) << 4)),
                         "r"(v[4 * q]), "r"(v[4 * q + 1]), "r"(v[4 * q + 2]), "r"(v[4 * q + 3])
                         : "memory");
          fence_async_smem();  // the tensor cores read what the generic proxy wrote
          __syncwarp();
          if (lane == 0) mbar_arrive_remote(full_leader[st]);
        }
        turn = turn + 1 == T::groups ? 0 : turn + 1;
        if (++rs == RAW) {
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
    regs_more<T::r_epi>();
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const uint32_t lane_base = tmem_base + ((uint32_t)(quarter * 32) << 16) + half * COLS;
    const uint32_t empty_leader[2] = {mapa_shared(smem_u32(&acc_empty[0]), 0),
                                      mapa_shared(smem_u32(&acc_empty[1]), 0)};
    const int r_cta = quarter * 32 + lane;
    uint32_t aph[2] = {0, 0};
    int unit = 0;
    I8Join jn{&join[0], &join[1], reinterpret_cast<volatile unsigned *>(s_tmem + 2), 0};
    for_segments(j, pair, [&](int t, int s0, int s1, int cut) -> bool {
      int tc, tt;
      tile_coords(t, j.tiles_c, j.tiles_t, tc, tt);
      const int tok0 = tt * NT + half * COLS;
      // the tokens' scales, a lane each, long before they are used: read one by one
      // at the end they cost a miss every 8 columns (10000 cycles a tile)
      constexpr int SL = (COLS + 31) / 32;
      float sa[SL];
#pragma unroll
      for (int i = 0; i < SL; i++)
        sa[i] = tok0 + i * 32 + lane < j.m ? j.sa[tok0 + i * 32 + lane] : 0.f;
      int sum[COLS];
#pragma unroll
      for (int i = 0; i < COLS; i++) sum[i] = 0;
      for (int c0 = s0; c0 < s1; c0 += kChunk, unit++) {
        const int buf = unit & 1;
        const bool ok = __all_sync(
            0xffffffffu, mbar_wait_bounded(&acc_full[buf], aph[buf], s_abort, kWaitLimit));
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
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(empty_leader[buf]);
      }
      if (cut >= 0) {
        // this CTA's part to its slot; the last CTA of a tile (its rank's rows)
        // adds up the others'
        if (!OS2_DBG_GUARD(cut < j.rest && pair < j.workers, status)) return true;
        int *mine = j.slots + ((size_t)pair * 2 + rank) * NT * 128;
#pragma unroll
        for (int i = 0; i < COLS; i += 4)
          __stcg(reinterpret_cast<int4 *>(mine) + (half * COLS + i) / 4 * 128 + r_cta,
                 make_int4(sum[i], sum[i + 1], sum[i + 2], sum[i + 3]));
        const int last = last_part(jn, &j.done[cut * 2 + rank], s1 - s0, j.stages,
                                   threadIdx.x == 4 * 32, s_abort);
        if (last < 0) return gave_up();
        if (!last) return true;
        for (int p = cut * j.parts; p < (cut + 1) * j.parts; p++) {
          if (p == pair) continue;
          const int *o = j.slots + ((size_t)p * 2 + rank) * NT * 128;
#pragma unroll
          for (int i = 0; i < COLS; i += 4) {
            const int4 v = __ldcg(reinterpret_cast<const int4 *>(o) + (half * COLS + i) / 4 * 128 + r_cta);
            sum[i] += v.x;
            sum[i + 1] += v.y;
            sum[i + 2] += v.z;
            sum[i + 3] += v.w;
            if (i % 16 == 12) asm volatile("" ::: "memory");  // no more in flight than registers
          }
        }
      }
      const int ch = tc * 2 * kHalf + (int)rank * kHalf + r_cta;
      const bool in = ch < j.n && OS2_DBG_GUARD(ch >= 0 && j.ldy >= j.n, status);
      const float sb = in ? j.sb[ch] : 0.f, b = in && j.bias ? j.bias[ch] : 0.f;
      const int left = in ? j.m - tok0 : 0;
      __syncwarp();
      // the type is chosen outside the loop: inside, it cost 14000 cycles a tile
      auto store = [&](auto *y, auto round) {
        auto *o = y + (size_t)tok0 * j.ldy + ch;
#pragma unroll
        for (int i = 0; i < COLS; i++) {
          const float v = (float)sum[i] * __shfl_sync(0xffffffffu, sa[i / 32], i % 32) * sb + b;
          if (i < left) *o = round(v);
          o += j.ldy;
        }
      };
      if (j.out_dtype == OS2_F32)
        store(static_cast<float *>(j.y), [](float v) { return v; });
      else if (j.out_dtype == OS2_BF16)
        store(static_cast<__nv_bfloat16 *>(j.y), [](float v) { return __float2bfloat16_rn(v); });
      else
        store(static_cast<__half *>(j.y), [](float v) { return __float2half_rn(v); });
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

// The tiles of nt tokens, how the ones left over are cut, and the time in cycles: a
// stage takes about 1350 (64 and 128 tokens: the widening bounds it) or 1450 (256);
// joining takes 5000, writing a part 700 for every 64 tokens, and reading another
// part 1300.  (At 256 x 4096 x 4096, where those were measured.)
I8Job plan(int m, int n, int k, int nt, double *cycles) {
  I8Job j = {};
  j.m = m;
  j.n = n;
  j.tiles_c = (n + 2 * kHalf - 1) / (2 * kHalf);
  j.tiles_t = (m + nt - 1) / nt;
  j.stages = (k + kStageK - 1) / kStageK;
  const long tiles = (long)j.tiles_c * j.tiles_t;
  j.workers = (int)std::min<long>(std::max(os2_sm_count() / 2, 1), tiles);
  j.waves = (int)(tiles / j.workers);
  j.rest = (int)(tiles - (long)j.waves * j.workers);
  const int all = std::max(os2_sm_count() / 2, 1);
  if (tiles < all) {  // no whole wave: all tiles may be cut
    j.waves = 0;
    j.rest = (int)tiles;
    j.workers = all;
  }
  const double stage = nt == 256 ? 1450 : 1350;
  double least = 1e30;
  for (int parts = 1; j.rest && parts <= j.workers / j.rest && parts <= j.stages; parts++) {
    const double t = stage * ((j.stages + parts - 1) / parts) +
                     (parts > 1 ? 5000 + nt / 64 * (700 + 1300. * (parts - 1)) : 0);
    if (t < least) {
      least = t;
      j.parts = parts;
    }
  }
  if (!j.rest) {
    j.parts = 1;
    least = 0;
  }
  if (!j.waves) j.workers = j.rest * j.parts;
  *cycles = stage * j.waves * j.stages + least;
  return j;
}

// The tile width with the least time.
I8Job plan(int m, int n, int k, int *nt) {
  I8Job best = {};
  double least = 1e30;
  for (const int w : {64, 128, 256}) {
    double t;
    const I8Job j = plan(m, n, k, w, &t);
    if (t < least) {
      least = t;
      best = j;
      *nt = w;
    }
  }
  return best;
}

template <int NT>
cudaError_t launch(const I8Args &a, I8Job j, cudaStream_t s) {
  using T = Threads<NT>;
  static PerDevice ready;
  const cudaError_t attr_err = set_up(ready, k_i8tc<NT>, smem_tc<NT>(), T::all,
                                      128 * T::r_misc + 256 * T::r_epi + T::conv * T::r_conv);
  if (attr_err != cudaSuccess) return attr_err;
  CUtensorMap mw, mt;
  if (!map_w(&mw, a.W, a.k, a.n, a.ldw) ||
      !make_map(&mt, a.tokens, false, a.k, a.m, a.pitch, false, NT / 2))
    return cudaErrorInvalidValue;
  i8_fill(j, a);
  return launch_after(k_i8tc<NT>, 2 * j.workers, T::all, smem_tc<NT>(), s, mw, mt, j,
                      a.status);
}

}  // namespace

I8Sizes i8tc_sizes(int m, int n, int k) {
  int nt;
  const I8Job j = plan(m, n, k, &nt);
  return {j.parts > 1 ? 2 * j.rest : 0, j.parts > 1 ? (size_t)j.workers * 2 * nt * 128 : 0};
}

cudaError_t launch_i8tc(const I8Args &a, cudaStream_t s) {
  int nt;
  const I8Job j = plan(a.m, a.n, a.k, &nt);
  return nt == 64 ? launch<64>(a, j, s) : nt == 128 ? launch<128>(a, j, s) : launch<256>(a, j, s);
}
