// The matrix product of the vocabulary-head operators: D = A B^T of 16-bit
// operands on SM pairs, FP32 accumulators in tensor memory, the result handed
// to an epilogue functor tile by tile.
//
// A CTA pair (cluster of 2) owns 256 x 256 output tiles (tcgen05.mma
// cta_group::2, kind::f16), each CTA 128 rows of the A tile and 128 rows of the
// B tile; the pairs walk the tiles persistently.  A stage of the shared-memory
// ring holds 128 terms of both operands (64 KB a CTA), three stages.  Two
// accumulators of 256 TMEM columns alternate, so the epilogue of one unit (a
// tile, or a chunk of its terms) runs beside the MMAs of the next.
//
// Operands are K-major (rows of contiguous terms) or MN-major (terms are rows
// of contiguous entries, as a gradient's transposed operands are): both come by
// TMA in the 128-byte swizzle, and no transposed copy is made.  Entries outside
// a tensor map read as zero.
//
// Warps (384 threads): 0 TMA producer, 1 MMA issuer, 4-11 epilogue (each TMEM
// lane quarter twice: columns 0-127 and 128-255; 2 and 3 fill the first
// warpgroup).  Two epilogue warps a quarter, because the epilogues here do
// arithmetic on every entry, and most of the registers: one of them keeps 128
// sums a thread.
// A stage takes 1024 cycles of MMA.  2048 x 32768 x 2048 takes 149 to 154 us, whatever the
// operands' majors and the epilogue (1.8 PFLOP/s, 0.95 of cuBLAS's burst); 2048 x 38912 x
// 1024 100 us with the launches around it (1.63).
// Every wait is bounded; on expiry the CTA records OS2_ERR_TIMEOUT, lets its
// copies and MMAs drain (again bounded), frees its TMEM and returns.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "os2_internal.cuh"
#include "ptx.cuh"

namespace os2mm {

using namespace os2ptx;

constexpr int kHalf = 128;                      // rows of a tile that one CTA holds
constexpr int kBN = 256;
constexpr int kBK = 64;                         // terms of a k-block (128 bytes)
constexpr int kKbStage = 2;                     // k-blocks per stage
constexpr int kStageK = kBK * kKbStage;         // 128 terms
constexpr int kStages = 3;
constexpr uint32_t kBlockBytes = kHalf * kBK * 2;              // one operand, one k-block
constexpr uint32_t kOpBytes = kKbStage * kBlockBytes;          // one operand, one stage
constexpr int kEpiThreads = 256;
constexpr int kThreads = 128 + kEpiThreads;
// registers a thread: 384 x 168 at launch >= 128 x 64 + 256 x 216
constexpr int kRegsMisc = 64, kRegsEpi = 216;
static_assert(128 * kRegsMisc + 256 * kRegsEpi <= kThreads * 168, "registers");
constexpr uint32_t kScratch = 4096;             // an epilogue warp's own shared memory
constexpr size_t kSmem = 1024 + (size_t)kStages * 2 * kOpBytes + 512 + kEpiThreads / 32 * kScratch;
static_assert(kSmem <= 227 * 1024, "shared memory of the product kernel");
constexpr long long kWaitLimit = 4000000000LL;  // clock cycles (about 2 s)

// What one launch computes: an m x n output over k terms.
struct Job {
  int m, n, k;
  const int *m_dev;   // if set, the rows that count (<= m), known on the device only
  const int *k_dev;   // if set, the terms that count (<= k); the rest of the last stage is zero
  int chunk;          // stages per accumulation chunk (INT_MAX: the whole of k)
  int splits;         // parts of k, each a job of its own (at most the stages of k; 1 with k_dev)
  // Set where the launch in front is a product that this one reads nothing from
  // and that starts after all this one reads is there: it begins on the SMs that
  // the other leaves free, and ends after it.
  bool beside = false;
  const int *a_layer = nullptr;  // if set, the layer of A's map to take, known on the device only
};

__device__ __forceinline__ void set_status(int *status, int code) {
  if (status) atomicCAS(status, 0, code);
}

// Tile t of tiles_m x tiles_n in groups of 8 tile rows (the columns' operand
// tiles are reused from L2 within a group).
__device__ __forceinline__ void tile_coords(int t, int tiles_m, int tiles_n, int &tm, int &tn) {
  constexpr int GM = 8;
  const int group = t / (GM * tiles_n), first = group * GM;
  const int rows = min(GM, tiles_m - first), w = t - group * GM * tiles_n;
  tm = first + w % rows;
  tn = w / rows;
}

// Epi: a copyable struct with
//   void unit(uint32_t taddr, int row, int col0, int split, bool first, bool last, int m,
//             const CUtensorMap *mapD, uint8_t *scratch, int *status)
//   void finish()
// called by every lane of an epilogue warp (converged) with the TMEM address of
// its lane quarter's 128 columns, its own row of the output and the first of
// its 128 columns.  It reads TMEM with tcgen05.ld and waits for the loads; rows
// from m on and columns past the output are its business.  It may keep state
// between the chunks of a job (first, last).  scratch: kScratch bytes of the
// warp's own, on a 512-byte boundary; mapD: the output's tensor map, where it has
// one.  finish is called once, at the end.
template <bool BF16, bool A_MN, bool B_MN, class Epi>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    k_mm2(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapB,
          const __grid_constant__ CUtensorMap mapD, const Job job, const Epi epi_in, int *status) {
  constexpr uint32_t IDESC = idesc_f16_f32(2 * kHalf, kBN) |
                             (BF16 ? (1u << 7) | (1u << 10) : 0u) | (A_MN ? 1u << 15 : 0u) |
                             (B_MN ? 1u << 16 : 0u);
  constexpr uint32_t TMEM_COLS = 512;

  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~uintptr_t(1023));
  uint8_t *sA = smem;
  uint8_t *sB = smem + kStages * kOpBytes;
  uint64_t *full = reinterpret_cast<uint64_t *>(sB + kStages * kOpBytes);
  uint64_t *empty = full + kStages;
  uint64_t *acc_full = empty + kStages, *acc_empty = acc_full + 2, *mma_done = acc_empty + 2;
  uint32_t *s_tmem = reinterpret_cast<uint32_t *>(mma_done + 1);
  volatile int *s_abort = reinterpret_cast<volatile int *>(s_tmem + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = (int)(blockIdx.x >> 1), npairs = (int)(gridDim.x >> 1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; s++) {
      mbar_init(&full[s], 1);
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
    tma_prefetch_desc(&mapA);
    tma_prefetch_desc(&mapB);
  }
  if (warp == 1) {
    tmem_alloc2(s_tmem, TMEM_COLS);
    tmem_relinquish2();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the peer's barriers are initialised before any remote arrive / copy
  tc_fence_after();
  const uint32_t tmem_base = *s_tmem;

  // The next launch may start once all this one reads is there: a `beside` one, which reads
  // the same operands' kernel's output without waiting, relies on it.
  if (!job.beside) wait_for_previous();
  next_may_start();
  // counts known on the device only, never above the host's
  const int m = job.m_dev ? min(max(*job.m_dev, 0), job.m) : job.m;
  const int k = job.k_dev ? min(max(*job.k_dev, 0), job.k) : job.k;
  const int tiles_m = (m + 2 * kHalf - 1) / (2 * kHalf), tiles_n = (job.n + kBN - 1) / kBN;
  const int tiles = tiles_m * tiles_n, njobs = tiles * job.splits;
  // no term at all still runs one stage, of zeros, so that the epilogue writes its rows
  const int stages_k = max((k + kStageK - 1) / kStageK, 1);
  // job t: split t / tiles of tile t % tiles, over stages [stage0(t), stage1(t))
  auto stage0 = [&](int t) { return t / tiles * stages_k / job.splits; };
  auto stage1 = [&](int t) { return (t / tiles + 1) * stages_k / job.splits; };
  const int k_first = k == 0 ? (job.k + 255) / 256 * 256 : 0;  // past every map: zeros

  if (warp < 4) {
    regs_fewer<kRegsMisc>();
    if (warp == 0) {
      // ------------------------------------------------------------ producer
      if (lane == 0) {
        int stage = 0;
        uint32_t phase = 0, used = 0, last_par = 0;
        bool ok = true;
        const int la = job.a_layer ? *job.a_layer : 0;
        for (int t = pair; ok && t < njobs; t += npairs) {
          int tm, tn;
          tile_coords(t % tiles, tiles_m, tiles_n, tm, tn);
          const int ra = tm * 2 * kHalf + (int)rank * kHalf, rb = tn * kBN + (int)rank * kHalf;
          for (int ks = stage0(t); ks < stage1(t); ks++) {
            if (!mbar_wait_bounded(&empty[stage], phase ^ 1, s_abort, kWaitLimit)) {
              *s_abort = 1;
              set_status(status, OS2_ERR_TIMEOUT);
              ok = false;
              break;
            }
            const uint32_t fbar = mapa_shared(smem_u32(&full[stage]), 0);
            if (leader) mbar_arrive_expect_tx(&full[stage], 4 * kOpBytes);
#pragma unroll
            for (int h = 0; h < kKbStage; h++) {
              const int kx = k_first + ks * kStageK + h * kBK;
              uint8_t *da = sA + stage * kOpBytes + h * kBlockBytes;
              uint8_t *db = sB + stage * kOpBytes + h * kBlockBytes;
              if (A_MN) {  // two boxes of 64 rows of the tile x 64 terms
                tma_load_3d_pair(da, &mapA, fbar, ra, kx, la);
                tma_load_3d_pair(da + kBlockBytes / 2, &mapA, fbar, ra + 64, kx, la);
              } else {
                tma_load_3d_pair(da, &mapA, fbar, kx, ra, la);
              }
              if (B_MN) {
                tma_load_3d_pair(db, &mapB, fbar, rb, kx, 0);
                tma_load_3d_pair(db + kBlockBytes / 2, &mapB, fbar, rb + 64, kx, 0);
              } else {
                tma_load_3d_pair(db, &mapB, fbar, kx, rb, 0);
              }
            }
            used |= 1u << stage;
            last_par = (last_par & ~(1u << stage)) | (phase << stage);
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1;
            }
          }
        }
        // the pair's copies complete on the leader's barriers: it waits for the last of each stage
        if (leader)
          for (int s = 0; s < kStages; s++)
            if (used >> s & 1) {
              volatile int no_abort = 0;
              mbar_wait_bounded(&full[s], (last_par >> s) & 1, &no_abort, kWaitLimit);
            }
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer
      if (leader && lane == 0) {
        int stage = 0, unit = 0;
        uint32_t phase = 0;
        uint32_t aphase[2] = {0, 0};
        bool ok = true;
        for (int t = pair; ok && t < njobs; t += npairs) {
          const int begin = stage0(t), end = stage1(t);
          for (int ks0 = begin; ok && ks0 < end; unit++) {
            const int buf = unit & 1;
            if (!mbar_wait_bounded(&acc_empty[buf], aphase[buf] ^ 1, s_abort, kWaitLimit)) {
              *s_abort = 1;
              set_status(status, OS2_ERR_TIMEOUT);
              ok = false;
              break;
            }
            aphase[buf] ^= 1;
            tc_fence_after();
            const uint32_t d = tmem_base + (uint32_t)(buf * kBN);
            const int ks1 = end - ks0 > job.chunk ? ks0 + job.chunk : end;
            for (int ks = ks0; ks < ks1; ks++) {
              if (!mbar_wait_bounded(&full[stage], phase, s_abort, kWaitLimit)) {
                *s_abort = 1;
                set_status(status, OS2_ERR_TIMEOUT);
                ok = false;
                break;
              }
              tc_fence_after();
#pragma unroll
              for (int h = 0; h < kKbStage; h++) {
                const uint32_t a = smem_u32(sA + stage * kOpBytes + h * kBlockBytes);
                const uint32_t b = smem_u32(sB + stage * kOpBytes + h * kBlockBytes);
                // MN-major: 8-term atoms 1024 bytes apart, 64-row blocks 8192
                const uint64_t ad = A_MN ? sdesc_mn128(a, kBlockBytes / 2, 1024) : sdesc_k128(a);
                const uint64_t bd = B_MN ? sdesc_mn128(b, kBlockBytes / 2, 1024) : sdesc_k128(b);
                constexpr uint64_t AS = (A_MN ? 16 * 128 : 32) >> 4, BS = (B_MN ? 16 * 128 : 32) >> 4;
#pragma unroll
                for (int kk = 0; kk < kBK / 16; kk++)
                  umma2_f16(d, ad + AS * kk, bd + BS * kk, IDESC,
                            (ks > ks0 || h > 0 || kk > 0) ? 1u : 0u);
              }
              umma2_commit_mc(&empty[stage], 0x3);
              if (++stage == kStages) {
                stage = 0;
                phase ^= 1;
              }
            }
            if (ok) umma2_commit_mc(&acc_full[buf], 0x3);
            ks0 = ks1;
          }
        }
        umma2_commit_mc(mma_done, 0x1);
        volatile int no_abort = 0;
        mbar_wait_bounded(mma_done, 0, &no_abort, kWaitLimit);
      }
    }
  } else {
    regs_more<kRegsEpi>();
    // ------------------------------------------------------------ epilogue
    Epi epi = epi_in;
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const uint32_t lane_base = tmem_base + ((uint32_t)(quarter * 32) << 16) + half * 128;
    const uint32_t empty_leader[2] = {mapa_shared(smem_u32(&acc_empty[0]), 0),
                                      mapa_shared(smem_u32(&acc_empty[1]), 0)};
    uint8_t *scratch = reinterpret_cast<uint8_t *>(full) + 512 + (warp - 4) * kScratch;
    uint32_t aphase[2] = {0, 0};
    int unit = 0;
    bool ok = true;
    for (int t = pair; ok && t < njobs; t += npairs) {
      int tm, tn;
      tile_coords(t % tiles, tiles_m, tiles_n, tm, tn);
      const int row = tm * 2 * kHalf + (int)rank * kHalf + quarter * 32 + lane;
      const int col0 = tn * kBN + half * 128;
      const int begin = stage0(t), end = stage1(t);
      for (int ks0 = begin; ks0 < end; unit++) {
        const int ks1 = end - ks0 > job.chunk ? ks0 + job.chunk : end;
        const int buf = unit & 1;
        // every lane waits (acquire), then the warp reconverges on one verdict
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&acc_full[buf], aphase[buf],
                                                               s_abort, kWaitLimit));
        if (!ok) {
          *s_abort = 1;
          set_status(status, OS2_ERR_TIMEOUT);
          break;
        }
        aphase[buf] ^= 1;
        tc_fence_after();
        epi.unit(lane_base + (uint32_t)(buf * kBN), row, col0, t / tiles, ks0 == begin, ks1 == end,
                 m, &mapD, scratch, status);
        tc_fence_before();
        mbar_arrive_remote(empty_leader[buf]);
        ks0 = ks1;
      }
    }
    epi.finish();
  }

  // what follows waits for this launch alone, so this one ends after the one in front
  if (job.beside) wait_for_previous();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no CTA leaves while its peer may still touch its shared memory or TMEM
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc2(tmem_base, TMEM_COLS);
  }
}

// ------------------------------------------------------------------- host --
inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// Row-major matrices (`layers` in turn) of 16-bit entries: `rows` rows of `cols` entries,
// `pitch` entries apart.  mn: the terms run along the rows (box 64 x 64), else along
// the columns (box 64 x box_rows).  base and pitch * 2 must be multiples of 16.
inline bool make_map(CUtensorMap *map, const void *base, bool bf16, long cols, long rows,
                     long pitch, bool mn, int box_rows = kHalf, int layers = 1) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)layers};
  cuuint64_t strides[2] = {(cuuint64_t)pitch * 2, (cuuint64_t)pitch * 2 * (cuuint64_t)rows};
  cuuint32_t box[3] = {(cuuint32_t)kBK, (cuuint32_t)(mn ? kBK : box_rows), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
            const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Launches a kernel that waits (wait_for_previous) for the one in front of it.
template <class... P, class... A>
cudaError_t launch_after(void (*kernel)(P...), int grid, int block, size_t smem, cudaStream_t s,
                         const A &...args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// A row-major output that warps store (or add to) in blocks of 32 rows of 64 bytes,
// in the 64-byte swizzle; `layers` matrices of `rows` rows in turn.
inline bool make_store_map(CUtensorMap *map, void *base, CUtensorMapDataType type, int bytes,
                           long cols, long rows, long pitch, int layers = 1) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)layers};
  cuuint64_t strides[2] = {(cuuint64_t)pitch * bytes, (cuuint64_t)pitch * bytes * (cuuint64_t)rows};
  cuuint32_t box[3] = {(cuuint32_t)(64 / bytes), 32, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, type, 3, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Sets a kernel's shared memory, and checks that the block is launched with at
// least the registers that its roles take: a larger sum would wait for ever.
template <class K>
cudaError_t set_up(PerDevice &ready, K *kernel, size_t smem, int threads, int registers) {
  return os2_set_smem(ready, kernel, smem, [&]() -> cudaError_t {
    cudaFuncAttributes fa;
    const cudaError_t f = cudaFuncGetAttributes(&fa, kernel);
    if (f != cudaSuccess) return f;
    return fa.numRegs * threads < registers ? cudaErrorInvalidConfiguration : cudaSuccess;
  });
}

template <bool BF16, bool A_MN, bool B_MN, class Epi>
cudaError_t launch_mm2(const CUtensorMap &ma, const CUtensorMap &mb, const Job &job,
                       const Epi &epi, int *status, cudaStream_t s,
                       const CUtensorMap *md = nullptr) {
  static PerDevice ready;
  const cudaError_t attr_err = set_up(ready, k_mm2<BF16, A_MN, B_MN, Epi>, kSmem, kThreads,
                                      128 * kRegsMisc + 256 * kRegsEpi);
  if (attr_err != cudaSuccess) return attr_err;
  const long jobs = (long)((job.m + 2 * kHalf - 1) / (2 * kHalf)) * ((job.n + kBN - 1) / kBN) *
                    job.splits;
  if (jobs <= 0) return cudaSuccess;
  const int pairs = (int)std::min<long>(std::max(os2_sm_count() / 2, 1), jobs);
  return launch_after(k_mm2<BF16, A_MN, B_MN, Epi>, 2 * pairs, kThreads, kSmem, s, ma, mb,
                      md ? *md : ma, job, epi, status);
}

}  // namespace os2mm
