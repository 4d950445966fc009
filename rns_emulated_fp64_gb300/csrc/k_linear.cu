// A linear layer with bias, activation and residual in the product's epilogue, and its
// gradient:
//   z = x W^T + b,   y = r + act(z);     pre = z rounded, on request, for the gradient
//   D = dy act'(pre),   dx = D W,   dW = D^T x,   db = sum over the rows of D
//
// Products on the tensor cores (mm2.cuh; few tokens: k_linear_few.cu), sums FP32; y, pre, dx,
// dW and db are rounded once.  D is rounded to the operands' type, as an operand of the two
// products has to be (without an activation it is dy itself); db takes it unrounded.  In FP16, D is
// held times 7/8 where act' reaches 1.13, and dx and dW are multiplied by 8/7 before they are
// rounded: D would overflow where dy does not.  (A half would take a bit from D's smallest numbers.)
// Nothing is transposed in memory: W, D and x are read as they lie (MN-major operands).
//
// Bound by the tensor cores: 8192 x 16384 x 4096 BF16 with SiLU 555 us (1.98 PFLOP/s; in a loop, at
// the power cap, 645), 4096 x 16384 x 4096 with bias and GELU 304 and pre written, its gradient 680,
// of which D, bound by memory, is 75.  Small layers are bound by launches and the first tiles: 1000
// x 2047 x 1536 FP16 with a residual 22.5 us, its gradient 29.
#include "linear.cuh"
#include "mm2_epi.cuh"

using namespace os2mm;
using namespace os2lin;

namespace {

struct InLinear {};

// ------------------------------------------------------------------ forward
// A warp's 32 tokens x 128 outputs.  TMA: Y (and pre) leave in blocks of 32 x 32;
// otherwise through shared memory by rows.
template <bool BF16, bool TMA>
struct LinEpi {
  const void *bias;
  bool b32, bvec;      // bvec: on a 16-byte boundary
  int act;
  const uint16_t *R;
  long ldr;
  bool rvec;
  uint16_t *Y, *pre;
  long ldy, ldp;
  int n;
  BlockSender sender = {};

  // A block by rows: lane's own 64 bytes v to its row of out.
  __device__ __forceinline__ void rows(uint16_t *out, long ld, const uint4 (&v)[4], int row0, int m, int left, uint8_t *scratch) {
    const int lane = threadIdx.x & 31;
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 4; q++) *reinterpret_cast<uint4 *>(scratch + lane * 80 + q * 16) = v[q];
    __syncwarp();
#pragma unroll 8
    for (int rr = 0; rr < 32; rr++)
      if (row0 + rr < m && lane < left)
        out[(size_t)(row0 + rr) * ld + lane] = *reinterpret_cast<const uint16_t *>(scratch + rr * 80 + lane * 2);
  }

  __device__ __forceinline__ void unit(uint32_t taddr, int row, int col0, int, bool, bool, int m, const CUtensorMap *mapD,
                                       uint8_t *scratch, int *) {
    const int row0 = row - (int)(threadIdx.x & 31);
#pragma unroll 1
    for (int g = 0; g < 4; g++) {
      const int col = col0 + g * 32, left = n - col;
      if (left <= 0 || row0 >= m) break;  // the whole warp
      uint32_t r[32];
      __syncwarp();
      tmem_ld32(taddr + g * 32, r);
      uint4 res[4] = {};
      if (!TMA && R && !(rvec && left >= 32)) {
        // rows that are not on 16-byte boundaries: 64 bytes of one an instruction, through
        // shared memory
        const int lane = threadIdx.x & 31;
        __syncwarp();
#pragma unroll 8
        for (int rr = 0; rr < 32; rr++)
          if (row0 + rr < m && lane < left)
            *reinterpret_cast<uint16_t *>(scratch + rr * 80 + lane * 2) = R[(size_t)(row0 + rr) * ldr + col + lane];
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 4; q++) res[q] = *reinterpret_cast<const uint4 *>(scratch + lane * 80 + q * 16);
      } else if (R && row < m) {
        const uint16_t *p = R + (size_t)row * ldr + col;
        if (rvec && left >= 32) {
#pragma unroll
          for (int q = 0; q < 4; q++) res[q] = reinterpret_cast<const uint4 *>(p)[q];
        } else {
          uint32_t *w = reinterpret_cast<uint32_t *>(res);
#pragma unroll
          for (int i = 0; i < 32; i++)
            if (i < left) w[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
        }
      }
      tmem_wait_ld();
      float z[32];
#pragma unroll
      for (int i = 0; i < 32; i++) z[i] = __uint_as_float(r[i]);
      if (bias) {
        if (bvec && left >= 32 && b32) {
          const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(bias) + col);
#pragma unroll
          for (int q = 0; q < 8; q++) {
            const float4 f = __ldg(p + q);
            z[4 * q] += f.x, z[4 * q + 1] += f.y, z[4 * q + 2] += f.z, z[4 * q + 3] += f.w;
          }
        } else if (bvec && left >= 32) {
          const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(bias) + col);
#pragma unroll
          for (int q = 0; q < 4; q++) {
            const uint4 u = __ldg(p + q);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int e = 0; e < 8; e++) z[8 * q + e] += widen16<BF16>((uint16_t)(w[e >> 1] >> (16 * (e & 1))));
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; i++)
            if (i < left) z[i] += bias_at<BF16>(bias, b32, col + i);
        }
      }
      auto send = [&](uint16_t *out, long ld, const CUtensorMap *map) {
        uint4 v[4];
#pragma unroll
        for (int q = 0; q < 4; q++) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; i++) w[i] = pack2<BF16>(z[8 * q + 2 * i], z[8 * q + 2 * i + 1]);
          v[q] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        // (rows from m on and columns from n on are cut off by the map)
        if constexpr (TMA) sender.send(map, scratch, v, col, row0, 0, false);
        else rows(out + col, ld, v, row0, m, left, scratch);
      };
      if (pre) send(pre, ldp, mapD + 1);
      const uint32_t *w = reinterpret_cast<const uint32_t *>(res);
      os2act::values(z, act);
      if (R) {
#pragma unroll
        for (int i = 0; i < 32; i++) z[i] += widen16<BF16>((uint16_t)(w[i >> 1] >> (16 * (i & 1))));
      }
      send(Y, ldy, mapD);
    }
  }
  __device__ __forceinline__ void finish() {
    if (TMA) sender.finish();
  }
};

template <bool BF16>
cudaError_t forward(const LinearArgs &a, cudaStream_t s) {
  CUtensorMap mx, mw, my, mp;
  if (!make_map(&mx, a.X, BF16, a.k, a.m, a.ldx, false) || !make_map(&mw, a.W, BF16, a.k, a.n, a.ldw, false))
    return cudaErrorInvalidValue;
  const Job job{a.m, a.n, a.k, nullptr, nullptr, INT_MAX, 1};
  auto fill = [&](auto epi) {
    epi.bias = a.bias, epi.b32 = a.b32, epi.bvec = reinterpret_cast<uintptr_t>(a.bias) % 16 == 0;
    epi.act = a.act;
    epi.R = a.R, epi.ldr = a.ldr, epi.rvec = tma_rows(a.R, a.ldr);
    epi.Y = a.Y, epi.pre = a.pre, epi.ldy = a.ldy, epi.ldp = a.ldp;
    epi.n = a.n;
    return epi;
  };
  if (tma_rows(a.Y, a.ldy) && (!a.pre || tma_rows(a.pre, a.ldp))) {
    const CUtensorMapDataType type = BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    if (!make_store_map(&my, a.Y, type, 2, a.n, a.m, a.ldy) || (a.pre && !make_store_map(&mp, a.pre, type, 2, a.n, a.m, a.ldp)))
      return cudaErrorInvalidValue;
    return launch_mm2<BF16, false, false>(mx, mw, job, fill(LinEpi<BF16, true>{}), a.status, s, &my, a.pre ? &mp : nullptr);
  }
  return launch_mm2<BF16, false, false>(mx, mw, job, fill(LinEpi<BF16, false>{}), a.status, s);
}

// ----------------------------------------------------------------- backward
struct Slope {
  int m, n, act;
  const uint16_t *dY, *pre;
  long lddy, ldp;
  uint16_t *D;        // or null
  long pitch;
  float held;         // D is held times this
  float *part;        // [strips][part_pitch] sums of columns, or null
  long part_pitch;
  void *db;           // the sums themselves, where there is one strip
  bool db32;
  int strip;          // rows of a strip
  bool vec;
};

// A matrix whose rows TMA does not take, and where they go.
struct Copy {
  const uint16_t *src;
  long ld;
  uint16_t *dst;
  long pitch;
  int rows, k, ctas;
};

// What the products need besides, in one launch, by `slopes` CTAs: D = dy act'(pre), and the
// columns' sums over a strip of rows, 64 groups of 8 columns by 4 rows a CTA; bound by memory.  Rows
// that are not on 16-byte boundaries are read entry by entry, D's own are.  By the other CTAs:
// copies.
constexpr int kSlopeRows = 4;
template <bool BF16>
__global__ void __launch_bounds__(64 * kSlopeRows) k_linear_prepare(const Slope p, int slopes, const Copy c0, const Copy c1) {
  static_assert(64 * kSlopeRows == 256, "repack's threads");
  __shared__ float s[kSlopeRows][64][9];
  start_call();
  if ((int)blockIdx.x >= slopes) {
    const int cta = (int)blockIdx.x - slopes;
    if (cta < c0.ctas) repack(c0.src, c0.ld, c0.dst, c0.pitch, c0.rows, c0.k, cta, c0.ctas);
    else repack(c1.src, c1.ld, c1.dst, c1.pitch, c1.rows, c1.k, cta - c0.ctas, c1.ctas);
    return;
  }
  const int across = (p.n + 511) / 512, cx = (int)blockIdx.x % across, cy = (int)blockIdx.x / across;
  const int group = threadIdx.x & 63, lane_row = threadIdx.x >> 6;
  const int col = (cx * 64 + group) * 8, left = p.n - col;
  const int r0 = cy * p.strip, r1 = min(p.m, r0 + p.strip);
  float sum[8] = {};
  if (left > 0)
#pragma unroll 4
    for (int row = r0 + lane_row; row < r1; row += kSlopeRows) {
      uint4 g = make_uint4(0, 0, 0, 0), z = g;
      auto take = [&](const uint16_t *q) {
        if (p.vec && left >= 8) return __ldg(reinterpret_cast<const uint4 *>(q));
        uint32_t w[4] = {};
#pragma unroll
        for (int i = 0; i < 8; i++)
          if (i < left) w[i >> 1] |= (uint32_t)__ldg(q + i) << (16 * (i & 1));
        return make_uint4(w[0], w[1], w[2], w[3]);
      };
      g = take(p.dY + (size_t)row * p.lddy + col);
      if (p.act != OS2_ACT_NONE) {
        z = take(p.pre + (size_t)row * p.ldp + col);
        z = make_uint4(os2act::near0<BF16>(z.x), os2act::near0<BF16>(z.y), os2act::near0<BF16>(z.z), os2act::near0<BF16>(z.w));
      }
      const uint32_t gw[4] = {g.x, g.y, g.z, g.w}, zw[4] = {z.x, z.y, z.z, z.w};
      float d[8], at[8];
#pragma unroll
      for (int i = 0; i < 8; i++) {
        d[i] = widen16<BF16>((uint16_t)(gw[i >> 1] >> (16 * (i & 1))));
        at[i] = widen16<BF16>((uint16_t)(zw[i >> 1] >> (16 * (i & 1))));
      }
      os2act::slopes(d, at, p.act);
#pragma unroll
      for (int i = 0; i < 8; i++) sum[i] += d[i];
      if (p.D) {
        if (!BF16)
#pragma unroll
          for (int i = 0; i < 8; i++) d[i] *= p.held;
        *reinterpret_cast<uint4 *>(p.D + (size_t)row * p.pitch + col) =
            make_uint4(pack2<BF16>(d[0], d[1]), pack2<BF16>(d[2], d[3]), pack2<BF16>(d[4], d[5]), pack2<BF16>(d[6], d[7]));
      }
    }
  if (!p.part && !p.db) return;
#pragma unroll
  for (int i = 0; i < 8; i++) s[lane_row][group][i] = sum[i];
  __syncthreads();
  for (int i = threadIdx.x; i < 512; i += 64 * kSlopeRows) {
    const int c = cx * 512 + i;
    float x = 0.f;
#pragma unroll
    for (int r = 0; r < kSlopeRows; r++) x += s[r][i >> 3][i & 7];
    if (c >= p.n) continue;
    if (!p.db) p.part[(size_t)cy * p.part_pitch + c] = x;
    else if (p.db32) static_cast<float *>(p.db)[c] = x;
    else static_cast<uint16_t *>(p.db)[c] = pack1<BF16>(x);
  }
}

// A product's result rounded once, in FP16 times `by` before it: by TMA where its rows allow it, else by rows.
template <bool BF16, bool TMA>
struct RoundEpi {
  uint16_t *out;
  long ld;
  int n;
  float by;
  BlockSender sender = {};

  __device__ __forceinline__ void unit(uint32_t taddr, int row, int col0, int, bool, bool, int m, const CUtensorMap *mapD,
                                       uint8_t *scratch, int *) {
    const int lane = threadIdx.x & 31, row0 = row - lane;
#pragma unroll 1
    for (int g = 0; g < 4; g++) {
      const int left = n - (col0 + g * 32);
      if (left <= 0 || row0 >= m) break;  // the whole warp
      uint32_t r[32];
      __syncwarp();
      tmem_ld32(taddr + g * 32, r);
      tmem_wait_ld();
      float z[32];
#pragma unroll
      for (int i = 0; i < 32; i++) z[i] = BF16 ? __uint_as_float(r[i]) : __uint_as_float(r[i]) * by;
      uint4 v[4];
#pragma unroll
      for (int q = 0; q < 4; q++) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; i++) w[i] = pack2<BF16>(z[8 * q + 2 * i], z[8 * q + 2 * i + 1]);
        v[q] = make_uint4(w[0], w[1], w[2], w[3]);
      }
      if constexpr (TMA) {
        sender.send(mapD, scratch, v, col0 + g * 32, row0, 0, false);
      } else {
#pragma unroll
        for (int q = 0; q < 4; q++) *reinterpret_cast<uint4 *>(scratch + lane * 80 + q * 16) = v[q];
        __syncwarp();
        uint16_t *dst = out + col0 + g * 32;
#pragma unroll 8
        for (int rr = 0; rr < 32; rr++)
          if (row0 + rr < m && lane < left)
            dst[(size_t)(row0 + rr) * ld + lane] = *reinterpret_cast<const uint16_t *>(scratch + rr * 80 + lane * 2);
      }
    }
  }
  __device__ __forceinline__ void finish() {
    if (TMA) sender.finish();
  }
};

// What is left after the products: their parts added up in their order, and db's strips, each
// rounded once, in one launch.
struct Parts {
  const float *acc;   // [parts][layer]
  int parts, rows;
  long layer, pitch;
  int cols;
  void *out;
  long ld;
  bool vec, f32;
  float by;           // in FP16, the sums times this
  int groups() const { return parts ? (int)std::min<long>(((cols + 3L) / 4 * rows + 255) / 256, 1 << 20) : 0; }
};
struct Finish {
  Parts p[3];
};
template <bool BF16>
__global__ void __launch_bounds__(256) k_linear_finish(const Finish f, int g0, int g1, bool early) {
  // CTAs up to g0 take the first, up to g1 the second, the rest the third.  Behind a product
  // (early) db's CTAs need not wait for its end: the strips were there before it began.  But they
  // end after it, as what follows waits for this launch alone.
  const int which = (int)blockIdx.x < g0 ? 0 : (int)blockIdx.x < g1 ? 1 : 2;
  next_may_start();
  if (which != 2 || !early) wait_for_previous();
  const Parts &p = f.p[which];
  const int first = which == 0 ? 0 : which == 1 ? g0 : g1, ctas = (which == 0 ? g0 : which == 1 ? g1 : (int)gridDim.x) - first;
  if (which == 2) {
    // db: 32 columns a CTA, 32 threads for each four of them a strip in 32 each (128 columns and 8
    // threads: 390 strips of 1280 columns took 11 us more)
    __shared__ float4 s[32][9];
    const int strip = threadIdx.x >> 3, h = ((int)(blockIdx.x - first) * 8 + (threadIdx.x & 7)) * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (h < p.cols)
#pragma unroll 4
      for (int t = strip; t < p.parts; t += 32) {
        const float4 v = __ldg(reinterpret_cast<const float4 *>(p.acc + t * p.layer + h));
        x.x += v.x, x.y += v.y, x.z += v.z, x.w += v.w;
      }
    s[strip][threadIdx.x & 7] = x;
    __syncthreads();
    const int i = threadIdx.x, c = (int)(blockIdx.x - first) * 32 + i;
    if (i < 32 && c < p.cols) {
      float sum = 0.f;
#pragma unroll
      for (int t = 0; t < 32; t++) sum += reinterpret_cast<const float *>(&s[t][0])[i];
      if (p.f32) static_cast<float *>(p.out)[c] = sum;
      else static_cast<uint16_t *>(p.out)[c] = pack1<BF16>(sum);
    }
    if (early) wait_for_previous();
    return;
  }
  const int per = (p.cols + 3) / 4;
  const long total = (long)per * p.rows;
  for (long i = (long)(blockIdx.x - first) * 256 + threadIdx.x; i < total; i += (long)ctas * 256) {
    const long row = i / per;
    const int h = (int)(i - row * per) * 4;
    const float *a = p.acc + row * p.pitch + h;
    float x[4] = {};
    for (int p0 = 0; p0 < p.parts; p0 += 8) {
      float4 v[8];
#pragma unroll
      for (int u = 0; u < 8; u++)
        v[u] = p0 + u < p.parts ? __ldg(reinterpret_cast<const float4 *>(a + (p0 + u) * p.layer)) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int u = 0; u < 8; u++) x[0] += v[u].x, x[1] += v[u].y, x[2] += v[u].z, x[3] += v[u].w;
    }
    if (!BF16)
#pragma unroll
      for (int q = 0; q < 4; q++) x[q] *= p.by;
    uint16_t *dst = static_cast<uint16_t *>(p.out) + row * p.ld + h;
    if (p.vec && h + 4 <= p.cols) {
      *reinterpret_cast<uint2 *>(dst) = make_uint2(pack2<BF16>(x[0], x[1]), pack2<BF16>(x[2], x[3]));
    } else {
#pragma unroll
      for (int q = 0; q < 4; q++)
        if (h + q < p.cols) dst[q] = pack1<BF16>(x[q]);
    }
  }
}

// y (and pre) of a product whose terms were cut into parts: added up in their order, four outputs a thread.
struct Join {
  LinearArgs a;
  const float *acc;   // [parts][layer]
  int parts;
  long layer, pitch;
  bool rwhole, ywhole, pwhole;  // four entries on a boundary of their own
};
template <bool BF16>
__global__ void __launch_bounds__(256) k_linear_join(const Join j) {
  next_may_start();
  wait_for_previous();
  const LinearArgs &a = j.a;
  const int per = (a.n + 3) / 4;
  const long total = (long)per * a.m;
  for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < total; i += (long)gridDim.x * 256) {
    const long row = i / per;
    const int h = (int)(i - row * per) * 4, left = a.n - h;
    const float *p = j.acc + row * j.pitch + h;
    const uint2 r = a.R ? load4(a.R + row * a.ldr + h, left, j.rwhole) : make_uint2(0, 0);
    float z[4] = {};
    for (int p0 = 0; p0 < j.parts; p0 += 4) {
      float4 v[4];
#pragma unroll
      for (int u = 0; u < 4; u++)
        v[u] = p0 + u < j.parts ? __ldg(reinterpret_cast<const float4 *>(p + (p0 + u) * j.layer)) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int u = 0; u < 4; u++) z[0] += v[u].x, z[1] += v[u].y, z[2] += v[u].z, z[3] += v[u].w;
    }
    if (a.bias)
#pragma unroll
      for (int q = 0; q < 4; q++)
        if (q < left) z[q] += bias_at<BF16>(a.bias, a.b32, h + q);
    if (a.pre) store4(a.pre + row * a.ldp + h, make_uint2(pack2<BF16>(z[0], z[1]), pack2<BF16>(z[2], z[3])), left, j.pwhole);
    os2act::values(z, a.act);
    if (a.R) {
      const uint32_t w[2] = {r.x, r.y};
#pragma unroll
      for (int q = 0; q < 4; q++) z[q] += widen16<BF16>((uint16_t)(w[q >> 1] >> (16 * (q & 1))));
    }
    store4(a.Y + row * a.ldy + h, make_uint2(pack2<BF16>(z[0], z[1]), pack2<BF16>(z[2], z[3])), left, j.ywhole);
  }
}

// db where D is dy as it lies: 64 columns a CTA, 32 rows at a time; beside a product of the same call
// (which waited for what lies before the call) and ending after it, or alone.
constexpr int kSumsRows = 1024;
template <bool BF16>
__global__ void __launch_bounds__(256) k_linear_sums(const uint16_t *dY, long ld, int m, int n, void *db, bool f32, bool beside) {
  __shared__ float s[32][65];
  if (!beside) wait_for_previous();
  next_may_start();
  const int group = threadIdx.x & 7, r0 = threadIdx.x >> 3, col = blockIdx.x * 64 + group * 8, left = n - col;
  float sum[8] = {};
  if (left > 0)
#pragma unroll 8
    for (int row = r0; row < m; row += 32) {
      const uint16_t *q = dY + (size_t)row * ld + col;
      uint32_t w[4] = {};
      if (left >= 8) {
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(q));
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
      } else {
#pragma unroll
        for (int i = 0; i < 8; i++)
          if (i < left) w[i >> 1] |= (uint32_t)__ldg(q + i) << (16 * (i & 1));
      }
#pragma unroll
      for (int i = 0; i < 8; i++) sum[i] += widen16<BF16>((uint16_t)(w[i >> 1] >> (16 * (i & 1))));
    }
#pragma unroll
  for (int i = 0; i < 8; i++) s[r0][group * 8 + i] = sum[i];
  __syncthreads();
  const int c = blockIdx.x * 64 + (int)threadIdx.x;
  if (threadIdx.x < 64 && c < n) {
    float x = 0.f;
#pragma unroll
    for (int r = 0; r < 32; r++) x += s[r][threadIdx.x];
    if (f32) static_cast<float *>(db)[c] = x;
    else static_cast<uint16_t *>(db)[c] = pack1<BF16>(x);
  }
  if (beside) wait_for_previous();
}

// Parts of a product of rows x cols over `terms`: as many as let all SM pairs work, by an
// estimate in microseconds (0.55 a stage; the parts written and read once at 5 TB/s).
int parts_of(long rows, long cols, int terms, double *us = nullptr) {
  const long tiles = (rows + 255) / 256 * ((cols + 255) / 256), pairs = std::max(os2_sm_count() / 2, 1);
  const int stages = (terms + kStageK - 1) / kStageK;
  const double bytes = (double)os2_round_up((size_t)rows, 256) * os2_round_up((size_t)cols, 256) * 8;
  int best = 1;
  double least = 1e30;
  for (int s = 1; s <= std::min(stages, 32); s++) {
    if (s > 1 && bytes / 2 * s > 268435456.) break;
    const double t = (double)((tiles * s + pairs - 1) / pairs) * ((stages + s - 1) / s) * 0.55 + (s > 1 ? bytes * s / 5e6 + 4 : 0);
    if (t < least) least = t, best = s;
  }
  if (us) *us = 2.3 + least + (best > 1 ? 0. : 2.);
  return best;
}

// What one of the gradient's products asks for: its result is rows x cols.
struct Product {
  int rows, cols, parts;
  size_t acc_bytes() const {
    return parts > 1 ? (size_t)parts * os2_round_up((size_t)rows, 256) * os2_round_up((size_t)cols, 256) * 4 : 0;
  }
};

template <bool BF16, bool A_MN>
cudaError_t product(const CUtensorMap &ma, const CUtensorMap &mb, const Product &p, int terms, bool beside, uint16_t *out,
                    long ld, float by, float *acc, int *status, cudaStream_t s) {
  const Job job{p.rows, p.cols, terms, nullptr, nullptr, INT_MAX, p.parts, beside};
  CUtensorMap mo;
  if (p.parts > 1) {
    const long pitch = (long)os2_round_up((size_t)p.cols, 256), rows = (long)os2_round_up((size_t)p.rows, 256);
    if (!make_store_map(&mo, acc, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, pitch, rows, pitch, p.parts)) return cudaErrorInvalidValue;
    return launch_mm2<BF16, A_MN, true>(ma, mb, job, SumEpi<InLinear>{false}, status, s, &mo);
  }
  if (tma_rows(out, ld)) {
    if (!make_store_map(&mo, out, BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, p.cols, p.rows, ld))
      return cudaErrorInvalidValue;
    return launch_mm2<BF16, A_MN, true>(ma, mb, job, RoundEpi<BF16, true>{out, ld, p.cols, by}, status, s, &mo);
  }
  return launch_mm2<BF16, A_MN, true>(ma, mb, job, RoundEpi<BF16, false>{out, ld, p.cols, by}, status, s);
}

Parts parts_of_product(const Product &p, const float *acc, void *out, long ld, float by) {
  const long pitch = (long)os2_round_up((size_t)p.cols, 256), rows = (long)os2_round_up((size_t)p.rows, 256);
  return {acc, p.parts > 1 ? p.parts : 0, p.rows, rows * pitch, pitch, p.cols, out, ld, tma_rows(out, ld), false, by};
}

// --------------------------------------------------------------------- host
struct Forward {
  size_t x, w, total;  // copies of X and W, where TMA does not take them as they lie
  long pitch;
};
Forward forward_layout(int m, int n, int k, const void *X, long ldx, const void *W, long ldw) {
  Forward f = {};
  f.pitch = (long)os2_round_up((size_t)k, 8);
  auto take = [&](size_t bytes) {
    const size_t o = f.total;
    f.total += os2_round_up(bytes, 256);
    return o;
  };
  if (!tma_rows(X, ldx)) f.x = take((size_t)m * f.pitch * 2);
  if (!tma_rows(W, ldw)) f.w = take((size_t)n * f.pitch * 2);
  f.total = std::max<size_t>(f.total, 256);
  return f;
}

// The 2-SM product's time by an estimate in microseconds (fitted as linear_few_plan): a start of 2.3, 0.57
// a stage of 128 terms; a tile's epilogue takes `epi` beside the next tile's stages.
double tiles_us(int m, int n, int k, double epi) {
  const long tiles = (long)((m + 255) / 256) * ((n + 255) / 256), pairs = std::max(os2_sm_count() / 2, 1);
  const double waves = (double)((tiles + pairs - 1) / pairs), stages = ((k + kStageK - 1) / kStageK) * 0.57;
  return std::max(2.3 + stages + (waves - 1) * std::max(stages, epi) + epi, 4.6 + 2. * n * k / 6.3e6);
}

// The parts that y's product would be cut into, their memory and the time by an estimate (as tiles_us;
// the parts written and read at 6 TB/s and 4.5 for the second launch): none where that gains nothing
// whatever the epilogue.  us with and without: 400 x 4096 x
// 4096 21.1 and 23.4, 600 x 2000 x 5000 with GELU 20.3 and 35.9, 2048 x 600 x 4096 16.4 and 22.2.
struct Cut {
  int parts;
  size_t bytes;
  double us;
};
Cut cut_of(int m, int n, int k) {
  const long tiles = (long)((m + 255) / 256) * ((n + 255) / 256), pairs = std::max(os2_sm_count() / 2, 1);
  const int stages = (k + kStageK - 1) / kStageK;
  Cut best = {1, 0, tiles_us(m, n, k, 12.9)};
  if (m <= 16) return best;
  for (int s = 2; s <= std::min(stages, 8) && tiles * s <= 2 * pairs; s++) {
    const size_t bytes = Product{m, n, s}.acc_bytes();
    const double t = 2.3 + (double)((tiles * s + pairs - 1) / pairs) * ((stages + s - 1) / s) * 0.57 + bytes * 2. / 6e6 + 4.5;
    if (t < best.us) best = {s, bytes, t};
  }
  return best;
}

struct Backward {
  Forward f;
  bool d;              // whether D is there (an activation, or dY that TMA does not take)
  long pitch;          // of D
  int strips, strip;
  bool few;            // dx by k_linear_few.cu
  Product dx, dw;
  size_t D, part, accx, accw, total;
};
Backward backward_layout(int m, int n, int k, const void *X, long ldx, const void *W, long ldw, const void *dY, long lddy, int act) {
  Backward b = {};
  b.f = forward_layout(m, n, k, X, ldx, W, ldw);
  b.total = b.f.total;
  auto take = [&](size_t bytes) {
    const size_t o = b.total;
    b.total += os2_round_up(bytes, 256);
    return o;
  };
  b.d = act != OS2_ACT_NONE || !tma_rows(dY, lddy);
  b.pitch = (long)os2_round_up((size_t)n, 8);
  // strips of rows: eight CTAs an SM, of at least 8 rows (32: 1000 x 2047 x 1536 44 us, now 35)
  const int across = (n + 511) / 512;
  b.strip = std::max(8, (int)(((long)m * across + 8 * os2_sm_count() - 1) / (8 * os2_sm_count())));
  b.strips = (m + b.strip - 1) / b.strip;
  double here;
  b.dx = {m, k, parts_of(m, k, n, &here)};
  b.few = m <= 16 || linear_few_plan(m, k, n, false).us <= here;
  if (b.few) b.dx.parts = 1;
  b.dw = {n, k, parts_of(n, k, m)};
  if (b.d) b.D = take((size_t)m * b.pitch * 2);
  b.part = take((size_t)b.strips * b.pitch * 4);
  b.accx = take(b.dx.acc_bytes());
  b.accw = take(b.dw.acc_bytes());
  return b;
}

// The way that a call takes: few tokens' tiles, those of the 2-SM product, or these with their terms
// cut into parts.  Epilogues of 256 x 256 here: 2.3 us, an activation 1.7, pre 1.2, a
// residual 0.7, rows that TMA does not store or take 7.  1024 tokens of 8192 x 256 with GELU 15 us
// here and 33 there, of 1024 x 8192 43 and 22.
enum Way { kFew, kTiles, kParts };
Way way_of(int m, int n, int k, bool act, bool pre, bool residual, bool rows, const Cut &cut) {
  if (m <= 16) return kFew;
  const double epi = 2.3 + (act ? 1.7 : 0.) + (pre ? 1.2 : 0.) + (residual ? 0.7 : 0.) + (rows ? 0. : 7.);
  const double few = linear_few_plan(m, n, k, act || pre).us, tiles = tiles_us(m, n, k, epi);
  if (cut.parts > 1 && cut.us < std::min(few, tiles)) return kParts;
  return few <= tiles ? kFew : kTiles;
}

template <class T>
T *at(void *ws, size_t off) {
  return reinterpret_cast<T *>(static_cast<char *>(ws) + off);
}

template <bool BF16>
cudaError_t in_parts(const LinearArgs &a, int parts, float *acc, cudaStream_t s) {
  const long pitch = (long)os2_round_up((size_t)a.n, 256), rows = (long)os2_round_up((size_t)a.m, 256);
  CUtensorMap mx, mw, mo;
  if (!make_map(&mx, a.X, BF16, a.k, a.m, a.ldx, false) || !make_map(&mw, a.W, BF16, a.k, a.n, a.ldw, false) ||
      !make_store_map(&mo, acc, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, pitch, rows, pitch, parts))
    return cudaErrorInvalidValue;
  const Job job{a.m, a.n, a.k, nullptr, nullptr, INT_MAX, parts};
  const cudaError_t e = launch_mm2<BF16, false, false>(mx, mw, job, SumEpi<InLinear>{false}, a.status, s, &mo);
  if (e != cudaSuccess) return e;
  auto whole = [](const void *p, long ld) { return reinterpret_cast<uintptr_t>(p) % 8 == 0 && ld % 4 == 0; };
  const Join j{a, acc, parts, rows * pitch, pitch, whole(a.R, a.ldr), whole(a.Y, a.ldy), whole(a.pre, a.ldp)};
  const long total = (a.n + 3L) / 4 * a.m;
  return launch_after(k_linear_join<BF16>, (int)std::min<long>((total + 255) / 256, 8L * os2_sm_count()), 256, 0, s, j);
}

// X and W (null: not read) as TMA takes them, beside D and db.
template <bool BF16>
cudaError_t prepare(const Forward &f, LinearArgs &a, void *ws, const Slope *slope, int strips, cudaStream_t s) {
  Copy c[2] = {};
  auto copy = [&](Copy &c, const uint16_t *&p, long &ld, int rows, size_t off) {
    if (!p || tma_rows(p, ld)) return;
    c = {p, ld, at<uint16_t>(ws, off), f.pitch, rows, a.k, repack_ctas(f.pitch, rows)};
    p = c.dst, ld = f.pitch;
  };
  copy(c[0], a.X, a.ldx, a.m, f.x);
  copy(c[1], a.W, a.ldw, a.n, f.w);
  const int slopes = slope ? (a.n + 511) / 512 * strips : 0, ctas = slopes + c[0].ctas + c[1].ctas;
  return ctas ? launch_after(k_linear_prepare<BF16>, ctas, 64 * kSlopeRows, 0, s, slope ? *slope : Slope{}, slopes, c[0], c[1])
              : cudaSuccess;
}

template <bool BF16>
cudaError_t backward(LinearArgs a, const Backward &b, const uint16_t *dY, long lddy, const uint16_t *pre, long ldp, uint16_t *dX,
                     long lddx, uint16_t *dW, long lddw, void *db, int db_dtype, void *ws, cudaStream_t s) {
  float *part = at<float>(ws, b.part), *accx = at<float>(ws, b.accx), *accw = at<float>(ws, b.accw);
  const bool products = dX || dW;
  const uint16_t *D = dY;
  long ldd = lddy;
  Slope p = {};
  const bool steep = !BF16 && a.act != OS2_ACT_NONE && a.act != OS2_ACT_RELU;
  const float by = steep ? 8.f / 7.f : 1.f;
  p.held = steep ? 0.875f : 1.f;
  // (not b.d: TMA takes dY, and so does k_linear_sums; by what it is given alone, so that db does not
  // depend on what else is asked for)
  const bool sums = db && !b.d && a.m <= kSumsRows;
  const bool slope = (db && !sums) || (b.d && products), one = b.strips == 1 || sums;
  if (slope) {
    p.m = a.m, p.n = a.n, p.act = a.act;
    p.dY = dY, p.lddy = lddy, p.pre = pre, p.ldp = ldp;
    p.vec = tma_rows(dY, lddy) && (a.act == OS2_ACT_NONE || tma_rows(pre, ldp));
    p.part = db && !one ? part : nullptr;
    p.part_pitch = b.pitch;
    p.db = db && one ? db : nullptr;
    p.db32 = db_dtype == OS2_F32;
    p.strip = b.strip;
    if (b.d && products) {
      p.D = at<uint16_t>(ws, b.D), p.pitch = b.pitch;
      D = p.D, ldd = b.pitch;
    }
  }
  if (!dX) a.W = nullptr;
  if (!dW) a.X = nullptr;
  cudaError_t e = prepare<BF16>(b.f, a, ws, slope ? &p : nullptr, b.strips, s);
  if (e != cudaSuccess) return e;
  auto finish = [&](const Parts &x, const Parts &w) {
    Finish f = {{x, w, {}}};
    if (db && !one) f.p[2] = {part, b.strips, 1, b.pitch, b.pitch, a.n, db, b.pitch, false, db_dtype == OS2_F32, 1.f};
    const int most = 8 * os2_sm_count(), g0 = std::min(f.p[0].groups(), most), g1 = g0 + std::min(f.p[1].groups(), most),
              g2 = g1 + (db && !one ? (a.n + 31) / 32 : 0);
    return g2 ? launch_after(k_linear_finish<BF16>, g2, 256, 0, s, f, g0, g1, products) : cudaSuccess;
  };
  auto add_up = [&]() {
    return launch_after(k_linear_sums<BF16>, (a.n + 63) / 64, 256, 0, s, dY, lddy, a.m, a.n, db, db_dtype == OS2_F32, products);
  };
  if (!products) return sums ? add_up() : finish({}, {});
  CUtensorMap md, mdt, mw, mx;
  if (dX && b.few) {
    LinearArgs f = {};
    f.m = a.m, f.n = a.k, f.k = a.n;
    f.bf16 = BF16;
    f.X = D, f.ldx = ldd, f.W = a.W, f.ldw = a.ldw;
    f.Y = dX, f.ldy = lddx;
    f.by = by;
    f.status = a.status;
    e = launch_linear_few(f, true, s);
    if (e != cudaSuccess) return e;
  } else if (dX) {
    if (!make_map(&md, D, BF16, a.n, a.m, ldd, false) || !make_map(&mw, a.W, BF16, a.k, a.n, a.ldw, true))
      return cudaErrorInvalidValue;
    e = product<BF16, false>(md, mw, b.dx, a.n, false, dX, lddx, by, accx, a.status, s);
    if (e != cudaSuccess) return e;
  }
  if (dW) {
    if (!make_map(&mdt, D, BF16, a.n, a.m, ldd, true) || !make_map(&mx, a.X, BF16, a.k, a.m, a.ldx, true))
      return cudaErrorInvalidValue;
    // (dW's product reads nothing of dX's)
    e = product<BF16, true>(mdt, mx, b.dw, a.m, dX != nullptr, dW, lddw, by, accw, a.status, s);
    if (e != cudaSuccess) return e;
  }
  if (sums) {
    e = add_up();
    if (e != cudaSuccess) return e;
  }
  return finish(dX ? parts_of_product(b.dx, accx, dX, lddx, by) : Parts{}, dW ? parts_of_product(b.dw, accw, dW, lddw, by) : Parts{});
}

bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
constexpr int kMaxRows = 1 << 22;

os2_status check(int m, int n, int k, int dtype, const void *X, int ldx, const void *W, int ldw, int act) {
  if (m < 0 || n < 1 || k < 1 || ldx < k || ldw < k || act < OS2_ACT_NONE || act > OS2_ACT_SILU) return OS2_ERR_INVALID_ARG;
  if (dtype != OS2_F32 && dtype != OS2_F16 && dtype != OS2_BF16) return OS2_ERR_INVALID_ARG;
  if (!W || !aligned(W, 2) || (m > 0 && (!X || !aligned(X, 2)))) return OS2_ERR_INVALID_ARG;
  if (dtype == OS2_F32) return OS2_ERR_UNSUPPORTED;
  if (m > kMaxRows || n > kMaxRows || k >= (1 << 24)) return OS2_ERR_UNSUPPORTED;
  return OS2_OK;
}

}  // namespace

extern "C" size_t os2_linear_workspace_size(int m, int n, int k, const void *X, int ldx, const void *W, int ldw) {
  if (m < 0 || n < 1 || k < 1 || ldx < k || ldw < k || m > kMaxRows || n > kMaxRows || k >= (1 << 24)) return 0;
  return forward_layout(m, n, k, X, ldx, W, ldw).total + cut_of(m, n, k).bytes;
}

extern "C" os2_status os2_linear(int m, int n, int k, int dtype, const void *X, int ldx, const void *W, int ldw, const void *bias,
                                 int bias_dtype, int activation, const void *R, int ldr, void *Y, int ldy, void *pre, int ldp,
                                 void *workspace, size_t workspace_bytes, void *stream) {
  const os2_status st = check(m, n, k, dtype, X, ldx, W, ldw, activation);
  if (st) return st;
  if (ldy < n || (R && ldr < n) || (pre && ldp < n)) return OS2_ERR_INVALID_ARG;
  if (bias && ((bias_dtype != OS2_F32 && bias_dtype != dtype) || !aligned(bias, bias_dtype == OS2_F32 ? 4 : 2)))
    return OS2_ERR_INVALID_ARG;
  if (m == 0) return OS2_OK;
  if (!Y || !aligned(Y, 2) || !aligned(R, 2) || !aligned(pre, 2) || pre == Y) return OS2_ERR_INVALID_ARG;
  const Forward f = forward_layout(m, n, k, X, ldx, W, ldw);
  const Cut cut = cut_of(m, n, k);
  if (!workspace || workspace_bytes < f.total + cut.bytes || !aligned(workspace, 256)) return OS2_ERR_WORKSPACE;
  LinearArgs a = {};
  a.status = os2_status_ptr();
  if (!a.status) return OS2_ERR_CUDA;
  a.m = m, a.n = n, a.k = k;
  a.bf16 = dtype == OS2_BF16;
  a.X = static_cast<const uint16_t *>(X), a.ldx = ldx;
  a.W = static_cast<const uint16_t *>(W), a.ldw = ldw;
  a.bias = bias, a.b32 = bias_dtype == OS2_F32;
  a.act = activation;
  a.R = static_cast<const uint16_t *>(R), a.ldr = ldr;
  a.Y = static_cast<uint16_t *>(Y), a.ldy = ldy;
  a.pre = static_cast<uint16_t *>(pre), a.ldp = ldp;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = prepare<true>(f, a, workspace, nullptr, 0, s);  // (copies, the same for both types)
  if (e != cudaSuccess) return OS2_ERR_CUDA;
  const bool rows = tma_rows(a.Y, a.ldy) && (!a.pre || tma_rows(a.pre, a.ldp)) && (!a.R || tma_rows(a.R, a.ldr));
  const Way way = way_of(m, n, k, a.act != OS2_ACT_NONE, a.pre, a.R, rows, cut);
  float *const acc = at<float>(workspace, f.total);
  if (way == kFew) e = launch_linear_few(a, false, s);
  else if (way == kTiles) e = a.bf16 ? forward<true>(a, s) : forward<false>(a, s);
  else e = a.bf16 ? in_parts<true>(a, cut.parts, acc, s) : in_parts<false>(a, cut.parts, acc, s);
  return e == cudaSuccess ? OS2_OK : OS2_ERR_CUDA;
}

extern "C" os2_status os2_linear_ways(int m, int n, int k, int activation, int pre, int residual, int rows16,
                                     os2_linear_ways_t *ways) {
  if (!ways || m < 1 || n < 1 || k < 1 || activation < OS2_ACT_NONE || activation > OS2_ACT_SILU) return OS2_ERR_INVALID_ARG;
  if (m > kMaxRows || n > kMaxRows || k >= (1 << 24)) return OS2_ERR_UNSUPPORTED;
  const bool act = activation != OS2_ACT_NONE;
  const Cut cut = cut_of(m, n, k);
  const Way way = way_of(m, n, k, act, pre, residual, rows16, cut);
  const Backward b = backward_layout(m, n, k, nullptr, k, nullptr, k, nullptr, n, activation);
  const LinearPlan y = linear_few_plan(m, n, k, act || pre), dx = linear_few_plan(m, k, n, false);
  *ways = {way, way == kFew ? y.nt : 256, way == kFew ? y.cluster : 2, way == kParts ? cut.parts : 1,
           b.few ? kFew : b.dx.parts > 1 ? kParts : kTiles, b.few ? dx.nt : 256, b.few ? dx.cluster : 2, b.dx.parts, b.dw.parts};
  return OS2_OK;
}

extern "C" size_t os2_linear_backward_workspace_size(int m, int n, int k, const void *X, int ldx, const void *W, int ldw,
                                                     const void *dY, int lddy, int activation) {
  if (m < 0 || n < 1 || k < 1 || ldx < k || ldw < k || lddy < n || m > kMaxRows || n > kMaxRows || k >= (1 << 24) ||
      activation < OS2_ACT_NONE || activation > OS2_ACT_SILU)
    return 0;
  if (m == 0) return 256;
  return backward_layout(m, n, k, X, ldx, W, ldw, dY, lddy, activation).total;
}

extern "C" os2_status os2_linear_backward(int m, int n, int k, int dtype, const void *X, int ldx, const void *W, int ldw,
                                          const void *dY, int lddy, const void *pre, int ldp, int activation, void *dX, int lddx,
                                          void *dW, int lddw, void *db, int db_dtype, void *workspace, size_t workspace_bytes,
                                          void *stream) {
  const os2_status st = check(m, n, k, dtype, X, ldx, W, ldw, activation);
  if (st) return st;
  const bool slope = activation != OS2_ACT_NONE;
  if (lddy < n || (slope && ldp < n) || (dX && lddx < k) || (dW && lddw < k)) return OS2_ERR_INVALID_ARG;
  if (db && ((db_dtype != OS2_F32 && db_dtype != dtype) || !aligned(db, db_dtype == OS2_F32 ? 4 : 2))) return OS2_ERR_INVALID_ARG;
  if (!aligned(dX, 2) || !aligned(dW, 2)) return OS2_ERR_INVALID_ARG;
  if (m > 0 && (!dY || !aligned(dY, 2) || (slope && (!pre || !aligned(pre, 2))))) return OS2_ERR_INVALID_ARG;
  if (!dX && !dW && !db) return OS2_OK;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (m == 0) {
    cudaError_t e = cudaSuccess;
    if (dW) e = cudaMemset2DAsync(dW, (size_t)lddw * 2, 0, (size_t)k * 2, (size_t)n, s);
    if (e == cudaSuccess && db) e = cudaMemsetAsync(db, 0, (size_t)n * (db_dtype == OS2_F32 ? 4 : 2), s);
    return e == cudaSuccess ? OS2_OK : OS2_ERR_CUDA;
  }
  const Backward b = backward_layout(m, n, k, X, ldx, W, ldw, dY, lddy, activation);
  if (!workspace || workspace_bytes < b.total || !aligned(workspace, 256)) return OS2_ERR_WORKSPACE;
  LinearArgs a = {};
  a.status = os2_status_ptr();
  if (!a.status) return OS2_ERR_CUDA;
  a.m = m, a.n = n, a.k = k;
  a.bf16 = dtype == OS2_BF16;
  a.X = static_cast<const uint16_t *>(X), a.ldx = ldx;
  a.W = static_cast<const uint16_t *>(W), a.ldw = ldw;
  a.act = activation;
  const uint16_t *g = static_cast<const uint16_t *>(dY), *z = static_cast<const uint16_t *>(pre);
  uint16_t *dx = static_cast<uint16_t *>(dX), *dw = static_cast<uint16_t *>(dW);
  const cudaError_t e = a.bf16 ? backward<true>(a, b, g, lddy, z, ldp, dx, lddx, dw, lddw, db, db_dtype, workspace, s)
                               : backward<false>(a, b, g, lddy, z, ldp, dx, lddx, dw, lddw, db, db_dtype, workspace, s);
  return e == cudaSuccess ? OS2_OK : OS2_ERR_CUDA;
}
