// Softmax cross entropy of a vocabulary head, z = H W^T, with its gradient,
// without the logits in memory.
//
//   forward   lse_i = log sum_v exp z_iv,  loss_i = lse_i - z_i,y(i)
//   backward  d_iv = g_i (exp(z_iv - lse_i) - [v = y_i]),  dH = D W,  dW = D^T H
//
// Rows whose label is the ignored one are taken out first: k_xent_prep packs
// the rows that count into the workspace (their number stays on the device),
// so they cost no products, and what they hold (Inf, NaN) reaches nothing.
// Forward: one product (mm2.cuh) whose epilogue keeps each row's running
// maximum and sum over 128 columns and writes that pair; a second kernel joins
// a row's pairs in their order.  Backward, for each piece of the vocabulary:
// the logits' product again, whose epilogue writes D in the operands' type,
// then D W (added in FP32 over the pieces) and D^T H, which take W, D and H as
// they lie (MN-major operands: nothing is transposed in memory).
// The tensor cores bound all three products for more than some 300 rows (2 n
// flop a byte of W), the weights' bytes below that.  Up to 16 rows the forward pass
// is a stream of W (k_xent_few.cu).
// Measured: the four products of 2048 rows, k 2048, v 32768 take 149, 150, 154 and
// 152 us, 1.79 to 1.84 PFLOP/s (0.93 to 0.96 of cuBLAS's burst); forward and gradient of
// 4096 rows, k 4096, v 65536 4.9 to 5.0 ms (8.8 TFLOP, 1.75 to 1.79 PFLOP/s), of 256 rows,
// k 512, v 8192 43 us: eight launches that wait for one another.
#include "xent.cuh"

using namespace os2mm;
using namespace os2xent;

namespace {

// The logits' gradients D are held divided by the largest |g| of the rows and times a
// power of two, so that |d| <= 2^14 in FP16 and 2^40 in BF16: |g_i / g_max| p_iv keeps its
// full precision down to 2^-28 and 2^-166 and vanishes below 2^-38 and 2^-173.  dW adds
// rows up, and what vanishes there is that small beside the largest row's part.  A row of
// dH is its own g_i times a sum, however small g_i: where the rows' |g| are further
// apart than 2^6, D in FP16 is written once more for dH, each row divided by its
// own |g_i|, and dH's rows are scaled back one by one (the whole gradient of 2048 rows, k
// 2048, v 32768 then takes 556 us instead of 491).  Up to 2^6 apart, a probability keeps
// its full precision down to 2^-22, the mean one of the largest vocabulary.
constexpr int kGradExp16 = 14, kGradExpB = 40;
constexpr float kSpread = 0x1p-6f;

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if (BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return reinterpret_cast<const uint32_t &>(v);
  }
  const __half2 v = __floats2half2_rn(a, b);
  return reinterpret_cast<const uint32_t &>(v);
}
template <bool BF16>
__device__ __forceinline__ uint16_t pack1(float a) {
  return (uint16_t)(pack2<BF16>(a, 0.f) & 0xFFFFu);
}

// ------------------------------------------------------------ rows that count
struct Prep {
  int n, k, v;
  const uint16_t *H;
  long ldh;
  const long long *labels;
  long long ignore;
  int rows_cta;          // rows of H a CTA takes
  // packed
  int *count;            // rows that count
  int *rowmap, *label;   // [n]
  uint16_t *Hc;          // [npad][kp]
  long kp, npad;
  // forward
  float *loss, *lse;     // zeroed for the others
  // backward
  const float *lse_in, *grad;
  float *lse_c, *grad_c; // [n]
  float *scale;          // {1 / max |g|, 2^-E max |g|}, g finite
  int *spread;           // whether dH has a D of its own (FP16)
  bool f16;
  uint16_t *dH;          // zeroed for the others (may be null)
  long lddh;
  int *status;
};

__device__ __forceinline__ bool counts(long long y, const Prep &p) {
  return y != p.ignore && y >= 0 && y < p.v;
}

// Each CTA counts the labels before its rows for itself (n labels from L2; a
// few microseconds at most beside a product over the rows), so packing takes
// one launch: 5 us for 256 rows of 512, latency; 25 us for 8192 of 4096 (5.3 TB/s).
constexpr int kPrepThreads = 256;
__global__ void __launch_bounds__(kPrepThreads) k_xent_prep(const Prep p) {
  __shared__ int s_sum[2];
  __shared__ float s_max[kPrepThreads / 32], s_min[kPrepThreads / 32];
  __shared__ int s_pos[kPrepThreads], s_warp[kPrepThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r0 = blockIdx.x * p.rows_cta, r1 = min(p.n, r0 + p.rows_cta);
  start_call();
  if (tid < 2) s_sum[tid] = 0;
  __syncthreads();
  int before = 0, total = 0;
  float gmax = 0.f, gmin = INFINITY;  // of the finite |g|, the least but 0
  for (int i = tid; i < p.n; i += kPrepThreads) {
    const bool c = counts(p.labels[i], p);
    total += c;
    before += c && i < r0;
    if (p.grad && c && blockIdx.x == 0) {
      const float g = fabsf(p.grad[i]);
      if (g < INFINITY) gmax = fmaxf(gmax, g);
      if (g > 0.f) gmin = fminf(gmin, g);
    }
  }
  before = __reduce_add_sync(0xffffffffu, before);
  total = __reduce_add_sync(0xffffffffu, total);
  if (lane == 0) {
    atomicAdd(&s_sum[0], before);
    atomicAdd(&s_sum[1], total);
  }
  if (p.grad && blockIdx.x == 0) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      gmax = fmaxf(gmax, __shfl_xor_sync(0xffffffffu, gmax, o));
      gmin = fminf(gmin, __shfl_xor_sync(0xffffffffu, gmin, o));
    }
    if (lane == 0) s_max[warp] = gmax, s_min[warp] = gmin;
  }
  __syncthreads();
  int base = s_sum[0];
  const int nv = s_sum[1];
  if (blockIdx.x == 0 && tid == 0) {
    *p.count = nv;
    if (p.grad) {
      // The logits' gradients are held divided by the largest finite |g| (a row whose g is
      // not finite has no finite gradient, and takes nothing from the others) and times 2^E
      // (kGradExp).  Where all g are equal, as a mean's are, the entry of the label,
      // the largest of its row, then lies just below a power of two, where rounding
      // is finest: dH and dW are 1.2 times as far off as by their own rounding
      // alone, against 1.7 times for a g whose leading digits are just above one.
      float g = 0.f, least = INFINITY;
      for (int w = 0; w < kPrepThreads / 32; w++) {
        g = fmaxf(g, s_max[w]);
        least = fminf(least, s_min[w]);
      }
      *p.spread = p.f16 && least < g * kSpread;
      if (!(g > 1e-30f)) g = 1.f;
      p.scale[0] = 1.f / g;
      p.scale[1] = g * exp2f((float)-(p.f16 ? kGradExp16 : kGradExpB));
    }
  }
  const bool vec = (p.ldh % 8 == 0) && (reinterpret_cast<uintptr_t>(p.H) % 16 == 0);
  for (int c0 = r0; c0 < r1; c0 += kPrepThreads) {
    const int i = c0 + tid;
    const long long y = i < r1 ? p.labels[i] : p.ignore;
    const bool c = i < r1 && counts(y, p);
    if (i < r1 && !c && y != p.ignore) set_status(p.status, OS2_ERR_RANGE);
    const unsigned b = __ballot_sync(0xffffffffu, c);
    if (lane == 0) s_warp[warp] = __popc(b);
    __syncthreads();
    int pos = base + __popc(b & ((1u << lane) - 1));
    int all = 0;
    for (int w = 0; w < kPrepThreads / 32; w++) {
      pos += w < warp ? s_warp[w] : 0;
      all += s_warp[w];
    }
    s_pos[tid] = c ? pos : -1;
    if (c && OS2_DBG_GUARD(pos >= 0 && pos < p.n, p.status)) {
      p.rowmap[pos] = i;
      p.label[pos] = (int)y;
      if (p.grad) {
        p.lse_c[pos] = p.lse_in[i];
        p.grad_c[pos] = p.grad[i];
      }
    } else if (i < r1 && p.loss) {
      p.loss[i] = 0.f;
      p.lse[i] = 0.f;
    }
    __syncthreads();
    const int rows = min(kPrepThreads, r1 - c0);
    if (vec) {
      // 16-byte pieces of all rows over all threads, four in flight
      const int per = p.k / 8;
      const long total = (long)rows * per;
      for (long i0 = tid; i0 < total; i0 += 4 * kPrepThreads) {
        uint4 v[4];
        long to[4];
#pragma unroll
        for (int u = 0; u < 4; u++) {
          const long i = i0 + u * kPrepThreads;
          to[u] = -1;
          if (i < total) {
            const int r = (int)(i / per), h = (int)(i - (long)r * per) * 8, at = s_pos[r];
            if (at >= 0 && OS2_DBG_GUARD(at < p.npad && p.k <= p.kp, p.status)) {
              to[u] = (long)at * p.kp + h;
              v[u] = __ldg(reinterpret_cast<const uint4 *>(p.H + (size_t)(c0 + r) * p.ldh + h));
            }
          }
        }
#pragma unroll
        for (int u = 0; u < 4; u++)
          if (to[u] >= 0) *reinterpret_cast<uint4 *>(p.Hc + to[u]) = v[u];
      }
    }
    const int h0 = vec ? p.k / 8 * 8 : 0;
    // the rest element by element, a warp a row, or all threads where rows are few (40 rows of
    // 2999, one a CTA: 7.5 us against 17 with a warp)
    const int team = rows < kPrepThreads / 32 ? kPrepThreads : 32, me = tid % team;
    for (int r = tid / team; r < rows; r += kPrepThreads / team) {
      const int at = s_pos[r];
      if (at >= 0 && OS2_DBG_GUARD(at < p.npad && p.k <= p.kp, p.status)) {
        const uint16_t *src = p.H + (size_t)(c0 + r) * p.ldh;
        uint16_t *dst = p.Hc + (size_t)at * p.kp;
#pragma unroll 4
        for (int h = h0 + me; h < p.k; h += team) dst[h] = __ldg(src + h);
      } else if (at < 0 && p.dH) {
        uint16_t *dst = p.dH + (size_t)(c0 + r) * p.lddh;
        for (int h = me; h < p.k; h += team) dst[h] = 0;
      }
    }
    base += all;
    __syncthreads();
  }
  // the last stage's rows past the count take part in D^T H: zeros
  if (!p.grad) return;
  const int end = (int)min((long)(nv + kStageK - 1) / kStageK * kStageK, p.npad);
  for (int r = nv + blockIdx.x * (kPrepThreads / 32) + warp; r < end;
       r += gridDim.x * (kPrepThreads / 32))
    for (long h = lane * 8; h < p.kp; h += 256)
      *reinterpret_cast<uint4 *>(p.Hc + (size_t)r * p.kp + h) = make_uint4(0, 0, 0, 0);
}

// W's rows at a pitch and base that TMA takes (only where W's own are not): 16
// bytes a thread, read as the words that straddle them.  50021 x 1001: 36 us, 5.7 TB/s
// read and written, beside 41 of the product over 333 rows.
__global__ void __launch_bounds__(256)
    k_repack(const uint16_t *src, long ld, uint16_t *dst, long pitch, int rows, int k) {
  next_may_start();
  wait_for_previous();
  const long per = pitch / 8, total = per * rows;
  for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < total; i += (long)gridDim.x * 256) {
    const long r = i / per;
    const int h = (int)(i - r * per) * 8;
    if (h >= k) continue;
    const uint16_t *p = src + r * ld + h;
    uint32_t w[4];
    if (h >= 2 && h + 10 <= k) {
      const int o = (int)(reinterpret_cast<uintptr_t>(p) & 3);  // 0 or 2
      const uint32_t *q = reinterpret_cast<const uint32_t *>(reinterpret_cast<const char *>(p) - o);
      uint32_t x[5];
#pragma unroll
      for (int e = 0; e < 5; e++) x[e] = __ldg(q + e);
#pragma unroll
      for (int e = 0; e < 4; e++) w[e] = __funnelshift_r(x[e], x[e + 1], 8 * o);
    } else {
#pragma unroll
      for (int e = 0; e < 4; e++) w[e] = 0;
#pragma unroll
      for (int e = 0; e < 8; e++)
        if (h + e < k) w[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
    }
    *reinterpret_cast<uint4 *>(dst + r * pitch + h) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// ------------------------------------------------------------ epilogues
// Forward: maximum (times log2 e) and sum of exponentials of 128 columns.
// CHUNKED (k > 1024): the tensor cores' sums, which lose up to 2^-23 a step, are
// added up in registers every 1024 terms: lse and loss are 4e-7 off at any k,
// instead of 1.6e-6 at 4096 and 3.3e-6 at 8192, for no time (the epilogue runs
// beside the next chunk's MMAs).  Below, too, the product bounds: 333 x 50021 x 1000 takes 48.1
// us with its launches, 46.6 with a quarter of the epilogue.
template <bool CHUNKED>
struct StatsEpi {
  const int *label;
  float *zlabel;
  float2 *part;   // [rows][parts]
  int parts, v;
  float z[CHUNKED ? 8 : 1][16];

  // N columns' logits x, `left` of which exist; y: the label's place among them
  template <int N>
  __device__ __forceinline__ void group(const float (&x)[N], int left, int y, int row, float &top,
                                        float &sum) {
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; i++) mx = fmaxf(mx, i < left ? x[i] : -INFINITY);
    const float t = fmaxf(top, mx * kLog2e);
    // a row of -inf so far: exponents against 0 (every term is 0)
    const float t0 = t == -INFINITY ? 0.f : t;
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      s0 += i < left ? ex2(fmaf(x[i], kLog2e, -t0)) : 0.f;
      s1 += i + 1 < left ? ex2(fmaf(x[i + 1], kLog2e, -t0)) : 0.f;
    }
    sum = sum * ex2(top - t0) + (s0 + s1);
    top = t;
    if ((unsigned)y < (unsigned)N) {
      float zy = 0.f;
#pragma unroll
      for (int i = 0; i < N; i++)
        if (i == y) zy = x[i];
      zlabel[row] = zy;
    }
  }

  __device__ __forceinline__ void unit(uint32_t taddr, int row, int col0, int, bool first,
                                       bool last, int m, const CUtensorMap *, uint8_t *,
                                       int *status) {
    if (row - (int)(threadIdx.x & 31) >= m) return;  // no row of this warp
    const int y = row < m ? label[row] - col0 : -1;
    float top = -INFINITY, sum = 0.f;
    if (CHUNKED) {
#pragma unroll
      for (int g = 0; g < 8; g++) {
        uint32_t r[16];
        __syncwarp();
        tmem_ld16(taddr + g * 16, r);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; i++)
          z[g][i] = first ? __uint_as_float(r[i]) : z[g][i] + __uint_as_float(r[i]);
      }
      if (!last) return;
#pragma unroll
      for (int g = 0; g < 8; g++)
        if (v > col0 + g * 16) group<16>(z[g], v - (col0 + g * 16), y - g * 16, row, top, sum);
    } else {
#pragma unroll 1
      for (int g = 0; g < 4; g++) {
        const int left = v - (col0 + g * 32);  // columns of this group that exist
        if (left <= 0) break;
        uint32_t r[32];
        __syncwarp();
        tmem_ld32(taddr + g * 32, r);
        tmem_wait_ld();
        float x[32];
#pragma unroll
        for (int i = 0; i < 32; i++) x[i] = __uint_as_float(r[i]);
        group<32>(x, left, y - g * 32, row, top, sum);
      }
    }
    if (row < m && OS2_DBG_GUARD((col0 >> 7) < parts, status))
      part[(size_t)row * parts + (col0 >> 7)] = make_float2(top, sum);
  }
  __device__ __forceinline__ void finish() {}
};

// A warp's blocks of 32 rows of 64 bytes (16 x 4 bytes a lane, its row) leave by TMA to
// (col, row0, layer), stored or added.  Two blocks of the scratch memory take turns over
// all that the warp sends, from tile to tile too: a tile may end after an odd number, and a
// turn that began anew there would write the block whose copy is the one still allowed to be
// reading.
struct BlockSender {
  int turn = 0;

  __device__ __forceinline__ void send(const CUtensorMap *map, uint8_t *scratch,
                                       const uint4 (&v)[4], int col, int row0, int layer,
                                       bool add) {
    const int lane = threadIdx.x & 31;
    uint8_t *block = scratch + turn * 2048;
    turn ^= 1;
    if (lane == 0) bulk_wait_read<1>();  // the block before the last has left
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 4; q++)
      *reinterpret_cast<uint4 *>(block + lane * 64 + ((q ^ (lane >> 1 & 3)) << 4)) = v[q];
    fence_async_smem();
    __syncwarp();
    if (lane == 0) {
      if (add)
        tma_add_3d(map, block, col, row0, layer);
      else
        tma_store_3d(map, block, col, row0, layer);
      bulk_commit();
    }
  }
  __device__ __forceinline__ void finish() {
    if ((threadIdx.x & 31) == 0) bulk_wait_all();
    __syncwarp();
  }
};

// Backward: D of one piece (columns v0 .. v0 + v) in the operands' type.  Its
// rounding is that of one operand of a product whose sums are FP32, as H's and
// W's own roundings are.  Rows and columns past the ends are zeros: they are
// terms of the next products.  Blocks leave by TMA: with lanes that stored their own rows,
// 16 bytes of 32 rows at a time, 2048 x 32768 x 2048 took 162 us, now 150 (1.83 PFLOP/s).
template <bool BF16>
struct GradEpi {
  const int *label;
  const float *lse, *grad, *scale;
  const int *spread;    // or null
  int v0, v;
  BlockSender sender = {};

  __device__ __forceinline__ void unit(uint32_t taddr, int row, int col0, int, bool, bool, int m,
                                       const CUtensorMap *mapD, uint8_t *scratch, int *) {
    const int row0 = row - (int)(threadIdx.x & 31);
    // no row of this warp: zeros, as far as the last stage of D^T H reads
    if (row0 >= (m + kStageK - 1) / kStageK * kStageK) return;
    const bool in = row < m;
    const int y = in ? label[row] - v0 - col0 : -1;
    // 2^E p = 2^(z log2 e - lse log2 e + E), so that p's own range does not cut it
    constexpr int E = BF16 ? kGradExpB : kGradExp16;
    constexpr float c = (float)(1ull << E);
    const float l = in ? fmaf(lse[row], kLog2e, -(float)E) : 0.f;
    const float gr = in ? grad[row] * scale[0] : 0.f;
    const bool twice = !BF16 && spread && *spread;  // (FP16) dH's own D, the second layer
    const float sign = in ? copysignf(1.f, grad[row]) : 0.f;
#pragma unroll 1
    for (int g = 0; g < 4; g++) {
      uint32_t r[32];
      __syncwarp();
      tmem_ld32(taddr + g * 32, r);
      tmem_wait_ld();
      const int left = v - (col0 + g * 32), yg = y - g * 32;
      float x[32];
#pragma unroll
      for (int i = 0; i < 32; i++) x[i] = ex2(fmaf(__uint_as_float(r[i]), kLog2e, -l));
      if ((unsigned)yg < 32u) {
#pragma unroll
        for (int i = 0; i < 32; i++)
          if (i == yg) x[i] -= c;
      }
      auto layer = [&](int l, float f) {
        uint4 o[4];
#pragma unroll
        for (int q = 0; q < 4; q++) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; i++) {
            const int a = 8 * q + 2 * i;
            w[i] = pack2<BF16>((in && a < left) ? x[a] * f : 0.f,
                               (in && a + 1 < left) ? x[a + 1] * f : 0.f);
          }
          o[q] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        sender.send(mapD, scratch, o, col0 + g * 32, row0, l, false);
      };
      layer(0, gr);
      if (twice) layer(1, sign);
    }
  }
  __device__ __forceinline__ void finish() { sender.finish(); }
};

// What a row of dH is scaled back by; spread may be null.
__device__ __forceinline__ float dh_scale(const int *spread, const float *grad, const float *scale,
                                          int row) {
  constexpr float own = 1.f / (1 << kGradExp16);
  return spread && *spread ? fabsf(grad[row]) * own : scale[1];
}

// dW, and dH where it comes out of one product: scaled back, rounded once, to the
// row that a packed row came from.  Written straight from a lane's own row, 16 bytes
// of 32 rows at a time, dW of 32000 x 2048 from 8 rows took 55 us, 719 with rows that
// are not aligned.  So the rows go through shared memory: dW's 32 x 32 blocks leave
// by TMA (aligned rows), two of them on their way while the next is made; else
// eight rows' 64 bytes an instruction, or one row's where rows are not aligned.  Now 8
// rows' dW takes 69 us with the logits' product and all launches, 219 not aligned;
// 2048 x 32768 x 2048 152 us (1.81 PFLOP/s).
template <bool BF16, bool TMA>
struct StoreEpi {
  uint16_t *out;
  long ld;
  const int *rowmap;    // or null
  const float *scale;
  const int *spread;    // dH's (FP16) or null
  const float *grad;
  int rows, n;          // of `out`
  bool vec;             // rows of `out` are 16-byte aligned
  BlockSender sender = {};

  __device__ __forceinline__ void unit(uint32_t taddr, int row, int col0, int, bool, bool, int m,
                                       const CUtensorMap *mapD, uint8_t *scratch, int *status) {
    const int lane = threadIdx.x & 31, row0 = row - lane;
    const float s = row < m ? dh_scale(spread, grad, scale, row) : 0.f;
    int mine = row < m ? (rowmap ? rowmap[row] : row) : -1;  // where this lane's row goes
    if (!OS2_DBG_GUARD(mine < rows && n <= ld, status)) mine = -1;
#pragma unroll 1
    for (int g = 0; g < 4; g++) {
      const int left = n - (col0 + g * 32);
      if (left <= 0 || row0 >= m) break;  // the whole warp
      uint32_t r[32];
      __syncwarp();
      tmem_ld32(taddr + g * 32, r);
      tmem_wait_ld();
      uint4 v[4];
#pragma unroll
      for (int q = 0; q < 4; q++) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; i++)
          w[i] = pack2<BF16>(__uint_as_float(r[8 * q + 2 * i]) * s,
                             __uint_as_float(r[8 * q + 2 * i + 1]) * s);
        v[q] = make_uint4(w[0], w[1], w[2], w[3]);
      }
      if constexpr (TMA) {
        // (rows from m on are cut off by the map)
        sender.send(mapD, scratch, v, col0 + g * 32, row0, 0, false);
      } else {
#pragma unroll
        for (int q = 0; q < 4; q++) *reinterpret_cast<uint4 *>(scratch + lane * 80 + q * 16) = v[q];
        __syncwarp();
        uint16_t *dst = out + col0 + g * 32;
        if (left >= 32 && vec) {
#pragma unroll
          for (int i = 0; i < 4; i++) {
            const int rr = i * 8 + (lane >> 2), to = __shfl_sync(0xffffffffu, mine, rr);
            if (to >= 0)
              reinterpret_cast<uint4 *>(dst + (size_t)to * ld)[lane & 3] =
                  *reinterpret_cast<const uint4 *>(scratch + rr * 80 + (lane & 3) * 16);
          }
        } else {
#pragma unroll 8
          for (int rr = 0; rr < 32; rr++) {
            const int to = __shfl_sync(0xffffffffu, mine, rr);
            if (to >= 0 && lane < left)
              dst[(size_t)to * ld + lane] =
                  *reinterpret_cast<const uint16_t *>(scratch + rr * 80 + lane * 2);
          }
        }
      }
    }
  }
  __device__ __forceinline__ void finish() {
    if (TMA) sender.finish();
  }
};

// dH out of several products (pieces of the vocabulary, parts of one): FP32 sums,
// one array for each part, written by the first piece and added to by each further
// one, in their order.  Like dW's, the blocks leave through shared memory by TMA, which
// also adds: 13 parts of 256 x 512 over 8192 terms took 14.9 us with lanes that wrote
// their own rows, now 11.5.
struct SumEpi {
  bool add;
  BlockSender sender = {};

  __device__ __forceinline__ void unit(uint32_t taddr, int row, int col0, int split, bool, bool,
                                       int m, const CUtensorMap *mapD, uint8_t *scratch, int *) {
    const int row0 = row - (int)(threadIdx.x & 31);
    if (row0 >= m) return;  // no row of this warp (rows past m within it: sums that nothing reads)
#pragma unroll 1
    for (int g = 0; g < 8; g++) {
      uint32_t r[16];
      __syncwarp();
      tmem_ld16(taddr + g * 16, r);
      tmem_wait_ld();
      const uint4 v[4] = {make_uint4(r[0], r[1], r[2], r[3]), make_uint4(r[4], r[5], r[6], r[7]),
                          make_uint4(r[8], r[9], r[10], r[11]),
                          make_uint4(r[12], r[13], r[14], r[15])};
      sender.send(mapD, scratch, v, col0 + g * 16, row0, split, add);
    }
  }
  __device__ __forceinline__ void finish() { sender.finish(); }
};

// dH from those sums, the parts in their order: four columns a thread, eight parts
// on their way at once.
// (256 x 512 from 13 parts: 7 us alone, latency.)
template <bool BF16>
__global__ void __launch_bounds__(256)
    k_dh_join(const int *count, const int *rowmap, const float *scale, const int *spread,
              const float *grad, const float *acc, int splits, long rows, long pitch, int k,
              uint16_t *out, long ld, bool vec) {
  next_may_start();
  wait_for_previous();
  const int per = (k + 3) / 4;
  const long total = (long)per * *count;
  for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < total; i += (long)gridDim.x * 256) {
    const long row = i / per;
    const int h = (int)(i - row * per) * 4;
    const float *a = acc + (size_t)row * pitch + h;
    const int to = rowmap[row];
    const float s = dh_scale(spread, grad, scale, (int)row);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p0 = 0; p0 < splits; p0 += 8) {
      float4 v[8];
#pragma unroll
      for (int u = 0; u < 8; u++)
        v[u] = p0 + u < splits
                   ? __ldg(reinterpret_cast<const float4 *>(a + (size_t)(p0 + u) * rows * pitch))
                   : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int u = 0; u < 8; u++) x.x += v[u].x, x.y += v[u].y, x.z += v[u].z, x.w += v[u].w;
    }
    uint16_t *dst = out + (size_t)to * ld + h;
    if (vec && h + 4 <= k) {
      *reinterpret_cast<uint2 *>(dst) =
          make_uint2(pack2<BF16>(x.x * s, x.y * s), pack2<BF16>(x.z * s, x.w * s));
    } else {
      const float e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int q = 0; q < 4; q++)
        if (h + q < k) dst[q] = pack1<BF16>(e[q] * s);
    }
  }
}

// ------------------------------------------------------------ joining a row
__global__ void __launch_bounds__(256)
    k_xent_join(const int *count, const int *rowmap, const float *zlabel, const float2 *part,
                int parts, float *loss, float *lse) {
  next_may_start();
  wait_for_previous();
  const int row = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= *count) return;
  const float2 *p = part + (size_t)row * parts;
  float top = -INFINITY, sum = 0.f;
  for (int i = lane; i < parts; i += 32) {
    const float2 v = p[i];
    add_exp(top, sum, v.x, v.y);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float x = __shfl_xor_sync(0xffffffffu, top, o), y = __shfl_xor_sync(0xffffffffu, sum, o);
    add_exp(top, sum, x, y);
  }
  if (lane == 0) {
    const float l = top * kLn2 + logf(sum);
    const int to = rowmap[row];
    lse[to] = l;
    loss[to] = l - zlabel[row];
  }
}

// ------------------------------------------------------------------- host --
bool tma_rows(const void *p, long ld) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0;
}

// D's piece of the vocabulary: at most 2^27 entries (256 MB a layer) of packed rows x
// columns, at least 2048 columns, pieces of equal size.  Larger pieces read and
// write dH's FP32 sums less often; D leaves L2 either way.
int piece_columns(long npad, int v) {
  const long most = std::max<long>((1L << 27) / npad / 256 * 256, 2048);
  const long pieces = (v + most - 1) / most;
  return (int)os2_round_up((size_t)((v + pieces - 1) / pieces), 256);
}

// Parts of dH's product over a piece of the vocabulary: as many as let all SM
// pairs work, by an estimate in microseconds (0.55 a stage; the sums written and
// read once at 5 TB/s).
int dh_splits(long npad, int k, int vc, int pieces) {
  const long tiles = npad / 256 * ((k + 255) / 256), pairs = std::max(os2_sm_count() / 2, 1);
  const int stages = (vc + kStageK - 1) / kStageK;
  const double bytes = (double)npad * os2_round_up((size_t)k, 256) * 8;
  int best = 1;
  double least = 1e30;
  for (int s = 1; s <= std::min(stages, 32); s++) {
    if (s > 1 && bytes / 2 * s > 268435456.) break;
    const double t = (double)((tiles * s + pairs - 1) / pairs) * ((stages + s - 1) / s) * 0.55 * pieces +
                     (s > 1 || pieces > 1 ? bytes * s / 5e6 + 3 : 0);
    if (t < least) {
      least = t;
      best = s;
    }
  }
  return best;
}

// D is there once, in FP16 twice (kSpread).
constexpr int d_layers(bool bf16) { return bf16 ? 1 : 2; }

struct Layout {
  long npad, kp;
  int parts, vc, pieces, splits;
  size_t count, rowmap, label, zlabel, part, Hc, Wc, lse_c, grad_c, scale, d, acc, total;
};

// layers: of D in the backward pass, 0 in the forward one.
Layout layout(int n, int k, int v, const void *W, int ldw, int layers) {
  Layout L = {};
  L.npad = (long)os2_round_up((size_t)n, 256);
  L.kp = (long)os2_round_up((size_t)k, 64);
  L.parts = n <= kXentFew ? os2_sm_count() : (v + kBN - 1) / kBN * 2;
  L.vc = piece_columns(std::max(L.npad, 256L), v);
  L.pieces = (v + L.vc - 1) / L.vc;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += os2_round_up(bytes, 256);
    return o;
  };
  L.count = take(4);
  L.rowmap = take((size_t)n * 4);
  L.label = take((size_t)n * 4);
  L.Hc = take((size_t)L.npad * L.kp * 2);
  if (!tma_rows(W, ldw)) L.Wc = take((size_t)v * L.kp * 2);
  if (layers) {
    L.lse_c = take((size_t)n * 4);
    L.grad_c = take((size_t)n * 4);
    L.scale = take(12);
    L.d = take((size_t)L.npad * L.vc * 2 * layers);
    L.splits = dh_splits(L.npad, k, std::min(L.vc, v), L.pieces);
    if (L.pieces * L.splits > 1)
      L.acc = take((size_t)L.splits * L.npad * os2_round_up((size_t)k, 256) * 4);
  } else {
    L.zlabel = take((size_t)n * 4);
    L.part = take((size_t)n * L.parts * 8);
  }
  L.total = at;
  return L;
}

template <class T>
T *at(void *ws, size_t off) {
  return reinterpret_cast<T *>(static_cast<char *>(ws) + off);
}

// Packs the rows, and W where TMA cannot take it as it lies (W, ldw: in, out).
cudaError_t prepare(const Layout &L, Prep &p, const uint16_t *&W, long &ldw, void *ws,
                    cudaStream_t s) {
  p.count = at<int>(ws, L.count);
  p.rowmap = at<int>(ws, L.rowmap);
  p.label = at<int>(ws, L.label);
  p.Hc = at<uint16_t>(ws, L.Hc);
  p.kp = L.kp;
  p.npad = L.npad;
  // few rows: one a CTA; at least 16 CTAs where the rows past the count are zeroed
  p.rows_cta = (p.n + 4 * os2_sm_count() - 1) / (4 * os2_sm_count());
  const int grid = std::max((p.n + p.rows_cta - 1) / p.rows_cta, p.grad ? 16 : 1);
  cudaError_t e = launch_after(k_xent_prep, grid, kPrepThreads, 0, s, p);
  if (e == cudaSuccess && !tma_rows(W, ldw)) {
    uint16_t *wc = at<uint16_t>(ws, L.Wc);
    e = launch_after(
        k_repack, (int)std::min<long>((L.kp / 8 * p.v + 255) / 256, 16L * os2_sm_count()), 256, 0, s,
        W, ldw, wc, L.kp, p.v, p.k);
    W = wc;
    ldw = L.kp;
  }
  return e;
}

template <bool BF16>
cudaError_t forward(Prep p, const uint16_t *W, long ldw, void *ws, const Layout &L,
                    cudaStream_t s) {
  cudaError_t e = prepare(L, p, W, ldw, ws, s);
  if (e != cudaSuccess) return e;
  float *zlabel = at<float>(ws, L.zlabel);
  float2 *part = at<float2>(ws, L.part);
  if (p.n <= kXentFew) {
    XentFewArgs a{p.n, p.k, p.v, BF16, p.Hc, L.kp, W, ldw, !L.Wc, p.count, p.label, zlabel, part,
                  p.status};
    int parts = 0;
    e = launch_xent_few(a, &parts, s);
    if (e != cudaSuccess) return e;
    return launch_after(k_xent_join, (p.n + 7) / 8, 256, 0, s, p.count, p.rowmap, zlabel, part, parts,
                        p.loss, p.lse);
  }
  CUtensorMap mh, mw;
  if (!make_map(&mh, p.Hc, BF16, p.k, p.n, L.kp, false) ||
      !make_map(&mw, W, BF16, p.k, p.v, ldw, false))
    return cudaErrorInvalidValue;
  auto product = [&](auto epi, int chunk) {
    epi.label = p.label;
    epi.zlabel = zlabel;
    epi.part = part;
    epi.parts = L.parts;
    epi.v = p.v;
    return launch_mm2<BF16, false, false>(mh, mw, Job{p.n, p.v, p.k, p.count, nullptr, chunk, 1},
                                          epi, p.status, s);
  };
  e = p.k > 1024 ? product(StatsEpi<true>{}, 1024 / kStageK) : product(StatsEpi<false>{}, INT_MAX);
  if (e != cudaSuccess) return e;
  return launch_after(k_xent_join, (p.n + 7) / 8, 256, 0, s, p.count, p.rowmap, zlabel, part, L.parts,
                      p.loss, p.lse);
}

template <bool BF16>
cudaError_t backward(Prep p, const uint16_t *W, long ldw, uint16_t *dW, long lddw, void *ws,
                     const Layout &L, cudaStream_t s) {
  p.lse_c = at<float>(ws, L.lse_c);
  p.grad_c = at<float>(ws, L.grad_c);
  p.scale = at<float>(ws, L.scale);
  p.spread = at<int>(ws, L.scale) + 2;
  cudaError_t e = prepare(L, p, W, ldw, ws, s);
  if (e != cudaSuccess) return e;
  uint16_t *d = at<uint16_t>(ws, L.d);
  float *acc = at<float>(ws, L.acc);
  const long acc_pitch = (long)os2_round_up((size_t)p.k, 256);
  const int layers = d_layers(BF16);
  const int *spread = !BF16 && p.dH ? p.spread : nullptr;
  CUtensorMap mh, mht, mw, mwt, md, mdt, mds, msum;
  const CUtensorMapDataType type =
      BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  if (!make_map(&mh, p.Hc, BF16, p.k, p.n, L.kp, false) ||
      !make_map(&mht, p.Hc, BF16, p.k, L.npad, L.kp, true) ||
      !make_map(&md, d, BF16, L.vc, L.npad, L.vc, false, kHalf, layers) ||
      !make_map(&mdt, d, BF16, L.vc, L.npad, L.vc, true) ||
      !make_store_map(&mds, d, type, 2, L.vc, L.npad, L.vc, layers))
    return cudaErrorInvalidValue;
  const bool sums = L.pieces * L.splits > 1;
  if (p.dH && sums &&
      !make_store_map(&msum, acc, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, acc_pitch, L.npad, acc_pitch,
                      L.splits))
    return cudaErrorInvalidValue;
  for (int i = 0; i < L.pieces; i++) {
    const int v0 = i * L.vc, vn = std::min(L.vc, p.v - v0);
    const uint16_t *Wi = W + (size_t)v0 * ldw;
    if (!make_map(&mw, Wi, BF16, p.k, vn, ldw, false) ||
        !make_map(&mwt, Wi, BF16, p.k, vn, ldw, true))
      return cudaErrorInvalidValue;
    const GradEpi<BF16> ge{p.label, p.lse_c, p.grad_c, p.scale, spread, v0, vn};
    e = launch_mm2<BF16, false, false>(mh, mw, Job{p.n, vn, p.k, p.count, nullptr, INT_MAX, 1}, ge,
                                       p.status, s, &mds);
    if (e != cudaSuccess) return e;
    if (p.dH) {
      // (a shorter last piece may have fewer stages than parts: those add nothing)
      const Job job{p.n, p.k, vn, p.count, nullptr, INT_MAX, L.splits, false, spread};
      e = sums
              ? launch_mm2<BF16, false, true>(md, mwt, job, SumEpi{i > 0}, p.status, s, &msum)
              : launch_mm2<BF16, false, true>(
                    md, mwt, job,
                    StoreEpi<BF16, false>{p.dH, p.lddh, p.rowmap, p.scale, spread, p.grad_c, p.n, p.k,
                                   tma_rows(p.dH, p.lddh)},
                    p.status, s);
      if (e != cudaSuccess) return e;
    }
    if (dW) {
      uint16_t *out = dW + (size_t)v0 * lddw;
      // (dW reads D as dH does, and nothing of dH)
      const Job job{vn, p.k, p.n, nullptr, p.count, INT_MAX, 1, p.dH != nullptr};
      if (tma_rows(dW, lddw)) {
        CUtensorMap mo;
        if (!make_store_map(&mo, out, type, 2, p.k, vn, lddw)) return cudaErrorInvalidValue;
        e = launch_mm2<BF16, true, true>(
            mdt, mht, job, StoreEpi<BF16, true>{out, lddw, nullptr, p.scale, nullptr, nullptr, vn, p.k, true}, p.status,
            s, &mo);
      } else {
        e = launch_mm2<BF16, true, true>(
            mdt, mht, job, StoreEpi<BF16, false>{out, lddw, nullptr, p.scale, nullptr, nullptr, vn, p.k, false},
            p.status, s);
      }
      if (e != cudaSuccess) return e;
    }
  }
  if (!p.dH || !sums) return cudaSuccess;
  const long groups = (p.k + 3L) / 4 * p.n;
  return launch_after(k_dh_join<BF16>, (int)std::min<long>((groups + 255) / 256, 16L * os2_sm_count()),
                      256, 0, s, p.count, p.rowmap, p.scale, spread, p.grad_c, acc, L.splits, L.npad,
                      acc_pitch, p.k, p.dH, p.lddh, tma_rows(p.dH, p.lddh));
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int kMaxRows = 1 << 22;

os2_status check(int n, int k, int v, int dtype, const void *H, int ldh, const void *W, int ldw,
                 const long long *labels) {
  if (n < 0 || k < 1 || v < 1 || ldh < k || ldw < k) return OS2_ERR_INVALID_ARG;
  if (dtype != OS2_F32 && dtype != OS2_F16 && dtype != OS2_BF16) return OS2_ERR_INVALID_ARG;
  if (!W || !aligned(W, 2)) return OS2_ERR_INVALID_ARG;
  if (n > 0 && (!H || !labels || !aligned(H, 2) || !aligned(labels, 8))) return OS2_ERR_INVALID_ARG;
  if (dtype == OS2_F32) return OS2_ERR_UNSUPPORTED;
  if (n > kMaxRows || v > kMaxRows || k >= (1 << 24)) return OS2_ERR_UNSUPPORTED;
  return OS2_OK;
}

}  // namespace

extern "C" size_t os2_xent_workspace_size(int n, int k, int v, const void *W, int ldw,
                                          int backward) {
  if (n < 0 || k < 1 || v < 1 || ldw < k || n > kMaxRows || v > kMaxRows || k >= (1 << 24))
    return 0;
  return layout(n, k, v, W, ldw, backward ? d_layers(backward == OS2_XENT_BACKWARD_BF16) : 0).total;
}

extern "C" os2_status os2_xent(int n, int k, int v, int dtype, const void *H, int ldh,
                               const void *W, int ldw, const long long *labels,
                               long long ignore_index, float *loss, float *lse, void *workspace,
                               size_t workspace_bytes, void *stream) {
  const os2_status st = check(n, k, v, dtype, H, ldh, W, ldw, labels);
  if (st) return st;
  if (n == 0) return OS2_OK;
  if (!loss || !lse || !aligned(loss, 4) || !aligned(lse, 4)) return OS2_ERR_INVALID_ARG;
  const Layout L = layout(n, k, v, W, ldw, 0);
  if (!workspace || workspace_bytes < L.total || !aligned(workspace, 256))
    return OS2_ERR_WORKSPACE;
  Prep p = {};
  p.status = os2_status_ptr();
  if (!p.status) return OS2_ERR_CUDA;
  p.n = n;
  p.k = k;
  p.v = v;
  p.H = static_cast<const uint16_t *>(H);
  p.ldh = ldh;
  p.labels = labels;
  p.ignore = ignore_index;
  p.loss = loss;
  p.lse = lse;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const uint16_t *w = static_cast<const uint16_t *>(W);
  const cudaError_t e = dtype == OS2_BF16 ? forward<true>(p, w, ldw, workspace, L, s)
                                          : forward<false>(p, w, ldw, workspace, L, s);
  return e == cudaSuccess ? OS2_OK : OS2_ERR_CUDA;
}

extern "C" os2_status os2_xent_backward(int n, int k, int v, int dtype, const void *H, int ldh,
                                        const void *W, int ldw, const long long *labels,
                                        long long ignore_index, const float *lse,
                                        const float *grad, void *dH, int lddh, void *dW, int lddw,
                                        void *workspace, size_t workspace_bytes, void *stream) {
  const os2_status st = check(n, k, v, dtype, H, ldh, W, ldw, labels);
  if (st) return st;
  if ((dH && (lddh < k || !aligned(dH, 2))) || (dW && (lddw < k || !aligned(dW, 2))))
    return OS2_ERR_INVALID_ARG;
  if (n > 0 && (!lse || !grad || !aligned(lse, 4) || !aligned(grad, 4))) return OS2_ERR_INVALID_ARG;
  if (!dH && !dW) return OS2_OK;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (n == 0) {
    if (!dW) return OS2_OK;
    return cudaMemset2DAsync(dW, (size_t)lddw * 2, 0, (size_t)k * 2, (size_t)v, s) == cudaSuccess
               ? OS2_OK
               : OS2_ERR_CUDA;
  }
  const Layout L = layout(n, k, v, W, ldw, d_layers(dtype == OS2_BF16));
  if (!workspace || workspace_bytes < L.total || !aligned(workspace, 256))
    return OS2_ERR_WORKSPACE;
  Prep p = {};
  p.status = os2_status_ptr();
  if (!p.status) return OS2_ERR_CUDA;
  p.n = n;
  p.k = k;
  p.v = v;
  p.H = static_cast<const uint16_t *>(H);
  p.ldh = ldh;
  p.labels = labels;
  p.ignore = ignore_index;
  p.lse_in = lse;
  p.grad = grad;
  p.f16 = dtype == OS2_F16;
  p.dH = static_cast<uint16_t *>(dH);
  p.lddh = lddh;
  const uint16_t *w = static_cast<const uint16_t *>(W);
  uint16_t *dw = static_cast<uint16_t *>(dW);
  const cudaError_t e = dtype == OS2_BF16
                            ? backward<true>(p, w, ldw, dw, lddw, workspace, L, s)
                            : backward<false>(p, w, ldw, dw, lddw, workspace, L, s);
  return e == cudaSuccess ? OS2_OK : OS2_ERR_CUDA;
}
