// pa_decode_q8: decode attention over the 8-bit cache (pa_q8.cuh), on the
// Blackwell tensor cores (tcgen05 + TMEM) with TMA loads.
//
//   out = sum_t p_t V_t / sum_t p_t,   p_t = 2^(s_t - m),
//   s_t = log2(e) * scale * q . K_t,   K_t = code * k_scale[block][head], V_t alike
//
// Bound: the cache's bytes, 2 per (token, KV head, dim), over HBM bandwidth.  So
// the codes go from HBM to shared memory to the tensor cores as they are, and
// everything 16- or 32-bit is brought to them:
//   - q is split into three e4m3 digits of four bits, q = s (d0 + d1/16 + d2/256)
//     with s the power of two that brings the row's largest |q| to (224, 448].  The last
//     digit's steps are 2^-17 s: all of bf16's 8 bits of an element from 2^-10 s on (2^-17
//     of the largest), all of fp16's 11 from 2^-7 s on (2^-14 of it); what is smaller is off
//     by 2^-18 s, under 2^-25 of the largest;
//   - the softmax weights, times the block's V scale, in units of their own largest
//     in the tile (of each head, a power of two), are split the same way: each is off by
//     2^-13.6 of itself (a single digit would be off by 2^-4), or 2^-25 of the largest
//     where that is more.  The unit follows weight and scale together: a block of a large
//     scale and no weight takes nothing from the others.
// Products of digits are exact and the sums are fp32.  K scales multiply the
// finished scores.
//
// The cache rows are the M side of both products, so that the G query heads of a
// KV head are columns and no row is wasted:
//   S^T[128 x N] = K_tile[128 x 128 B] . Qdigits^T          (one column per digit and head)
//   O^T[128 B x N] = V_tile^T . Pdigits^T
// A tile is 128 rows of 128 bytes: 128 tokens at head_dim 128.  At head_dim 64 a
// row is two tokens; the digits of q appear in two sets of columns, one with
// zeros over the second half of the row and one over the first, and of O^T only
// the quarter where token parity and column set agree is used.
//
// Work: the tiles of all (sequence, KV head, head chunk) items in a row, cut into
// windows of equal cost, one per CTA (two CTAs per SM); an item costs its tiles and
// something for its beginning and end (pa_q8_window.cuh).  An item that a window
// boundary cuts leaves partial (m, l, acc) in the workspace; the join kernel takes them
// together: M = max m, out = sum acc 2^(m - M) / sum l 2^(m - M).
//
// Roles (224 threads): warp 0 block ids and TMA; warp 1 TMEM and MMA issue; warp 2
// q digits; warps 3-6 softmax and sums, one thread per tile row, then one per
// row of O^T.  K and V tiles alternate in a ring of 16 KB stages.  Every wait is
// bounded; one that runs out sets an abort flag, copies and MMAs in flight are
// drained, TMEM is freed and PA_ERR_TIMEOUT is reported through status_dev.
//
// Measured (GB300, 8 KV heads of 128, graph of calls; of a plain copy's bandwidth):
//   8 sequences of 32,768..131,072, 8 query heads each: 204-207 us, 6.5 TB/s, 0.98
//   2,048 sequences of 16..1,024, 4 heads: 349-351 us, 6.33 TB/s, 0.95
//   64 sequences of 128..4,096, 4 heads: 50.3-50.9 us, 5.5 TB/s, 0.82; 8 heads 55.6,
//     16 heads 96, 4 heads of 64 36, 8 heads of 64 46
//   one sequence of 50,001, 5 heads: 27.4 us, 3.73 TB/s, 0.56
//   4 sequences of at most 64, 4 heads of 64: 4.8-5.5 us
// About 9 us of a call do not shrink with its bytes: lengths -> window -> block ids ->
// first tile 4 us, last tile and partials 2 us, join 2.7 us.  With 16 heads to a KV head
// (two chunks read the cache twice) and with head_dim 64 and 8 heads the softmax warps
// are the bound.
#include <math.h>
#include <math_constants.h>

#include <mutex>

#include "pa_common.cuh"
#include "pa_internal.h"
#include "pa_q8.cuh"
#include "pa_q8_window.cuh"
#include "pa_sm100.cuh"

namespace pa {
namespace {

using namespace sm100;

constexpr int kThreads = 224;
constexpr int kTileRows = 128;
constexpr int kStageBytes = kTileRows * 128;
constexpr int kMaxGrid = 320;                  // CTAs at most (two per SM)
constexpr uint64_t kLimitNs = 2000000000ull;
constexpr unsigned kAll = 0xFFFFFFFFu;

struct Q8Args {
  void* out;
  const void* q;
  const float* k_scale;
  const float* v_scale;
  const int32_t* tables;
  const int32_t* lens;
  int B, Hq, H, bs, bs_shift, max_blocks, num_blocks, max_seq_len;
  int chunks, hch;               // chunks of a KV head's query heads, heads per chunk
  int rows_total;                // 128-byte rows of a pool
  float scale_log2;
  int dtype;
  Window* info;                  // [grid]
  float* ws_m;                   // [2 grid, hch]
  float* ws_l;
  float* ws_acc;                 // [2 grid, hch, D]
  int32_t* status_dev;
};

// Columns of one digit set: three digits of GP heads for each token of a row.
template <int D, int GP>
struct Shape {
  static constexpr int kTpr = 128 / D;                         // tokens per row
  static constexpr int kTokens = kTileRows * kTpr;             // tokens per tile
  static constexpr int kUsed = 3 * GP * kTpr;
  static constexpr int kN = (kUsed + 15) / 16 * 16;
  // as many as let two CTAs fit an SM: 96 or 80 KB each are on their way
  static constexpr int kStages = kN <= 16 ? 6 : 5;
  static constexpr uint32_t kCols = 4 * kN <= 64 ? 64 : (4 * kN <= 128 ? 128 : 256);
  static constexpr int kOperand = kN * 128;                    // bytes of a digit operand
  static constexpr int kQOff = kStages * kStageBytes;
  static constexpr int kPOff = kQOff + 2 * kOperand;
  static constexpr int kTailOff = kPOff + 2 * kOperand;
};

// An item's cost is 4 for a tile and this for its beginning and end (sums over the
// rows, a new q, the output; measured: 0.2-0.5 us with four heads, 1.1 us with eight, of
// 1.25 us a tile).
template <int D, int GP>
constexpr int item_cost() {
  return GP * (128 / D) <= 2 ? 0 : (GP * (128 / D) <= 4 ? 1 : (GP * (128 / D) <= 5 ? 2 : 4));
}

template <int D, int GP>
struct Tail {
  uint64_t full[6], empty[6];
  uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], o_full[2], red_bar[2];
  uint64_t sum_bar, drain;
  float qscale[2][GP];
  uint32_t q[2][GP][D / 2];      // q as it is, of a segment and the one behind it
  float inv[4][GP];              // per warp: 1 / the weights' sums of a finished segment
  float red[2][4][2 * GP];       // per warp: heads' maxima of s, then of s + log2(V scale)
  struct alignas(8) {            // per warp: heads' running maxima of s
    float now[GP];
  } top[4];
  struct alignas(8) {            // per warp: heads' 2^(before - now), then the weights' units
    float by[2 * GP];
  } fold[4][2];
  float lred[2][4][GP];          // of a finished segment, per warp: weights' sums
  float mred[2][GP];             // ... and the maxima
  float half[2][D == 64 ? GP * 64 : 1];   // head_dim 64: the other parity's sums, by segment
  int2 sums[kThreads / 32];      // per warp: tiles, sequences that have any
  int start[4];                  // window's first sequence, item, tile; its length
  int64_t lin[2], final;         // its first tile and the next window's, of all; see Window
  uint32_t tmem;
  int abort_flag;
};

template <int D, int GP>
constexpr int smem_bytes() {
  return Shape<D, GP>::kTailOff + (int)sizeof(Tail<D, GP>) + 1024;   // + alignment slack
}

__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tma_rows(void* dst, const CUtensorMap* map, uint64_t* bar, int row,
                                         uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(0), "r"(row), "l"(policy)
      : "memory");
}

// The first C columns from t on of this warp's 32 lanes, rounded up to what is
// loaded at once; loads and wait are one statement, so nothing reads them early.
template <int C>
__device__ __forceinline__ void load_cols(uint32_t t, float* v);

template <>
__device__ __forceinline__ void load_cols<4>(uint32_t t, float* v) {
  uint32_t r[4];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(t)
      : "memory");
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r[i]);
}

template <>
__device__ __forceinline__ void load_cols<8>(uint32_t t, float* v) {
  uint32_t r[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
        "=r"(r[6]), "=r"(r[7])
      : "r"(t)
      : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

template <>
__device__ __forceinline__ void load_cols<16>(uint32_t t, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
        "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
        "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(t)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

template <>
__device__ __forceinline__ void load_cols<24>(uint32_t t, float* v) {
  uint32_t r[24];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%24];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%16, %17, %18, %19, %20, %21, %22, %23}, [%25];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
        "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
        "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
        "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23])
      : "r"(t), "r"(t + 16)
      : "memory");
#pragma unroll
  for (int i = 0; i < 24; ++i) v[i] = __uint_as_float(r[i]);
}

template <>
__device__ __forceinline__ void load_cols<32>(uint32_t t, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
        "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
        "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
        "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
        "=r"(r[30]), "=r"(r[31])
      : "r"(t)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

template <>
__device__ __forceinline__ void load_cols<48>(uint32_t t, float* v) {
  uint32_t r[48];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%48];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47}, [%49];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
        "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
        "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
        "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
        "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]),
        "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]),
        "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47])
      : "r"(t), "r"(t + 32)
      : "memory");
#pragma unroll
  for (int i = 0; i < 48; ++i) v[i] = __uint_as_float(r[i]);
}

// Columns loaded for n used ones.
constexpr int cols_for(int n) {
  return n <= 4 ? 4 : (n <= 8 ? 8 : (n <= 16 ? 16 : (n <= 24 ? 24 : (n <= 32 ? 32 : 48))));
}

__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// The three digits of x (|x| <= 448): x = d0 + d1 / 16 + d2 / 256.  With 2^e <= |x| < 2^(e+1)
// a digit of four bits leaves 2^(e-4) at most; times 16 that is 2^e, whose digit leaves
// 2^(e-5), times 16 again 2^(e-1), and the last one leaves 2^(e-6), 2^-14 |x| in all, or half
// a subnormal step, 2^-18.  For two values at once; digit i of the first in byte 0 of d[i].
__device__ __forceinline__ void digits2(float x, float y, uint32_t (&d)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    d[i] = e4m3x2(x, y);
    if (i < 2) {
      const float2 v = e4m3_widen2(d[i]);
      x = (x - v.x) * 16.f;
      y = (y - v.y) * 16.f;
    }
  }
}

__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// The same of the weights, the bulk of the softmax warps' work: what the first digit leaves
// is exact in fp32 and goes on as fp16, two values to an instruction (2^-16 |x| more).
__device__ __forceinline__ void digits2_short(uint64_t x, uint32_t (&d)[3]) {
  float x0, x1;
  f2_unpack(x, x0, x1);
  d[0] = e4m3x2(x0, x1);
  const float2 v = e4m3_widen2(d[0]);
  const uint64_t left = f2_mul(f2_sub(x, f2_pack(v.x, v.y)), f2_pack(16.f, 16.f));
  f2_unpack(left, x0, x1);
  const __half2 h = __floats2half2_rn(x0, x1);
  d[1] = __nv_cvt_halfraw2_to_fp8x2(__half2_raw(h), __NV_SATFINITE, __NV_E4M3);
  const __half2 w(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)d[1], __NV_E4M3));
  d[2] = __nv_cvt_halfraw2_to_fp8x2(
      __half2_raw(__hmul2(__hsub2(h, w), __half2half2(__float2half(16.f)))), __NV_SATFINITE,
      __NV_E4M3);
}

__device__ __forceinline__ float lg2_approx(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 1 / x of a power of two from 2^-126 to 2^126.
__device__ __forceinline__ float inverse_pow2(float x) {
  return __uint_as_float((254u << 23) - __float_as_uint(x));
}

// Byte `col` of row n of a K-major operand with 128-byte rows and 128-byte swizzle.
__device__ __forceinline__ int swizzled(int n, int col) {
  return n * 128 + (((col >> 4) ^ (n & 7)) << 4) + (col & 15);
}

__device__ __forceinline__ int clamp_len(const Q8Args& a, int b) {
  return max(0, min(a.lens[b], a.max_seq_len));
}

// Walks a window's tiles in order: sequences, then their items (KV head, then head
// chunk), then tiles.
template <int TOKENS>
struct Walk {
  int b, L, nt, h, chunk, j, left;

  __device__ __forceinline__ void next(const Q8Args& a) {
    --left;
    if (++j < nt) return;
    j = 0;
    if (++chunk < a.chunks) return;
    chunk = 0;
    if (++h < a.H) return;
    h = 0;
    do {
      ++b;
      L = b < a.B && left > 0 ? clamp_len(a, b) : 0;
      nt = (L + TOKENS - 1) / TOKENS;
    } while (nt == 0 && left > 0 && b < a.B);
    if (nt == 0) left = 0;
  }
};

template <int D, int GP>
__global__ void __launch_bounds__(kThreads, 2)
decode_q8_kernel(const __grid_constant__ CUtensorMap map_k,
                 const __grid_constant__ CUtensorMap map_v, const Q8Args a) {
  using S = Shape<D, GP>;
  constexpr int TPR = S::kTpr, TOKENS = S::kTokens, N = S::kN, R = S::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  Tail<D, GP>* tail = reinterpret_cast<Tail<D, GP>*>(smem + S::kTailOff);
  volatile int* abort_flag = &tail->abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int items = a.H * a.chunks, G = a.Hq / a.H;

  allow_next_grid();
  if (tid == 0) {
    for (int i = 0; i < R; ++i) {
      mbar_init(&tail->full[i], 1);
      mbar_init(&tail->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tail->q_full[i], 1);
      mbar_init(&tail->q_empty[i], 5);       // MMA + four softmax warps
      mbar_init(&tail->s_full[i], 1);
      mbar_init(&tail->p_full[i], 4);
      mbar_init(&tail->o_full[i], 1);
      mbar_init(&tail->red_bar[i], 4);
    }
    mbar_init(&tail->sum_bar, 4);
    mbar_init(&tail->drain, 1);
    tail->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
  }
  if (warp == 1) {
    tmem_alloc(&tail->tmem, S::kCols);
    tmem_relinquish();
  }
  // digit operands: columns that no head uses, and the halves that stay zero
  for (int i = tid; i < 4 * S::kOperand / 16; i += kThreads)
    reinterpret_cast<uint4*>(smem + S::kQOff)[i] = make_uint4(0, 0, 0, 0);
  fence_async_smem();
  wait_prior_grid();

  // this CTA's window: tiles and sequences that have any, up to each thread's first
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  int tiles = 0, seqs = 0;
  for (int b = b0; b < b1; ++b) {
    const int nt = (clamp_len(a, b) + TOKENS - 1) / TOKENS;
    tiles += nt;
    seqs += nt > 0;
  }
  int tiles_to = tiles, seqs_to = seqs;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(kAll, tiles_to, o), n = __shfl_up_sync(kAll, seqs_to, o);
    if (lane >= o) {
      tiles_to += t;
      seqs_to += n;
    }
  }
  if (lane == 31) tail->sums[warp] = make_int2(tiles_to, seqs_to);
  tiles_to -= tiles;
  seqs_to -= seqs;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  int all_tiles = 0, all_seqs = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const int2 sum = tail->sums[w];
    tiles_to += w < warp ? sum.x : 0;
    seqs_to += w < warp ? sum.y : 0;
    all_tiles += sum.x;
    all_seqs += sum.y;
  }
  const Cut cut = cut_of(all_tiles, all_seqs, items, (int)gridDim.x, item_cost<D, GP>());
  const Share share = {b0, b1, tiles, seqs, tiles_to, seqs_to};
  const bool in = (int64_t)blockIdx.x < cut.ctas;
  auto len_of = [&](int b) { return clamp_len(a, b); };
  if (in && cut.ctas == cut.work) {             // a tile each: the shortest way, latency counts
    TilePlace p;
    if (place_of_tile<TOKENS>(share, items, (int)blockIdx.x, len_of, &p)) {
      tail->start[0] = p.b;
      tail->start[1] = p.item;
      tail->start[2] = p.j;
      tail->start[3] = p.len;
      tail->lin[0] = p.lin;
      tail->lin[1] = p.lin + 1;
      tail->final = p.final;
    }
  } else if (in) {
#pragma unroll 1
    for (int end = 0; end < 2; ++end) {
      const Bound w = bound_of(cut, items, blockIdx.x + end);
      if (w.at == cut.total) {
        if (tid == 0) tail->lin[end] = cut.work;
        continue;
      }
      TilePlace p;
      if (!place_of_cost<TOKENS>(cut, share, a.B, items, w, end == 0, len_of, &p)) continue;
      tail->lin[end] = p.lin;
      if (end == 0) {
        tail->start[0] = p.b;
        tail->start[1] = p.item;
        tail->start[2] = p.j;
        tail->start[3] = p.len;
        tail->final = p.final;
      }
    }
  } else if (tid < 4) {
    tail->start[tid] = 0;
    tail->lin[tid & 1] = 0;
  }
  __syncthreads();
  Walk<TOKENS> walk;
  walk.b = tail->start[0];
  walk.h = tail->start[1] / a.chunks;
  walk.chunk = tail->start[1] - walk.h * a.chunks;
  walk.j = tail->start[2];
  walk.left = (int)(tail->lin[1] - tail->lin[0]);
  walk.L = tail->start[3];
  walk.nt = (walk.L + TOKENS - 1) / TOKENS;
  if (tid == 0)
    a.info[blockIdx.x] = Window{walk.b, tail->start[1], walk.j, walk.left, tail->final,
                                cut.total};
  const uint32_t tmem = tail->tmem;
  const uint32_t ring = smem_addr(smem), qb = smem_addr(smem + S::kQOff),
                 pb = smem_addr(smem + S::kPOff);
  bool ok = true;

  if (warp == 0) {
    // ------------------------------------------------------------ block ids, TMA --
    const uint64_t policy = policy_evict_first();
    const int per_tile = TOKENS >> a.bs_shift, block_rows = a.bs / TPR;
    int stage = 0, phase = 0, used = 0;
    // a lane's block of the tile that w stands at
    auto block_of = [&](const Walk<TOKENS>& w) -> int {
      if (w.left <= 0 || w.j * TOKENS + lane * a.bs >= w.L || lane >= per_tile) return -1;
      return a.tables[(int64_t)w.b * a.max_blocks + w.j * per_tile + lane];
    };
    int id = block_of(walk);
    while (walk.left > 0) {
      const int n = min(TOKENS, walk.L - walk.j * TOKENS);
      const int nb = (n + a.bs - 1) >> a.bs_shift;
      const int h = walk.h;
      int row = a.rows_total;                   // outside the pool: the copy reads zeros
      if (lane < nb) {
        if (id >= 0 && id < a.num_blocks) row = (id * a.H + h) * block_rows;
        else report(a.status_dev, PA_ERR_BAD_BLOCK_ID);
      }
      walk.next(a);
      id = block_of(walk);
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        if (lane == 0) {
          ok = mbar_wait(&tail->empty[stage], phase ^ 1, abort_flag, kLimitNs);
          if (ok) mbar_arrive_expect_tx(&tail->full[stage], (uint32_t)(nb * block_rows * 128));
        }
        ok = __shfl_sync(kAll, (int)ok, 0) != 0;
        if (!ok) break;
        if (lane < nb)
          tma_rows(smem + stage * kStageBytes + lane * block_rows * 128, kv ? &map_v : &map_k,
                   &tail->full[stage], row, policy);
        ++used;
        if (++stage == R) {
          stage = 0;
          phase ^= 1;
        }
      }
      if (!ok) break;
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      report(a.status_dev, PA_ERR_TIMEOUT);
    }
    if (*abort_flag && lane == 0) {             // copies in flight land before the CTA ends
      for (int i = max(0, used - R); i < used; ++i)
        mbar_wait_drain(&tail->full[i % R], (i / R) & 1, kLimitNs);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issue --
    // K . q of tile t, then V . p of tile t - 1: the softmax of a tile runs while the
    // tensor cores have the next tile's scores.
    constexpr uint32_t idesc_s = idesc_f16(0, 0, 0, kTileRows, N);    // e4m3, K-major x K-major
    constexpr uint32_t idesc_o = idesc_f16(0, 1, 0, 128, N);          // V MN-major
    if (lane == 0) {
      int t = 0, seg = 0;
      bool fresh = true;
      auto issue_pv = [&](int p) -> bool {
        const int u = 2 * p + 1, slot = p & 1;
        // the weights are there, and with them: S of tile p and O of tile p - 2 are read
        if (!mbar_wait(&tail->full[u % R], (u / R) & 1, abort_flag, kLimitNs) ||
            !mbar_wait(&tail->p_full[slot], (p >> 1) & 1, abort_flag, kLimitNs))
          return false;
        tc_fence_after();
        const uint32_t va = ring + (u % R) * kStageBytes, pa_ = pb + slot * S::kOperand;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_f8(tmem + (2 + slot) * N, smem_desc_sw128(va + k * 32 * 128, kStageBytes, 1024),
                 smem_desc_sw128(pa_ + k * 32, 16, 1024), idesc_o, k > 0);
        mma_commit(&tail->empty[u % R]);
        mma_commit(&tail->o_full[slot]);
        return true;
      };
      while (walk.left > 0) {
        const int slot = t & 1, qs = seg & 1, u = 2 * t;
        ok = (!fresh || mbar_wait(&tail->q_full[qs], (seg >> 1) & 1, abort_flag, kLimitNs)) &&
             mbar_wait(&tail->full[u % R], (u / R) & 1, abort_flag, kLimitNs);
        if (!ok) break;
        // head_dim 64, an odd end: the last row's second token is no token, and 0 times
        // whatever stands there has to be 0
        if (TPR == 2) {
          const int n = walk.L - walk.j * TOKENS;
          if (n < TOKENS && (n & 1)) {
            uint8_t* kt = smem + (u % R) * kStageBytes;
#pragma unroll
            for (int c = 64; c < 128; c += 16)
              *reinterpret_cast<uint4*>(kt + swizzled(n >> 1, c)) = make_uint4(0, 0, 0, 0);
            fence_async_smem();
          }
        }
        tc_fence_after();
        const uint32_t ka = ring + (u % R) * kStageBytes, qa = qb + qs * S::kOperand;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_f8(tmem + slot * N, smem_desc_sw128(ka + k * 32, 16, 1024),
                 smem_desc_sw128(qa + k * 32, 16, 1024), idesc_s, k > 0);
        mma_commit(&tail->empty[u % R]);
        mma_commit(&tail->s_full[slot]);
        fresh = walk.j + 1 == walk.nt || walk.left == 1;       // a segment ends here
        if (fresh) {
          mma_commit(&tail->q_empty[qs]);
          ++seg;
        }
        if (t > 0) ok = issue_pv(t - 1);
        if (!ok) break;
        ++t;
        walk.next(a);
      }
      if (ok && t > 0) ok = issue_pv(t - 1);
      if (!ok) {
        *abort_flag = 1;
        report(a.status_dev, PA_ERR_TIMEOUT);
      }
      // every MMA and its arrivals end before TMEM is freed and the CTA ends
      if (in) {
        mma_commit(&tail->drain);
        mbar_wait_drain(&tail->drain, 0, kLimitNs);
      }
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------------- q digits --
    // Once per segment and a loop over heads: the code is cold, so it is kept short.
    constexpr int W = D / 64;                   // 32-bit words of a lane and head
    auto fetch_q = [&](const Walk<TOKENS>& w, int buf) {   // asynchronous, a segment ahead
      const int g0 = w.chunk * a.hch, gn = w.left > 0 ? min(a.hch, G - g0) : 0;
      const uint32_t* q = reinterpret_cast<const uint32_t*>(a.q) +
                          ((int64_t)w.b * a.Hq + w.h * G + g0) * (D / 2) + lane * W;
#pragma unroll 1
      for (int g = 0; g < gn; ++g)
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(
                         smem_addr(&tail->q[buf][g][lane * W])),
                     "l"(q + g * (D / 2)), "n"(4 * W)
                     : "memory");
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int seg = 0;
    fetch_q(walk, 0);
    while (walk.left > 0) {
      const int slot = seg & 1;
      const int gn = min(a.hch, G - walk.chunk * a.hch);
      const int skip = min(walk.nt - walk.j, walk.left) - 1;   // to the segment's last tile
      walk.j += skip;
      walk.left -= skip;
      walk.next(a);
      fetch_q(walk, slot ^ 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncwarp();
      if (!__all_sync(kAll, mbar_wait(&tail->q_empty[slot], ((seg >> 1) & 1) ^ 1, abort_flag,
                                      kLimitNs))) {
        ok = false;
        break;
      }
      uint8_t* op = smem + S::kQOff + slot * S::kOperand;
#pragma unroll 4
      for (int g = 0; g < gn; ++g) {
        float2 x[W];
        float m = 0.f;
        bool bad = false;
#pragma unroll
        for (int e = 0; e < W; ++e) {
          const uint32_t w = tail->q[slot][g][lane * W + e];
          x[e] = a.dtype == PA_BFLOAT16 ? widen2<PA_BFLOAT16>(w) : widen2<PA_FLOAT16>(w);
          m = fmaxf(m, fmaxf(finite_mag(x[e].x), finite_mag(x[e].y)));
          bad |= !(fabsf(x[e].x) < CUDART_INF_F) || !(fabsf(x[e].y) < CUDART_INF_F);
        }
        const float s = scale_for(warp_max(m)), inv = 1.f / s;
        bad = __any_sync(kAll, bad);
        uint32_t d[W][3];
#pragma unroll
        for (int e = 0; e < W; ++e) digits2(x[e].x * inv, x[e].y * inv, d[e]);
#pragma unroll
        for (int v = 0; v < TPR; ++v)
#pragma unroll
          for (int i = 0; i < 3; ++i) {
            uint8_t* to = op + swizzled((v * 3 + i) * GP + g, v * D + lane * 2 * W);
            if (W == 2) *reinterpret_cast<uint32_t*>(to) = d[0][i] | (d[W - 1][i] << 16);
            else *reinterpret_cast<uint16_t*>(to) = (uint16_t)d[0][i];
          }
        // a row with an infinity or a NaN has no finite scores
        if (lane == 0) tail->qscale[slot][g] = bad ? CUDART_NAN_F : s * a.scale_log2;
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tail->q_full[slot]);
      ++seg;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    // lengths out of range are reported; empty sequences get zero rows
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
      const int L = a.lens[b];
      if ((L < 0 || L > a.max_seq_len) && lane == 0) report(a.status_dev, PA_ERR_BAD_BLOCK_ID);
      if (L <= 0 || a.max_seq_len == 0) {
        uint4* row = static_cast<uint4*>(a.out) + (int64_t)b * a.Hq * (D / 8);
        for (int i = lane; i < a.Hq * (D / 8); i += 32) row[i] = make_uint4(0, 0, 0, 0);
      }
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      report(a.status_dev, PA_ERR_TIMEOUT);
    }
  } else {
    // ------------------------------------------------------------ softmax and sums --
    // Iteration t: weights of tile t; sums of tile t - 1, whose product has had most of
    // an iteration's time; scores and maxima of tile t + 1.  So neither the exchange of
    // the maxima nor a product is waited for as soon as it is asked for.
    const int wq = warp & 3;                    // TMEM lane quarter of this warp
    const int r = wq * 32 + lane;               // tile row; then row of O^T
    const uint32_t lanes = (uint32_t)(wq * 32) << 16;
    const int par = r / D;                      // head_dim 64: the token parity of this O^T row
    auto wait_all = [&](uint64_t* bar, int parity) -> bool {
      return __all_sync(kAll, mbar_wait(bar, parity, abort_flag, kLimitNs));
    };
    // the scales of this row's block in the tile that w stands at
    auto scales_of = [&](const Walk<TOKENS>& w, float& ks, float& vs) {
      ks = vs = 0.f;
      const int tok = w.j * TOKENS + r * TPR;
      if (w.left <= 0 || tok >= w.L) return;
      const int id = a.tables[(int64_t)w.b * a.max_blocks + (tok >> a.bs_shift)];
      if (id < 0 || id >= a.num_blocks) return;
      const int64_t at = (int64_t)id * a.H + w.h;
      ks = a.k_scale[at];
      vs = a.v_scale[at];
    };
    // where this row's byte of operand row n goes, by n & 7
    uint8_t* put[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) put[c] = smem + S::kPOff + (((r >> 4) ^ c) << 4) + (r & 15);
    float x[TPR][GP];                           // scores of the tile ahead
    float l[GP], acc[GP];
    float m_lane = -CUDART_INF_F;               // head `lane`: the running maximum
    int seg = 0;                                // segment of tile t

    // scores of tile u (n tokens left, segment sg) and their maxima, posted for all warps
    auto score_tile = [&](int u, int n, int sg, bool first, float ks, float vs) -> bool {
      const int slot = u & 1, qs = sg & 1;
      if (first && !wait_all(&tail->q_full[qs], (sg >> 1) & 1)) return false;
      if (!wait_all(&tail->s_full[slot], (u >> 1) & 1)) return false;
      tc_fence_after();
      float s[cols_for(S::kUsed)];
      load_cols<cols_for(S::kUsed)>(tmem + lanes + slot * N, s);
      // heads in pairs (two-wide fp32 arithmetic); a last odd one is paired with itself
      const uint64_t c16 = f2_pack(1.f / 16.f, 1.f / 16.f);
      const uint64_t c256 = f2_pack(1.f / 256.f, 1.f / 256.f);
      const uint64_t ks2 = f2_pack(ks, ks);
#pragma unroll
      for (int g = 0; g < GP; g += 2) {
        const int g1 = g + 1 < GP ? g + 1 : g;
        const uint64_t f = f2_mul(f2_pack(tail->qscale[qs][g], tail->qscale[qs][g1]), ks2);
#pragma unroll
        for (int v = 0; v < TPR; ++v) {
          const float* d = s + v * 3 * GP;
          const uint64_t sum =
              f2_fma(f2_pack(d[2 * GP + g], d[2 * GP + g1]), c256,
                     f2_fma(f2_pack(d[GP + g], d[GP + g1]), c16, f2_pack(d[g], d[g1])));
          float x0, x1;
          f2_unpack(f2_mul(sum, f), x0, x1);
          // rows behind the end hold anything
          const bool live = r * TPR + v < n;
          x[v][g] = live ? x0 : -CUDART_INF_F;
          if (g1 > g) x[v][g1] = live ? x1 : -CUDART_INF_F;
        }
      }
      const float lv = lg2_approx(vs);            // -inf: no token, or a bad block
      float mine = 0.f;
#pragma unroll
      for (int g = 0; g < GP; ++g) {
        const float s_row = TPR == 2 ? fmaxf(x[0][g], x[TPR - 1][g]) : x[0][g];
        const float w = warp_max(s_row), wv = warp_max(s_row + lv);
        if (lane == g) mine = w;
        if (lane == GP + g) mine = wv;
      }
      if (lane < 2 * GP) tail->red[slot][wq][lane] = mine;
      __syncwarp();
      if (lane == 0) mbar_arrive(&tail->red_bar[slot]);
      return true;
    };
    // acc <- acc 2^(m_before - m) + O, with tile u's factors
    auto add_tile = [&](int u) -> bool {
      const int slot = u & 1;
      if (!wait_all(&tail->o_full[slot], (u >> 1) & 1)) return false;
      tc_fence_after();
      float o[cols_for(3 * GP)];
      load_cols<cols_for(3 * GP)>(tmem + lanes + (2 + slot) * N + par * 3 * GP, o);
      const uint64_t c16 = f2_pack(1.f / 16.f, 1.f / 16.f);
      const uint64_t c256 = f2_pack(1.f / 256.f, 1.f / 256.f);
      const float* by = tail->fold[wq][slot].by;
#pragma unroll
      for (int g = 0; g < GP; g += 2) {
        const int g1 = g + 1 < GP ? g + 1 : g;
        const uint64_t sum =
            f2_fma(f2_pack(o[2 * GP + g], o[2 * GP + g1]), c256,
                   f2_fma(f2_pack(o[GP + g], o[GP + g1]), c16, f2_pack(o[g], o[g1])));
        const uint64_t was = f2_mul(f2_pack(acc[g], acc[g1]), f2_pack(by[g], by[g1]));
        float y0, y1;
        f2_unpack(f2_fma(sum, f2_pack(by[GP + g], by[GP + g1]), was), y0, y1);
        acc[g] = y0;
        if (g1 > g) acc[g1] = y1;
      }
      return true;
    };
    // the finished segment sg of (sequence b, item): to out, or to the workspace if cut
    auto finish = [&](int sg, int b, int h, int chunk, bool whole, bool alone) -> bool {
      if (D == 64 && par == 1) {
#pragma unroll
        for (int g = 0; g < GP; ++g) tail->half[sg & 1][g * 64 + r - 64] = acc[g];
      }
      // a tile behind the segment has its red_bar between lred's writes and here; half's
      // two sets: the set of the segment before last has been read by all, at its sum_bar
      if (D == 64 || alone) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&tail->sum_bar);
        if (!wait_all(&tail->sum_bar, D == 64 ? sg & 1 : 0)) return false;
      }
      // once per segment: short code, a head to a lane where that is possible
      const int g0 = chunk * a.hch, gn = min(a.hch, G - g0);
      const int64_t part = (2 * (int64_t)blockIdx.x + (sg > 0)) * a.hch;
      if (lane < gn) {
        const float* lr = &tail->lred[sg & 1][0][lane];
        const float sum = (lr[0] + lr[GP]) + (lr[2 * GP] + lr[3 * GP]);
        tail->inv[wq][lane] = 1.f / sum;
        if (!whole && wq == 0) {
          a.ws_m[part + lane] = tail->mred[sg & 1][lane];
          a.ws_l[part + lane] = sum;
        }
      }
      __syncwarp();
      if (r < D) {
        uint16_t* to = static_cast<uint16_t*>(a.out) + ((int64_t)b * a.Hq + h * G + g0) * D + r;
        float* ws = a.ws_acc + part * D + r;
#pragma unroll
        for (int g = 0; g < GP; ++g) {
          if (g < gn) {
            const float o = acc[g] + (D == 64 ? tail->half[sg & 1][g * 64 + (r & 63)] : 0.f);
            const float y = o * tail->inv[wq][g];
            if (whole) *to = (uint16_t)(a.dtype == PA_BFLOAT16 ? pack2<PA_BFLOAT16>(y, y)
                                                                 : pack2<PA_FLOAT16>(y, y));
            else *ws = o;
          }
          to += D;
          ws += D;
        }
      }
#pragma unroll
      for (int g = 0; g < GP; ++g) acc[g] = 0.f;
      return true;
    };

    // One pass more than tiles at both ends (t = -1: only scores; t = tiles: only sums),
    // so that each step stands once in the code: a second copy would be run cold.
    Walk<TOKENS> cur = walk;                    // tile t; walk stands at tile t + 1
    cur.left = 0;
    float vs_cur = 0.f, ks_next, vs_next;       // scales of tile t; of tile t + 1
    scales_of(walk, ks_next, vs_next);
    bool first = true, first_of_item = walk.j == 0;
    int fin_b = 0, fin_h = 0, fin_chunk = 0;    // the segment that tile t - 1 finished
    bool fin = false, fin_whole = false;
#pragma unroll
    for (int g = 0; g < GP; ++g) l[g] = acc[g] = 0.f;
    for (int t = -1; in; ++t) {
      const int slot = t & 1, seg_t = seg;
      const bool have = cur.left > 0;
      const bool ends = have && (cur.j + 1 == cur.nt || cur.left == 1);
      const Walk<TOKENS> ahead = walk;          // tile t + 1
      float ks2 = 0.f, vs2 = 0.f;
      if (ahead.left > 0) {
        walk.next(a);
        scales_of(walk, ks2, vs2);              // tile t + 2
      }
      if (have) {
        const int n = cur.L - cur.j * TOKENS;     // tokens left from this tile on
        if (first) {
          m_lane = -CUDART_INF_F;
#pragma unroll
          for (int g = 0; g < GP; ++g) l[g] = 0.f;
        }
        if (!wait_all(&tail->red_bar[slot], (t >> 1) & 1)) { ok = false; break; }
        {
          const float* red = &tail->red[slot][0][min(lane, 2 * GP - 1)];
          const float top =
              fmaxf(fmaxf(red[0], red[2 * GP]), fmaxf(red[4 * GP], red[6 * GP]));
          const float top_v = __shfl_sync(kAll, top, (lane + GP) & 31);
          if (lane < GP) {
            const float now = fmaxf(m_lane, top);
            // the largest weight times scale is 2^e or less; where it is below 2^-110 (a
            // tile that adds nothing to the running maximum's, or no live block), 2^-110
            const int e = min(127, __float2int_ru(fmaxf(top_v - now, -110.f)));
            tail->top[wq].now[lane] = now;
            tail->fold[wq][slot].by[lane] = ex2_approx(m_lane - now);
            tail->fold[wq][slot].by[GP + lane] = __uint_as_float((uint32_t)(127 - 8 + e) << 23);
            m_lane = now;
          }
          __syncwarp();
        }
        // weights times V scale, in units that leave 256 at most
        const float *top = tail->top[wq].now, *by = tail->fold[wq][slot].by;
        const uint64_t vs_both = f2_pack(vs_cur, vs_cur);
#pragma unroll
        for (int g = 0; g < GP; g += 2) {
          const int g1 = g + 1 < GP ? g + 1 : g;
          const uint64_t m2 = f2_pack(top[g], top[g1]);
          const uint64_t per_unit = f2_pack(inverse_pow2(by[GP + g]), inverse_pow2(by[GP + g1]));
          uint64_t sum = f2_mul(f2_pack(l[g], l[g1]), f2_pack(by[g], by[g1]));
#pragma unroll
          for (int v = 0; v < TPR; ++v) {
            float p0, p1;                         // 0 behind the end
            f2_unpack(f2_sub(f2_pack(x[v][g], x[v][g1]), m2), p0, p1);
            p0 = ex2_approx(p0);
            p1 = ex2_approx(p1);
            const uint64_t p2 = f2_pack(p0, p1);
            sum = f2_add(sum, p2);
            uint32_t d[3];
            digits2_short(f2_mul(f2_mul(p2, vs_both), per_unit), d);
#pragma unroll
            for (int i = 0; i < 3; ++i) {
              const int row = (v * 3 + i) * GP + g;
              put[row & 7][slot * S::kOperand + row * 128] = (uint8_t)d[i];
              if (g1 > g)
                put[(row + 1) & 7][slot * S::kOperand + (row + 1) * 128] = (uint8_t)(d[i] >> 8);
            }
          }
          float l0, l1;
          f2_unpack(sum, l0, l1);
          l[g] = l0;
          if (g1 > g) l[g1] = l1;
        }
        // tokens behind the end: zero their V, so that 0 times garbage stays 0
        if (n < TOKENS) {
          const int u = 2 * t + 1;
          if (!wait_all(&tail->full[u % R], (u / R) & 1)) { ok = false; break; }
          uint8_t* vt = smem + (u % R) * kStageBytes;
#pragma unroll
          for (int v = 0; v < TPR; ++v)
            if (r * TPR + v >= n) {
#pragma unroll
              for (int c = 0; c < D; c += 16)
                *reinterpret_cast<uint4*>(vt + swizzled(r, v * D + c)) = make_uint4(0, 0, 0, 0);
            }
        }
        fence_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tail->p_full[slot]);
        if (ends) {                               // what finish() needs of tile t's segment
#pragma unroll
          for (int g = 0; g < GP; ++g) {
            float sum = l[g];
#pragma unroll
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
            if (lane == g) tail->lred[seg & 1][wq][g] = sum;
          }
          if (wq == 0 && lane < GP) tail->mred[seg & 1][lane] = m_lane;
          if (lane == 0) mbar_arrive(&tail->q_empty[seg & 1]);
          ++seg;
        }
      }
      // what finish() reads is written again only behind the red_bar that score_tile posts
      if (t > 0 && !add_tile(t - 1)) { ok = false; break; }
      if (fin && !finish(seg_t - 1, fin_b, fin_h, fin_chunk, fin_whole, !have)) {
        ok = false;
        break;
      }
      if (ahead.left <= 0 && !have) break;
      if (ahead.left > 0 && !score_tile(t + 1, ahead.L - ahead.j * TOKENS, seg, t < 0 || ends,
                                        ks_next, vs_next)) {
        ok = false;
        break;
      }
      fin = ends;
      if (ends) {
        fin_b = cur.b;
        fin_h = cur.h;
        fin_chunk = cur.chunk;
        fin_whole = first_of_item && cur.j + 1 == cur.nt;
        first_of_item = true;                   // the next segment begins at tile 0
      }
      first = t < 0 || ends;
      cur = ahead;
      vs_cur = vs_next;
      ks_next = ks2;
      vs_next = vs2;
    }
    if (!ok) {
      *abort_flag = 1;
      if (lane == 0) report(a.status_dev, PA_ERR_TIMEOUT);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kCols);
  }
}

// Joins the partials of items that window boundaries cut: CTA c looks at the boundary
// where window c + 1 begins, and joins its item, of kJoinHeads heads at most, if that
// boundary is the item's first.  With kByItem, for few items and many parts of each, CTA
// (x, y) joins kJoinHeads heads of item x, and looks for its first boundary among all.
// Its time is the chain of loads (window, then all partials), so the partials are asked
// for before the weights are known: a warp takes a head's maximum and weights, the other
// threads are elements of a head, the parts dealt out to kJoinThreads / D groups of them.
constexpr int kJoinThreads = 512;
constexpr int kPartsAhead = 4;                 // parts of a group asked for at once

template <int D, int kJoinHeads, bool kByItem>
__global__ void __launch_bounds__(kJoinThreads, 2) join_q8_kernel(const Q8Args a, int grid) {
  constexpr int GROUPS = kJoinThreads / D;
  constexpr int kJoinAhead = kByItem ? 4 * kPartsAhead : kPartsAhead;
  static_assert(kMaxGrid <= kJoinThreads, "a thread per boundary");
  __shared__ float s_w[kJoinHeads][kMaxGrid];
  __shared__ float s_sum[GROUPS][kJoinHeads][D];
  allow_next_grid();
  wait_prior_grid();
  Window at;
  bool same;
  int c, h0 = 0;                               // boundary; first head of the chunk's
  if (kByItem) {
    __shared__ Window s_at;
    __shared__ int s_c, s_same;
    const int items = a.H * a.chunks, x = (int)blockIdx.x;
    if (threadIdx.x == 0) s_c = 0;
    __syncthreads();
    c = (int)threadIdx.x + 1;
    if (c < grid) {
      at = a.info[c];
      if (first_cut(at, a.info[c - 1], &same) && at.b * items + at.item == x) {
        s_at = at;
        s_same = same;
        s_c = c;
      }
    }
    __syncthreads();
    c = s_c;
    if (c == 0) return;                        // in one window
    at = s_at;
    same = s_same;
    h0 = (int)blockIdx.y * kJoinHeads;
  } else {
    c = (int)blockIdx.x + 1;
    at = a.info[c];
    if (!first_cut(at, a.info[c - 1], &same)) return;
  }
  const int parts = last_window(at, grid) - c + 2;
  const int h = at.item / a.chunks, G = a.Hq / a.H;
  const int g0 = (at.item - h * a.chunks) * a.hch + h0;
  const int n = min(kJoinHeads, min(a.hch - h0, G - g0));
  if (n <= 0) return;                          // a last chunk of fewer heads
  auto row = [&](int k) { return part_of_item(c, same, k) * a.hch + h0; };
  const int d = threadIdx.x % D, group = threadIdx.x / D;
  float x[kJoinAhead][kJoinHeads];
#pragma unroll
  for (int i = 0; i < kJoinAhead; ++i) {
    const int k = group + i * GROUPS;
#pragma unroll
    for (int g = 0; g < kJoinHeads; ++g)
      x[i][g] = k < parts && g < n ? a.ws_acc[(row(k) + g) * D + d] : 0.f;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp < n) {
    float top = -CUDART_INF_F;
    for (int k = lane; k < parts; k += 32) {
      const float m = a.ws_m[row(k) + warp];
      s_w[warp][k] = m;
      top = fmaxf(top, m);
    }
    top = warp_max(top);
    float l = 0.f;
    for (int k = lane; k < parts; k += 32) {
      const float w = ex2_approx(s_w[warp][k] - top);
      s_w[warp][k] = w;
      l = fmaf(w, a.ws_l[row(k) + warp], l);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(kAll, l, o);
    const float inv = 1.f / l;
    for (int k = lane; k < parts; k += 32) s_w[warp][k] *= inv;
  }
  __syncthreads();
  float sum[kJoinHeads] = {};
#pragma unroll
  for (int i = 0; i < kJoinAhead; ++i) {
    const int k = group + i * GROUPS;
#pragma unroll
    for (int g = 0; g < kJoinHeads; ++g)
      if (k < parts && g < n) sum[g] = fmaf(s_w[g][k], x[i][g], sum[g]);
  }
#pragma unroll 4
  for (int k = group + kJoinAhead * GROUPS; k < parts; k += GROUPS)
#pragma unroll
    for (int g = 0; g < kJoinHeads; ++g)
      if (g < n) sum[g] = fmaf(s_w[g][k], a.ws_acc[(row(k) + g) * D + d], sum[g]);
#pragma unroll
  for (int g = 0; g < kJoinHeads; ++g) s_sum[group][g][d] = sum[g];
  __syncthreads();
  for (int g = group; g < n; g += GROUPS) {
    float y = 0.f;
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) y += s_sum[i][g][d];
    static_cast<uint16_t*>(a.out)[((int64_t)at.b * a.Hq + h * G + g0 + g) * D + d] =
        a.dtype == PA_BFLOAT16 ? narrow<PA_BFLOAT16>(y) : narrow<PA_FLOAT16>(y);
  }
}

// ------------------------------------------------------------------ host side --

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000,
                                         cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  });
  return fn;
}

// A pool as rows of 128 bytes; a box is one block of one head.
bool encode_pool(CUtensorMap* map, const void* pool, int64_t rows, int block_rows) {
  const cuuint64_t dims[2] = {128, (cuuint64_t)rows}, strides[1] = {128};
  const cuuint32_t box[2] = {128, (cuuint32_t)block_rows}, ones[2] = {1, 1};
  return encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(pool), dims, strides,
                     box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Plan {
  int chunks, hch;               // of a KV head's query heads
  int64_t tiles;                 // of the longest sequence allowed
  size_t m_off, l_off, acc_off, total;
};

// Chunks of at most 8 query heads, of equal size: a softmax thread keeps a score, a sum
// and an accumulator per head, and two CTAs of an SM leave it 128 registers (seven warps are
// allotted as eight), all of them in use for 5 and 8 heads and from 4 heads of 64 on.  So the
// cache is read twice with 16 heads: 96 us where 8 take 56 (64 sequences of 128..4,096).
Plan plan_of(int Hq, int H, int D, int max_seq_len) {
  Plan p;
  const int G = Hq / H, most = 8;
  p.chunks = (G + most - 1) / most;
  p.hch = (G + p.chunks - 1) / p.chunks;
  const int tokens = kTileRows * 128 / D;
  p.tiles = ((int64_t)max_seq_len + tokens - 1) / tokens;
  auto align = [](size_t x) { return (x + 255) & ~(size_t)255; };
  const size_t rows = (size_t)2 * kMaxGrid * p.hch;
  p.m_off = align(kMaxGrid * sizeof(Window));
  p.l_off = p.m_off + align(rows * sizeof(float));
  p.acc_off = p.l_off + align(rows * sizeof(float));
  p.total = p.acc_off + align(rows * D * sizeof(float));
  return p;
}

template <int D, int GP>
cudaError_t launch_decode(const CUtensorMap& k, const CUtensorMap& v, const Q8Args& a, int grid,
                          int device, cudaStream_t stream) {
  constexpr int bytes = smem_bytes<D, GP>();
  static_assert(2 * (bytes + 1024) <= 233472, "two CTAs fit an SM");
  static std::mutex lock;
  static uint64_t done = 0;                    // devices whose attribute is set
  {
    std::lock_guard<std::mutex> hold(lock);
    if (device >= 64 || !(done >> device & 1)) {
      const cudaError_t e = taken(cudaFuncSetAttribute(
          decode_q8_kernel<D, GP>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
      if (e != cudaSuccess) return e;
      if (device < 64) done |= 1ull << device;
    }
  }
  return launch_pdl(decode_q8_kernel<D, GP>, dim3((unsigned)grid), kThreads, bytes, stream, k, v,
                    a);
}

template <int D>
cudaError_t launch_heads(const CUtensorMap& k, const CUtensorMap& v, const Q8Args& a, int grid,
                         int device, cudaStream_t stream) {
  if (a.hch <= 1) return launch_decode<D, 1>(k, v, a, grid, device, stream);
  if (a.hch <= 2) return launch_decode<D, 2>(k, v, a, grid, device, stream);
  if (a.hch <= 4) return launch_decode<D, 4>(k, v, a, grid, device, stream);
  if (a.hch <= 5) return launch_decode<D, 5>(k, v, a, grid, device, stream);
  return launch_decode<D, 8>(k, v, a, grid, device, stream);
}

// One CTA to a boundary and all of an item's heads: every CTA is resident at once (8
// sequences of 32,768..131,072: 202.7 us; with a CTA to every cut segment 204.9).
// Items of at least twice as many parts as such a CTA asks for at once: a CTA to an item
// and two heads, whose loads are all asked for at once (one sequence of 131,072 and one KV
// head of 5, 304 parts: 24.8 us for 30.2; one of 50,001 and eight of 5, 38 parts: 27.4 for
// 28.1; four of 8,000, 9 parts: 22.2 for 21.2, so not those).
template <int D>
cudaError_t launch_join(const Q8Args& a, int grid, cudaStream_t stream) {
  const int64_t items = (int64_t)a.B * a.H * a.chunks;
  if (items * 2 * kPartsAhead * (kJoinThreads / D) <= grid)
    return launch_pdl(join_q8_kernel<D, 2, true>,
                      dim3((unsigned)items, (unsigned)((a.hch + 1) / 2)), kJoinThreads, 0, stream,
                      a, grid);
  auto join = a.hch <= 2 ? join_q8_kernel<D, 2, false>
                         : (a.hch <= 4 ? join_q8_kernel<D, 4, false> : join_q8_kernel<D, 8, false>);
  return launch_pdl(join, dim3((unsigned)(grid - 1)), kJoinThreads, 0, stream, a, grid);
}

}  // namespace
}  // namespace pa

using namespace pa;

// Host checks shared by the call and its workspace query.
static pa_status check_q8(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                          int block_size, int max_seq_len) {
  if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || max_seq_len < 0)
    return PA_ERR_INVALID_ARG;
  if (num_q_heads % num_kv_heads) return PA_ERR_INVALID_ARG;
  if (!(head_dim == 64 || head_dim == 128)) return PA_ERR_UNSUPPORTED;
  if (!(block_size == 8 || block_size == 16 || block_size == 32 || block_size == 64))
    return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

extern "C" size_t pa_decode_q8_workspace_bytes(int num_seqs, int num_q_heads, int num_kv_heads,
                                               int head_dim, int block_size, int max_seq_len) {
  if (check_q8(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, max_seq_len) != PA_OK)
    return 0;
  return plan_of(num_q_heads, num_kv_heads, head_dim, max_seq_len).total;
}

extern "C" pa_status pa_decode_q8(void* out, const void* q, const void* k_pool, const void* v_pool,
                                  const float* k_scale, const float* v_scale,
                                  const int32_t* block_tables, const int32_t* seq_lens,
                                  int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                  int block_size, int max_blocks, int num_blocks, int max_seq_len,
                                  float scale, int dtype, void* workspace, size_t workspace_bytes,
                                  int32_t* status_dev, cudaStream_t stream) {
  if (max_blocks <= 0 || num_blocks <= 0) return PA_ERR_INVALID_ARG;
  const pa_status st =
      check_q8(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, max_seq_len);
  if (st != PA_OK) return st;
  if (dtype != PA_FLOAT16 && dtype != PA_BFLOAT16) return PA_ERR_UNSUPPORTED;
  if ((long long)max_seq_len > (long long)max_blocks * block_size) return PA_ERR_INVALID_ARG;
  if (!isfinite(scale)) return PA_ERR_INVALID_ARG;
  if (num_seqs == 0) return PA_OK;
  if (!out || !q || !k_pool || !v_pool || !k_scale || !v_scale || !block_tables || !seq_lens)
    return PA_ERR_INVALID_ARG;
  if ((((uintptr_t)out | (uintptr_t)q | (uintptr_t)k_pool | (uintptr_t)v_pool) & 15u) != 0 ||
      (((uintptr_t)k_scale | (uintptr_t)v_scale) & 3u) != 0)
    return PA_ERR_INVALID_ARG;
  const Plan p = plan_of(num_q_heads, num_kv_heads, head_dim, max_seq_len);
  if (!workspace || ((uintptr_t)workspace & 255u) || workspace_bytes < p.total)
    return PA_ERR_WORKSPACE;
  // 32-bit rows, tiles of all sequences, positions up to a tile of blocks behind the end, and
  // cost of one sequence's items (4 a tile and at most 4 an item, which the kernel takes
  // apart in 32 bits)
  const int block_rows = block_size * head_dim / 128;
  const long long rows = (long long)num_blocks * num_kv_heads * block_rows;
  if (rows >= (1ll << 31) || max_seq_len > 0x7FFFFFFF - 2047 ||
      (long long)num_seqs * p.tiles >= (1ll << 28) ||
      (long long)num_kv_heads * p.chunks >= (1ll << 20) ||
      4 * (p.tiles + 1) * num_kv_heads * p.chunks >= (1ll << 31))
    return PA_ERR_INVALID_ARG;
  int device = 0, sms = 0;
  if (!encode_fn() || taken(cudaGetDevice(&device)) != cudaSuccess ||
      taken(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device)) != cudaSuccess)
    return PA_ERR_CUDA;
  CUtensorMap k, v;
  if (!encode_pool(&k, k_pool, rows, block_rows) || !encode_pool(&v, v_pool, rows, block_rows))
    return PA_ERR_INVALID_ARG;

  Q8Args a;
  a.out = out;
  a.q = q;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.tables = block_tables;
  a.lens = seq_lens;
  a.B = num_seqs;
  a.Hq = num_q_heads;
  a.H = num_kv_heads;
  a.bs = block_size;
  a.bs_shift = block_size == 8 ? 3 : (block_size == 16 ? 4 : (block_size == 32 ? 5 : 6));
  a.max_blocks = max_blocks;
  a.num_blocks = num_blocks;
  a.max_seq_len = max_seq_len;
  a.chunks = p.chunks;
  a.hch = p.hch;
  a.rows_total = (int)rows;
  a.scale_log2 = (float)((double)scale * 1.4426950408889634);
  a.dtype = dtype;
  char* ws = static_cast<char*>(workspace);
  a.info = reinterpret_cast<Window*>(ws);
  a.ws_m = reinterpret_cast<float*>(ws + p.m_off);
  a.ws_l = reinterpret_cast<float*>(ws + p.l_off);
  a.ws_acc = reinterpret_cast<float*>(ws + p.acc_off);
  a.status_dev = status_dev;

  const long long work = (long long)num_seqs * p.tiles * num_kv_heads * p.chunks;
  const long long ctas = 2ll * sms < kMaxGrid ? 2ll * sms : kMaxGrid;
  const int grid = (int)(work < 1 ? 1 : (work < ctas ? work : ctas));
  if (work / grid >= (1ll << 31)) return PA_ERR_INVALID_ARG;
  cudaError_t e = head_dim == 128 ? launch_heads<128>(k, v, a, grid, device, stream)
                                  : launch_heads<64>(k, v, a, grid, device, stream);
  // an item of one tile is never cut
  if (e == cudaSuccess && p.tiles > 1 && grid > 1)
    e = head_dim == 128 ? launch_join<128>(a, grid, stream) : launch_join<64>(a, grid, stream);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
