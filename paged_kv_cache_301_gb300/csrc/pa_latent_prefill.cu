// pa_latent_prefill: causal attention in the expanded form of latent attention, on the
// Blackwell tensor cores (tcgen05 + TMEM) with TMA loads.
//
//   out = sum_t p_t v_t / sum_t p_t,  p_t = 2^(s_t - m),
//   s_t = log2(e) scale (q[:128] . k_t + q[128:] . r_t),   t = 0 .. the query's position
//
// One CTA: a sequence, a head and two adjacent query tiles A, B of 128 rows.  Every tile of
// 128 keys (48 KB: two slabs of the head's own part, one of the shared rotated part) and
// their values (32 KB) serves both:
//   S_k [128 x 128] = Q_k [128 x 192] . K^T    (TMEM, 128 columns)
//   P_k over the columns of S_k it came from, in the storage type (a second term behind it)
//   O_k [128 x 128] += P_k . V                  (P from TMEM, V from shared memory)
// The tensor cores alternate between the tiles, P_A . V, S_A of the next keys, P_B . V, S_B,
// while the softmax warps of the other tile work.  The running maximum is raised only where
// a tile exceeds it by more than 2^8.
//
// Shared memory holds both query tiles (96 KB), two tiles of keys and one of values: keys are
// asked for a tile ahead, values while S_B of the next keys runs.
//
// Weights are rounded to the storage type once (half a step: bf16 2^-8, fp16 2^-11 of each), or
// with PA_TWO_TERMS kept as two terms, the second behind the first over the columns of S and with
// a product of its own (331 us for the prompts below, 165 for the chunks).
//
// Bound: for 256 rows and 128 keys the tensor cores take 2,600 cycles and the exponentials
// 2,050; a query tile's own chain (scores, softmax, product, and the waits between them) takes
// 4,000 and two tiles overlap in part.
//
// Measured (GB300; cuBLAS 1,880 TFLOP/s): four prompts of 960 to 3,648 tokens, 32 heads, bf16
// 265 us, 978 TFLOP/s; six chunks of 500 tokens, the longest of a sequence of 6,488, 16 heads,
// fp16 123-127 us: that one's 51 tiles of keys are one CTA's chain.  Tried: values asked for in
// halves (287 us for the prompts, 269 then).
//
// Values that a row does not see have no part in it: those behind the sequence's end are
// zeroed in shared memory, and in the tiles that cut the diagonal so are rows that hold
// infinities or NaN; what they give to the rows that see them is added by the softmax warps.
//
// Roles (320 threads): warp 0 TMA, warp 1 tcgen05.mma, warps 2-5 tile A's softmax and warps
// 6-9 tile B's, one thread per row.  Every wait is bounded.
#include <math.h>
#include <math_constants.h>

#include <mutex>

#include "pa_common.cuh"
#include "pa_internal.h"
#include "pa_q8.cuh"
#include "pa_sm100.cuh"

namespace pa {
namespace {

using namespace sm100;

constexpr int kRows = 128;                    // query rows of a tile
constexpr int kKeys = 128;                    // keys of a tile
constexpr int kSlab = 128 * 128;              // 128 rows of 64 elements
constexpr int kQSlabs = 3, kVSlabs = 2;
constexpr int kDk = 64 * kQSlabs, kDv = 64 * kVSlabs, kRope = 64, kKv = kDk - kRope + kDv;
constexpr int kKTile = kQSlabs * kSlab, kVTile = kVSlabs * kSlab;
constexpr int kQOff = 0;                      // Q_A, then Q_B
constexpr int kKOff = 2 * kQSlabs * kSlab;    // two tiles of keys
constexpr int kVOff = kKOff + 2 * kKTile;
constexpr int kTailOff = kVOff + kVTile;
constexpr int kTailBytes = 1024;
constexpr int kSmem = kTailOff + kTailBytes + 1024;
static_assert(kSmem <= 232448, "fits an SM");
constexpr int kThreads = 64 + 256;
constexpr float kRaise = 8.f;                 // log2 by which a tile may exceed the maximum
constexpr uint64_t kLimitNs = 2000000000ull;
constexpr unsigned kAll = 0xFFFFFFFFu;
// TMEM: S/P_A at column 0, S/P_B at 128, O_A at 256, O_B at 384
constexpr uint32_t kCols = 512;

struct Args {
  void* out;
  const void* kv;
  const int32_t* q_start;
  const int32_t* kv_start;
  int B, total_q, total_kv, H, max_q, pairs;
  float scale_log2;
  int32_t* status_dev;
};

struct Tail {
  uint64_t k_full[2], k_empty[2], v_full, v_empty, q_full;
  uint64_t s_full[2], p_full[2], pv_done[2];     // of the query tiles
  uint64_t odd_full[2], drain;
  uint32_t odd[2][4];            // rows of V that are added apart, in A's tiles on the diagonal
  uint32_t odd_b[4];             // in the one behind them, B's own
  int keep[2];                   // O_k holds something before its first product
  uint32_t tmem;
  int abort_flag;
};
static_assert(sizeof(Tail) <= kTailBytes, "barrier block");

__device__ __forceinline__ void tma_slab(void* dst, const CUtensorMap* map, uint64_t* bar, int x,
                                         int h, int row) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(x), "r"(h), "r"(row)
      : "memory");
}

// mma_by_one with A in tensor memory.
__device__ __forceinline__ void mma_ts_by_one(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ uint32_t tmem_ld1(uint32_t t) {
  uint32_t r;
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r)
      : "r"(t)
      : "memory");
  return r;
}

// TERMS: storage-type terms of a softmax weight.
template <int DT, int TERMS>
__global__ void __launch_bounds__(kThreads, 1)
latent_prefill_kernel(const __grid_constant__ CUtensorMap map_q,
                      const __grid_constant__ CUtensorMap map_kv,
                      const __grid_constant__ CUtensorMap map_r, const Args a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  Tail* tl = reinterpret_cast<Tail*>(smem + kTailOff);
  volatile int* abort_flag = &tl->abort_flag;
  const int lane = threadIdx.x & 31;
  const int warp = __shfl_sync(kAll, threadIdx.x >> 5, 0);
  allow_next_grid();
  wait_prior_grid();
  // the pairs of query tiles with the longest causal work first, so that the last CTAs to run
  // are short (four prompts of 32 heads: 269 us; pairs of one sequence and head side by side,
  // whose keys and values stay in L2: 287)
  const int bhs = gridDim.x / a.pairs, bh = blockIdx.x % bhs;
  const int pair = a.pairs - 1 - (int)(blockIdx.x / bhs);
  const int b = bh / a.H, h = bh - b * a.H;
  const int qs = a.q_start[b], n = a.q_start[b + 1] - qs;
  const int ks = a.kv_start[b], L = a.kv_start[b + 1] - ks;
  if (qs < 0 || n < 0 || ks < 0 || L < 0 || n > L || n > a.max_q || n > a.total_q - qs ||
      L > a.total_kv - ks) {
    if (threadIdx.x == 0 && h == 0 && pair == 0) report(a.status_dev, PA_ERR_BAD_BLOCK_ID);
    return;
  }
  const int q0a = 2 * pair * kRows, q0b = q0a + kRows;
  if (q0a >= n) return;                        // no rows in this pair
  const int ctx = L - n;
  // key tiles 0 .. last of each query tile (-1: no rows); the first that not all rows of A see
  const int last_a = (ctx + min(q0a + kRows, n) - 1) / kKeys;
  const int last_b = q0b < n ? (ctx + min(q0b + kRows, n) - 1) / kKeys : -1;
  const int last_all = last_b >= 0 ? last_b : last_a;
  const int cut_a = (ctx + q0a + 1) / kKeys, cut_b = (ctx + q0b + 1) / kKeys;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tl->k_full[i], 1);
      mbar_init(&tl->k_empty[i], 1);
      mbar_init(&tl->s_full[i], 1);
      mbar_init(&tl->p_full[i], 4);
      mbar_init(&tl->pv_done[i], 1);
      mbar_init(&tl->odd_full[i], 4);
      tl->keep[i] = 0;
    }
    mbar_init(&tl->v_full, 1);
    mbar_init(&tl->v_empty, 1);
    mbar_init(&tl->q_full, 1);
    mbar_init(&tl->drain, 1);
    tl->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&map_q);
    tma_prefetch_desc(&map_kv);
    tma_prefetch_desc(&map_r);
  }
  if (warp == 1) {
    tmem_alloc(&tl->tmem, kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tl->tmem;
  auto set_abort = [&]() {
    tl->abort_flag = 1;
    report(a.status_dev, PA_ERR_TIMEOUT);
  };

  if (warp == 0) {
    // ---------------------------------------------------------------- producer --
    // rows behind the sequence's last are the next one's (or zeros): masked, and zeroed in V
    if (lane == 0) {
      bool ok = true;
      int k_used = 0, v_used = 0;
      mbar_arrive_expect_tx(&tl->q_full, (last_b >= 0 ? 2u : 1u) * kKTile);
      for (int k = 0; k < (last_b >= 0 ? 2 : 1); ++k)
        for (int x = 0; x < kQSlabs; ++x)
          tma_slab(smem + kQOff + (k * kQSlabs + x) * kSlab, &map_q, &tl->q_full, 64 * x, h,
                   qs + (k ? q0b : q0a));
      for (int t = 0; t <= last_all && ok; ++t) {
        const int row = ks + t * kKeys, s = t & 1;
        ok = mbar_wait(&tl->k_empty[s], ((t >> 1) & 1) ^ 1, abort_flag, kLimitNs);
        if (!ok) break;
        uint8_t* kt = smem + kKOff + s * kKTile;
        mbar_arrive_expect_tx(&tl->k_full[s], kKTile);
        tma_slab(kt, &map_kv, &tl->k_full[s], 0, h, row);
        tma_slab(kt + kSlab, &map_kv, &tl->k_full[s], 64, h, row);
        tma_slab(kt + 2 * kSlab, &map_r, &tl->k_full[s], 0, 0, row);
        ++k_used;
        ok = mbar_wait(&tl->v_empty, (t & 1) ^ 1, abort_flag, kLimitNs);
        if (!ok) break;
        mbar_arrive_expect_tx(&tl->v_full, kVTile);
        tma_slab(smem + kVOff, &map_kv, &tl->v_full, kDk - kRope, h, row);
        tma_slab(smem + kVOff + kSlab, &map_kv, &tl->v_full, kDk - kRope + 64, h, row);
        ++v_used;
      }
      if (!ok) set_abort();
      if (*abort_flag) {                       // copies in flight land before the CTA ends
        for (int t = max(0, k_used - 2); t < k_used; ++t)
          mbar_wait_drain(&tl->k_full[t & 1], (t >> 1) & 1, kLimitNs);
        if (v_used) mbar_wait_drain(&tl->v_full, (v_used - 1) & 1, kLimitNs);
        mbar_wait_drain(&tl->q_full, 0, kLimitNs);
      }
    }
  } else if (warp == 1) {
    // -------------------------------------------------------------- MMA issue --
    constexpr uint32_t ab = DT == PA_BFLOAT16 ? 1u : 0u;
    constexpr uint32_t idesc_s = idesc_f16(ab, 0, 0, kRows, kKeys);   // Q, K both K-major
    constexpr uint32_t idesc_o = idesc_f16(ab, 0, 1, kRows, kDv);     // P (TMEM), V MN-major
    const uint64_t q_desc = smem_desc_sw128(smem_addr(smem + kQOff), 16, 1024);
    const uint64_t k_desc = smem_desc_sw128(smem_addr(smem + kKOff), 16, 1024);
    const uint64_t v_desc = smem_desc_sw128(smem_addr(smem + kVOff), kSlab, 1024);
    bool ok = true, issued = false;
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(kAll, mbar_wait(bar, parity, abort_flag, kLimitNs));
    };
    auto issue_s = [&](int k, int t) {
      const uint64_t kd = k_desc + (uint32_t)((t & 1) * (kKTile >> 4));
      const uint64_t qd = q_desc + (uint32_t)(k * (kQSlabs * kSlab >> 4));
#pragma unroll
      for (int x = 0; x < 4 * kQSlabs; ++x) {
        const uint64_t off = (uint64_t)(((x >> 2) * kSlab + (x & 3) * 32) >> 4);
        mma_by_one(tmem + k * kKeys, qd + off, kd + off, idesc_s, x > 0);
      }
      commit_by_one(&tl->s_full[k]);
      issued = true;
    };
    auto issue_pv = [&](int k, int t) {
      const uint32_t keep = t > 0 || *const_cast<volatile int*>(&tl->keep[k]);
#pragma unroll
      for (int x = 0; x < kKeys / 16; ++x)
#pragma unroll
        for (int term = 0; term < TERMS; ++term)
          mma_ts_by_one(tmem + 256 + k * kDv, tmem + k * kKeys + term * (kKeys / 2) + x * 8,
                        v_desc + (uint64_t)(x * 16 * 128 >> 4), idesc_o,
                        x > 0 || term > 0 ? 1u : keep);
      commit_by_one(&tl->pv_done[k]);
    };
    ok = wait(&tl->q_full, 0) && wait(&tl->k_full[0], 0);
    if (ok) {
      tc_fence_after();
      issue_s(0, 0);
      if (last_b >= 0) issue_s(1, 0);
      commit_by_one(&tl->k_empty[0]);
    }
    for (int t = 0; t <= last_all && ok; ++t) {
      ok = wait(&tl->v_full, t & 1);
      bool next_k = false;
      for (int k = 0; k < 2 && ok; ++k) {
        const int last = k ? last_b : last_a;
        if (t > last) continue;
        ok = wait(&tl->p_full[k], t & 1);
        if (!ok) break;
        tc_fence_after();
        issue_pv(k, t);
        if (k == 1 || t > last_b) commit_by_one(&tl->v_empty);    // its last product
        if (t + 1 <= last) {
          // S of the next keys goes over P: once the product has read it
          ok = (next_k || wait(&tl->k_full[(t + 1) & 1], ((t + 1) >> 1) & 1)) &&
               wait(&tl->pv_done[k], t & 1);
          if (!ok) break;
          next_k = true;
          tc_fence_after();
          issue_s(k, t + 1);
        }
      }
      if (ok && t + 1 <= last_all) commit_by_one(&tl->k_empty[(t + 1) & 1]);
    }
    if (!ok && lane == 0) set_abort();
    // every product and commit issued here ends before TMEM is freed
    if (issued) {
      commit_by_one(&tl->drain);
      mbar_wait_drain(&tl->drain, 0, kLimitNs);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------ softmax and output rows --
    const int k = (warp - 2) >> 2, wq = warp & 3, r = wq * 32 + lane;
    const uint32_t quarter = (uint32_t)(wq * 32) << 16;
    const int i = (k ? q0b : q0a) + r;
    const bool row_valid = i < n;
    const int pos = row_valid ? ctx + i : -1;    // keys 0 .. pos are seen
    const uint32_t scol = tmem + quarter + k * kKeys, ocol = tmem + quarter + 256 + k * kDv;
    const float sl2 = a.scale_log2;
    // fp16 weights stand 2^7 higher: below 2^-14 they would lose bits
    constexpr float kShift = DT == PA_BFLOAT16 ? 0.f : 7.f;
    float m_run = -CUDART_INF_F, l_run = 0.f;
    // A wait that runs out, or finds that another's has, ends the waiting and nothing else: the
    // warp goes on through its tiles, so that every thread meets the named barrier (which has no
    // limit of its own).  Its rows are not stored.
    const uint32_t flag = smem_addr(&tl->abort_flag);
    auto wait_all = [&](uint64_t* bar, int parity) {
      if (!__all_sync(kAll, mbar_try_wait(bar, parity)) &&
          !__all_sync(kAll, mbar_wait_far<kLimitNs>(smem_addr(bar), parity, flag)))
        *abort_flag = 1;
    };
    const int my_last = k ? last_b : last_a;
    for (int t = 0; t <= my_last; ++t) {
      wait_all(&tl->s_full[k], t & 1);
      tc_fence_after();
      const int kc = t * kKeys;
      float sv[kKeys];
      {
        float h0[64], h1[64];
        tmem_ld64(scol, h0);
        tmem_ld64(scol + 64, h1);
#pragma unroll
        for (int e = 0; e < 64; ++e) {
          sv[e] = h0[e];
          sv[64 + e] = h1[e];
        }
      }
      if (kc + kKeys - 1 > pos) {
#pragma unroll
        for (int e = 0; e < kKeys; ++e) sv[e] = kc + e <= pos ? sv[e] : -CUDART_INF_F;
      }
      float mx4[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
      for (int e = 0; e < kKeys; e += 8) {
#pragma unroll
        for (int c = 0; c < 4; ++c) mx4[c] = fmax3(mx4[c], sv[e + 2 * c], sv[e + 2 * c + 1]);
      }
      const float m_tile = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * sl2;
      const bool raise = m_run != -CUDART_INF_F && m_tile > m_run + kRaise;
      const float alpha = raise ? ex2_approx(m_run - m_tile) : 1.f;
      if (m_run == -CUDART_INF_F || raise) m_run = m_tile;
      const float neg_m = (m_run == -CUDART_INF_F ? 0.f : -m_run) + kShift;
      const uint64_t sl2x2 = f2_pack(sl2, sl2), negm2 = f2_pack(neg_m, neg_m);
      uint64_t ls2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
      for (int g = 0; g < kKeys; g += 32) {
        uint32_t pw[16], pl[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          float x, y;
          f2_unpack(f2_fma(f2_pack(sv[g + e], sv[g + e + 1]), sl2x2, negm2), x, y);
          x = ex2_approx(x);
          y = ex2_approx(y);
          ls2[(e >> 1) & 1] = f2_add(ls2[(e >> 1) & 1], f2_pack(x, y));
          if (TERMS == 1) pw[e >> 1] = pack2<DT>(x, y);
          else split2<DT>(x, y, &pw[e >> 1], &pl[e >> 1]);
        }
        tmem_st16_nowait(scol + g / 2, pw);      // over S columns already read
        if (TERMS == 2) tmem_st16_nowait(scol + (kKeys + g) / 2, pl);
      }
      float ls4[4];
      f2_unpack(ls2[0], ls4[0], ls4[1]);
      f2_unpack(ls2[1], ls4[2], ls4[3]);
      l_run = fmaf(l_run, alpha, (ls4[0] + ls4[1]) + (ls4[2] + ls4[3]));
      // O is complete up to tile t - 1 and P . V of this one not issued yet
      if (__any_sync(kAll, raise)) {
        wait_all(&tl->pv_done[k], (t - 1) & 1);
        tc_fence_after();
#pragma unroll 1
        for (int c0 = 0; c0 < kDv; c0 += 32) {
          float o[32];
          tmem_ld32(ocol + c0, o);
          uint32_t ow[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) ow[e] = __float_as_uint(o[e] * alpha);
          tmem_st32(ocol + c0, ow);
        }
      }
      // V of keys behind the end, and in tiles on the diagonal, whose V the first query tile
      // that multiplies it looks through
      const bool on_a = t >= cut_a && t <= last_a;            // looked through by A
      const bool on_b = k == 1 && t > last_a && t >= cut_b;   // by B
      const bool mine = k == 0 ? on_a : on_b;
      const bool ends = kc + kKeys > L && (k == 0 || t > last_a);
      uint32_t* words = on_a ? tl->odd[(t - cut_a) & 1] : tl->odd_b;
      if (ends || mine) {
        wait_all(&tl->v_full, t & 1);
        // 16 bytes of the row at a time, lanes side by side over the banks
        auto part = [&](int x) {
          return smem + kVOff + (x >> 3) * kSlab + r * 128 + ((x ^ r) & 7) * 16;
        };
        bool zero = kc + r >= L;
        if (mine) {
          bool odd = false;
          if (!zero) {
#pragma unroll 4
            for (int x = 0; x < 16; ++x) {
              const uint4 w = *reinterpret_cast<const uint4*>(part(x));
              odd = odd || odd2<DT>(w.x) || odd2<DT>(w.y) || odd2<DT>(w.z) || odd2<DT>(w.w);
            }
          }
          const uint32_t rows = __ballot_sync(kAll, odd);
          if (lane == 0) words[wq] = rows;
          zero = zero || odd;
        }
        if (zero) {
#pragma unroll 4
          for (int x = 0; x < 16; ++x)
            *reinterpret_cast<uint4*>(part(x)) = make_uint4(0, 0, 0, 0);
        }
      }
      if (on_a || on_b) {
        bool apart;
        if (k == 0) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&tl->odd_full[(t - cut_a) & 1]);
        }
        if (on_a) {                                // once a barrier: t - cut_a is 0 or 1
          wait_all(&tl->odd_full[(t - cut_a) & 1], 0);
        } else {
          named_barrier(1, 128);                   // B's own warps
        }
        // all four are written, unless a wait has run out
        apart = !__any_sync(kAll, *abort_flag) && (words[0] | words[1] | words[2] | words[3]) != 0;
        if (apart) {
          // O += p v for each such row that this one sees
          tmem_wait_st();
          if (t > 0) {
            wait_all(&tl->pv_done[k], (t - 1) & 1);
            tc_fence_after();
          } else if (lane == 0 && wq == 0) {
            tl->keep[k] = 1;
          }
          bool fresh = t == 0;
#pragma unroll 1
          for (int w = 0; w < 4; ++w) {
            uint32_t rows = words[w];
            while (rows) {
              const int x = w * 32 + __ffs(rows) - 1;
              rows &= rows - 1;
              const bool seen = kc + x <= pos;
              float2 p2 = widen2<DT>(tmem_ld1(scol + x / 2));
              if (TERMS == 2) {
                const float2 rest = widen2<DT>(tmem_ld1(scol + (kKeys + x) / 2));
                p2 = make_float2(p2.x + rest.x, p2.y + rest.y);
              }
              const float p = x & 1 ? p2.y : p2.x;
              const uint32_t* v = static_cast<const uint32_t*>(a.kv) + (kDk - kRope) / 2 +
                                  ((int64_t)(ks + kc + x) * a.H + h) * (kKv / 2);
#pragma unroll 1
              for (int c0 = 0; c0 < kDv; c0 += 16) {
                float o[16];
                tmem_ld16(ocol + c0, o);
                uint32_t ow[16];
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                  const float2 y = widen2<DT>(v[(c0 + e) / 2]);
                  const float o0 = fresh ? 0.f : o[e], o1 = fresh ? 0.f : o[e + 1];
                  ow[e] = __float_as_uint(seen ? fmaf(p, y.x, o0) : o0);
                  ow[e + 1] = __float_as_uint(seen ? fmaf(p, y.y, o1) : o1);
                }
                tmem_st16_nowait(ocol + c0, ow);
                tmem_wait_st();
              }
              fresh = false;
            }
          }
        }
      }
      // consume P.V(t-1)'s completion before P(t) is released, so that the barrier cannot run
      // two phases ahead of a waiting warp
      if (t > 0) wait_all(&tl->pv_done[k], (t - 1) & 1);
      tmem_wait_st();                            // every P word is in tensor memory
      tc_fence_before();
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tl->p_full[k]);
    }
    if (my_last >= 0) {
      wait_all(&tl->pv_done[k], my_last & 1);
      if (__any_sync(kAll, *abort_flag)) {
        if (lane == 0) report(a.status_dev, PA_ERR_TIMEOUT);
      } else {
        tc_fence_after();
        const float inv = l_run == 0.f ? 0.f : 1.f / l_run;
        uint4* dst = reinterpret_cast<uint4*>(
            static_cast<uint16_t*>(a.out) +
            ((int64_t)(qs + (row_valid ? i : 0)) * a.H + h) * kDv);
#pragma unroll
        for (int c0 = 0; c0 < kDv; c0 += 32) {
          float o[32];
          tmem_ld32(ocol + c0, o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = inv == 0.f ? 0.f : o[e] * inv;
          if (row_valid) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
              dst[c0 / 8 + c] =
                  make_uint4(pack2<DT>(o[8 * c], o[8 * c + 1]),
                             pack2<DT>(o[8 * c + 2], o[8 * c + 3]),
                             pack2<DT>(o[8 * c + 4], o[8 * c + 5]),
                             pack2<DT>(o[8 * c + 6], o[8 * c + 7]));
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
}

// [rows, heads, width], rows `stride` elements apart; a box is 128 rows of 64 elements of a head.
bool encode_rows(CUtensorMap* map, const void* x, int dtype, int64_t rows, int heads, int width,
                 int64_t stride) {
  const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)width * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, 1, 128}, ones[3] = {1, 1, 1};
  return encode_fn()(map,
                     dtype == PA_BFLOAT16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                          : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                     3, const_cast<void*>(x), dims, strides, box, ones,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DT, int TERMS>
cudaError_t launch(const CUtensorMap (&m)[3], const Args& a, int ctas, int device,
                   cudaStream_t stream) {
  static std::mutex lock;
  static uint64_t done = 0;                    // devices whose attribute is set
  {
    std::lock_guard<std::mutex> hold(lock);
    if (device >= 64 || !(done >> device & 1)) {
      const cudaError_t e = taken(cudaFuncSetAttribute(
          latent_prefill_kernel<DT, TERMS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem));
      if (e != cudaSuccess) return e;
      if (device < 64) done |= 1ull << device;
    }
  }
  return launch_pdl(latent_prefill_kernel<DT, TERMS>, dim3((unsigned)ctas), kThreads, kSmem, stream,
                    m[0], m[1], m[2], a);
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" pa_status pa_latent_prefill(void* out, const void* q, const void* kv,
                                       const void* key_rope, const int32_t* q_start,
                                       const int32_t* kv_start, int num_seqs, int total_q,
                                       int total_kv, int64_t key_token_stride, int num_heads,
                                       int nope_dim, int rope_dim, int value_dim, int max_q_len,
                                       float scale, int dtype, int32_t* status_dev,
                                       cudaStream_t stream) {
  const bool two = dtype & PA_TWO_TERMS;
  dtype &= ~PA_TWO_TERMS;
  if (num_seqs < 0 || total_q < 0 || total_kv < 0 || num_heads <= 0 || max_q_len < 0 ||
      !(scale > 0.f) || !(scale < 3.0e38f) || (int64_t)total_q * num_heads >= (1ll << 31) ||
      (int64_t)total_kv * num_heads >= (1ll << 31))
    return PA_ERR_INVALID_ARG;
  if (nope_dim != kDk - kRope || rope_dim != kRope || value_dim != kDv ||
      (dtype != PA_FLOAT16 && dtype != PA_BFLOAT16))
    return PA_ERR_UNSUPPORTED;
  if (key_token_stride == 0) key_token_stride = rope_dim;
  if (key_token_stride < rope_dim || key_token_stride % 8 || key_token_stride >= (1ll << 38))
    return PA_ERR_INVALID_ARG;
  if (num_seqs == 0 || total_q == 0 || max_q_len == 0) return PA_OK;
  if (!out || !q || !q_start || !kv_start || (total_kv > 0 && (!kv || !key_rope)))
    return PA_ERR_INVALID_ARG;
  if ((((uintptr_t)out | (uintptr_t)q | (uintptr_t)kv | (uintptr_t)key_rope) & 15u) != 0)
    return PA_ERR_INVALID_ARG;
  const int64_t pairs = ((int64_t)max_q_len + 2 * kRows - 1) / (2 * kRows);
  // a factor at a time: the product of all three may pass 64 bits
  const int64_t most = 0x7FFFFFFF, heads_of_all = (int64_t)num_seqs * num_heads;
  if (heads_of_all > most || heads_of_all * pairs > most) return PA_ERR_INVALID_ARG;
  const int64_t ctas = heads_of_all * pairs;
  int device = 0;
  if (!encode_fn() || taken(cudaGetDevice(&device)) != cudaSuccess) return PA_ERR_CUDA;
  // without a token every sequence is bad or empty: the maps are not read
  const int64_t rows = total_kv > 0 ? total_kv : 1;
  CUtensorMap m[3];
  if (!encode_rows(&m[0], q, dtype, total_q, num_heads, kDk, (int64_t)num_heads * kDk) ||
      !encode_rows(&m[1], total_kv > 0 ? kv : q, dtype, rows, num_heads, kKv,
                   (int64_t)num_heads * kKv) ||
      !encode_rows(&m[2], total_kv > 0 ? key_rope : q, dtype, rows, 1, kRope, key_token_stride))
    return PA_ERR_INVALID_ARG;
  Args a;
  a.out = out;
  a.kv = kv;
  a.q_start = q_start;
  a.kv_start = kv_start;
  a.B = num_seqs;
  a.total_q = total_q;
  a.total_kv = total_kv;
  a.H = num_heads;
  a.max_q = max_q_len;
  a.pairs = (int)pairs;
  a.scale_log2 = (float)((double)scale * 1.4426950408889634);
  a.status_dev = status_dev;
  const auto f = dtype == PA_BFLOAT16 ? (two ? launch<PA_BFLOAT16, 2> : launch<PA_BFLOAT16, 1>)
                                      : (two ? launch<PA_FLOAT16, 2> : launch<PA_FLOAT16, 1>);
  const cudaError_t e = f(m, a, (int)ctas, device, stream);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
