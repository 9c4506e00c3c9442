// Attention of several new tokens per sequence over a paged cache, split over the length, on
// the Blackwell tensor cores (tcgen05 + TMEM) with TMA loads: pa_decode_tree (K and V per
// head) and pa_latent_decode (one row per token, whose first part is the value too).
//
//   out = sum_t p_t V_t / sum_t p_t,   p_t = 2^(s_t - m),   s_t = log2(e) scale q . K_t
//
// over the tokens t that a query token sees: all older ones, and the new ones of its set.
//
// The cache rows are the M side of both products and the columns are (new token, query head)
// pairs of one KV head, so that a tile of the cache is read once for up to 64 of them:
//   S^T[TOK x N] = K_tile . Q^T            O^T[Dv x N] += V_tile^T . P^T
// A thread of the softmax has a few columns in a few rows (tokens): sums over tokens stay in
// its registers until the item ends.  The running maximum of a column is raised only where a
// tile exceeds it by more than 2^8, or holds the first score of a column that has none yet (a
// drafted token need not see anything of the tile that a segment begins with), which one vote a
// tile finds out; only then, and in a segment's first tile, the column maxima are reduced over
// the tokens and O is rescaled.
//
// A tile stands in shared memory as the TMA unit writes it, [8-token group][64-element slab]
// [8 tokens][128 bytes] with the 128-byte swizzle, one copy to a block of any size.  The same
// bytes are K-major for S (group stride between its 8-row groups) and MN-major for O.
//
// Work: the tiles of all (sequence, KV head, pair of column groups) items in a row, cut into
// windows of equal cost (pa_multi_window.cuh), one to a set of `gs` CTAs: one CTA, or two that
// take the two column groups of a pair and read the same tiles at the same time, the second
// time from L2.  What a window boundary cuts leaves partial (m, l, acc) in the workspace, and
// the join kernel takes the parts together.
//
// Values that a row does not see have no part in it: tokens behind the end are zeroed in
// shared memory.  A new token's V may hold infinities or NaN that only some columns see, and
// 0 times those is no zero: such a row is zeroed too, and what it gives to the columns that
// see it is added by the softmax warps (rare, and as slow as it may be).
//
// Roles: warp 0 block ids and TMA; warp 1 TMEM and MMA issue; warp 2 q; the others, one or
// two groups of four with columns of their own, softmax and output.  Every wait is bounded; one
// that runs out sets an abort flag, copies and MMAs in flight are drained, TMEM is freed and
// PA_ERR_TIMEOUT is reported through status_dev.
//
// Measured (GB300, bf16; of a plain copy's 6.8 TB/s):
//   pa_decode_tree, 64 sequences of 128..4,096, 16 drafted, 32/8 heads of 128: 106-108 us, 5.35
//     TB/s, 0.79; one of 50,001, 60 drafted, 40/8: 147 us; 4 short ones of 4 heads: 7.7 us
//   pa_latent_decode, 64 sequences of 128..4,096, 128 heads: 78 us; 8 of 32,768..131,072, 16
//     heads, 3 drafted: 138 us, 5.5 TB/s, 0.80; 4 short ones of 16 heads, latent 256: 7.4 us
// From its release a CTA takes 12,000 (trees) to 14,600 cycles (128 heads) to its first tile, 4,700
// of them for its window; from its last product to its last store 900 (trees) to 4,500 (latent
// 512); the join of many parts takes 6.5 to 11 us.  In between trees and long latent sequences
// run at the memory's rate, 128 heads at 3,300 cycles a tile (the operands' reads from shared
// memory: 2,000).  A call of few short sequences is 12,100 cycles in all.
// Tried: tiles of 64 tokens for head_dim 128 (tree 138 us, was 125), a latent tile in halves (82,
// was 80), the second product always first (218, was 190), polls of tile and weights at once
// (they take the softmax's issue slots).
#pragma once

#include <math.h>
#include <math_constants.h>

#include <mutex>

#include "pa_common.cuh"
#include "pa_multi_window.cuh"
#include "pa_q8.cuh"
#include "pa_sm100.cuh"

namespace pa {
namespace multi {

using namespace sm100;

constexpr int kMaxCtas = 160;                  // CTAs at most (one per SM; GB300: 152)
constexpr uint64_t kLimitNs = 2000000000ull;
constexpr unsigned kAll = 0xFFFFFFFFu;
// cost of an item's ends, in quarters of a tile (16-token trees of 64 sequences: with 4 139 us,
// 8 129, 12 127, 16 126)
constexpr int kEnds = 12;
constexpr int kWidest = 64;                    // columns of a product
constexpr float kRaise = 8.f;                  // log2 by which a tile may exceed the maximum

struct Args {
  void* out;
  const void* v_src;             // the pool whose rows hold the values
  const int32_t* tables;
  const int32_t* lens;
  const int32_t* q_start;
  const int32_t* mask;
  int B, total_q, Hq, H, G, bs_shift, max_blocks, num_blocks, max_q, words, max_len;
  // columns of a group: gh heads of gn new tokens each; a KV head's heads are `chunks` of gh
  int gh, gn, chunks;
  int gs;                        // CTAs of a set, 1 or 2: column groups of an item
  int narrow;                    // costs fit 32 bits
  float scale_log2;
  Window* info;                  // [sets]
  float* ws_m;                   // [2 CTAs, N]
  float* ws_l;
  float* ws_acc;                 // [2 CTAs, N, Dv]
  int32_t* status_dev;
};

// Layout of one kernel.  TOK: tokens of a tile; QS: 64-element slabs of a key; VS: of a value;
// SHARED: the value is the key's first slabs (one tile holds both), else V has tiles of its
// own; N: columns; TERMS: storage-type terms of a softmax weight.
template <int TOK_, int QS_, int VS_, bool SHARED_, int N_, int TERMS_>
struct Shape {
  static constexpr int TOK = TOK_, QS = QS_, VS = VS_, N = N_, TERMS = TERMS_;
  static constexpr bool SHARED = SHARED_;
  static constexpr int DV = 64 * VS;
  static constexpr int VM = VS == 1 ? 64 : 128;          // rows of O^T in one product
  static constexpr int VT = DV / VM;
  static constexpr int GS = QS * 1024;                   // bytes between 8-token groups
  static constexpr int VGS = SHARED ? GS : VS * 1024;
  // softmax warpgroups, each with columns of its own
  static constexpr int GROUPS = N >= 32 ? 2 : 1;
  static constexpr int NC = N / GROUPS;
  static constexpr int kThreads = 96 + 128 * GROUPS;
  static constexpr int UNIT = TOK / 8 * GS;              // a tile of K (and V)
  static_assert(SHARED || VS == QS, "K and V tiles of one size share a ring");
  static constexpr int QBYTES = N * QS * 128;
  // the second term stands in the other half of a weight row, or in rows of its own
  static constexpr int PBYTES = SHARED ? 0 : TOK * 128 * (TERMS == 2 && N > 32 ? 2 : 1);
  static constexpr int kTailBytes = 6144;
  static constexpr int kBudget = 232448 - 1024 - kTailBytes;
  // two q operands where they leave room for as many tiles
  static constexpr int units_with(int qbufs) {
    return (kBudget - qbufs * QBYTES - 2 * PBYTES) / UNIT;
  }
  static constexpr int QBUFS = units_with(2) >= (SHARED ? 2 : 5) ? 2 : 1;
  static constexpr int RING = units_with(QBUFS) > 8 ? 8 : units_with(QBUFS);
  static_assert(RING >= (SHARED ? 2 : 3), "ring too shallow");
  static constexpr int kQOff = RING * UNIT;
  static constexpr int kPOff = kQOff + QBUFS * QBYTES;
  static constexpr int kTailOff = kPOff + 2 * PBYTES;
  static constexpr int kSmem = kTailOff + kTailBytes + 1024;
  static constexpr int kUsedCols = (2 + VT) * N;
  static constexpr uint32_t kCols =
      kUsedCols <= 32 ? 32 : (kUsedCols <= 64 ? 64 : (kUsedCols <= 128 ? 128
                                                      : (kUsedCols <= 256 ? 256 : 512)));
  static_assert(kUsedCols <= 512 && kSmem <= 232448, "fits an SM");
};

template <class S>
struct Tail {
  uint64_t full[8], empty[8];
  uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], o_free, drain;
  int64_t lin[2];                // the window's first tile, and the next one's
  int64_t sums[S::kThreads / 32][2];
  Window start;
  alignas(16) int out_row[S::N]; // a column's row of out, -1: none
  int query[S::N];               // its new token, -1: none
  uint32_t seen[S::N][S::TOK / 32];        // what it sees of a tile, a bit of a token
  alignas(16) float by[S::N];    // 2^(maximum before - now), then 1 / the weights' sum
  float red[4][S::N];            // per warp: columns' maxima
  float sum[4][S::N];            // per warp: columns' sums of weights
  float share[S::N];             // weights of a row whose values are added apart, -1: unseen
  uint32_t odd[S::GROUPS][4];    // such rows of a tile, a word of a warp
  uint32_t tmem;
  int abort_flag;
};

struct Seq {
  int L, n, qs, nt, items;
};

// Column groups of n new tokens.
__device__ __forceinline__ int groups_of(const Args& a, int n) {
  return (n + a.gn - 1) / a.gn * a.chunks;
}

// A sequence's lengths and work; nt 0: none.  *bad: it is skipped and reported.
template <class S>
__device__ __forceinline__ Seq seq_of(const Args& a, int b, bool* bad) {
  Seq s;
  s.L = a.lens[b];
  s.qs = b;
  s.n = 1;
  if (a.q_start) {
    s.qs = a.q_start[b];
    s.n = a.q_start[b + 1] - s.qs;
  }
  *bad = s.L < 0 || s.L > a.max_len ||
         (int64_t)s.L > ((int64_t)a.max_blocks << a.bs_shift) || s.qs < 0 || s.n < 0 ||
         s.n > a.max_q || s.n > a.total_q - s.qs || (a.q_start && s.n > s.L);
  s.nt = *bad || s.n == 0 ? 0 : (s.L + S::TOK - 1) / S::TOK;
  s.items = s.nt == 0 ? 0 : a.H * ((groups_of(a, s.n) + a.gs - 1) >> (a.gs - 1));
  return s;
}

// The window of a set, by the whole CTA: tail->start and tail->lin.
template <class S, class I>
__device__ __forceinline__ void find_window(const Args& a, Tail<S>* tail, int set, int sets) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = (a.B + S::kThreads - 1) / S::kThreads;
  Share<I> share;
  share.b0 = min(a.B, tid * per);
  share.b1 = min(a.B, share.b0 + per);
  share.tiles = share.items = 0;
  auto work_of = [&](int b) {
    bool bad;
    const Seq s = seq_of<S>(a, b, &bad);
    return Work{s.nt, s.items};
  };
  for (int b = share.b0; b < share.b1; ++b) {
    const Work w = work_of(b);
    share.tiles += (I)w.nt * w.items;
    share.items += w.items;
  }
  share.tiles_to = share.tiles;
  share.items_to = share.items;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const I t = __shfl_up_sync(kAll, share.tiles_to, o);
    const I n = __shfl_up_sync(kAll, share.items_to, o);
    if (lane >= o) {
      share.tiles_to += t;
      share.items_to += n;
    }
  }
  I (*sums)[2] = reinterpret_cast<I (*)[2]>(tail->sums);
  if (lane == 31) {
    sums[warp][0] = share.tiles_to;
    sums[warp][1] = share.items_to;
  }
  share.tiles_to -= share.tiles;
  share.items_to -= share.items;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  I tiles = 0, items = 0;
#pragma unroll
  for (int w = 0; w < S::kThreads / 32; ++w) {
    if (w < warp) {
      share.tiles_to += sums[w][0];
      share.items_to += sums[w][1];
    }
    tiles += sums[w][0];
    items += sums[w][1];
  }
  const Cut<I> cut = cut_of(tiles, items, sets, kEnds);
  if (set < cut.windows) {
    Place<I> p;
    if (place_of(cut, share, a.B, bound_of(cut, set), work_of, &p)) {
      tail->start = Window{p.b, p.item, p.j, 0};
      tail->lin[0] = p.lin;
    }
    if (set + 1 == cut.windows) {
      if (tid == 0) tail->lin[1] = cut.tiles;
    } else if (place_of(cut, share, a.B, bound_of(cut, set + 1), work_of, &p)) {
      tail->lin[1] = p.lin;
    }
  } else if (tid == 0) {
    tail->start = Window{0, -1, -1, 0};
    tail->lin[0] = tail->lin[1] = 0;
  }
  __syncthreads();
}

// Walks the segments of a window: its part of one item after another.
struct Segment {
  int b, h, i0, g0, j0, j1, nt, L, n, qs;       // i0, g0: the group's first token and head
  int part;                      // 0: the window's first segment, else 1
  bool active;                   // the CTA's column group has a column
};

template <class S>
struct Walk {
  Seq s;
  int b, item, j, left, part;

  __device__ __forceinline__ bool next(const Args& a, int r, Segment* g) {
    if (left <= 0) return false;
    while (j >= s.nt || item >= s.items) {
      j = 0;
      if (++item >= s.items) {
        item = 0;
        do {
          if (++b >= a.B) {
            left = 0;
            return false;
          }
          bool bad;
          s = seq_of<S>(a, b, &bad);
        } while (s.items == 0);
      }
    }
    const int pairs = s.items / a.H;
    g->b = b;
    g->h = item / pairs;
    const int group = (item - g->h * pairs) * a.gs + r, i = group / a.chunks;
    g->i0 = i * a.gn;
    g->g0 = (group - i * a.chunks) * a.gh;
    g->active = g->i0 < s.n;
    g->j0 = j;
    g->j1 = s.nt - j <= left ? s.nt : j + left;
    g->nt = s.nt;
    g->L = s.L;
    g->n = s.n;
    g->qs = s.qs;
    g->part = part;
    part = 1;
    left -= g->j1 - j;
    j = g->j1;
    return true;
  }
};

// One block of the cache to shared memory: [8-token groups][slabs][8][64].
__device__ __forceinline__ void tma_block(void* dst, const CUtensorMap* map, uint64_t* bar,
                                          int group, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(0), "r"(0), "r"(0),
      "r"(group), "l"(policy)
      : "memory");
}

__device__ __forceinline__ void tma_block_head(void* dst, const CUtensorMap* map, uint64_t* bar,
                                               int group, int h, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5, %6, %7}], [%2], %8;" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(0), "r"(0), "r"(0),
      "r"(group), "r"(h), "l"(policy)
      : "memory");
}

// The same block to L2 only.
__device__ __forceinline__ void prefetch_block(const CUtensorMap* map, int group, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.prefetch.tensor.4d.L2.global.tile.L2::cache_hint [%0, {%1, %2, %3, %4}], "
      "%5;" ::"l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(0), "r"(0), "r"(group), "l"(policy)
      : "memory");
}

// One slab of q: [new tokens][heads][64].
__device__ __forceinline__ void tma_q(void* dst, const CUtensorMap* map, uint64_t* bar, int head,
                                      int row, int slab) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(0), "r"(head), "r"(row),
      "r"(slab)
      : "memory");
}

// Has the phase of this parity completed?  Does not wait.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Is any of `count` threads' predicates true?
__device__ __forceinline__ bool any_of(int id, int count, bool x) {
  uint32_t y;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(y)
      : "r"(id), "r"(count), "r"((uint32_t)x)
      : "memory");
  return y != 0;
}

// 16 lanes x NC columns of tensor memory over a warp: of every eight columns lane l gets
// columns 2 (l % 4) and the next one of row l / 4, then of row l / 4 + 8.
template <int NC>
__device__ __forceinline__ void load_scores(uint32_t t, float (&v)[NC / 8][4]) {
  uint32_t r[NC / 2];
  if constexpr (NC == 32) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(t)
        : "memory");
  } else {
    static_assert(NC == 16, "columns of a softmax group");
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7])
        : "r"(t)
        : "memory");
  }
#pragma unroll
  for (int i = 0; i < NC / 2; ++i) v[i / 4][i % 4] = __uint_as_float(r[i]);
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

template <class S, int DT>
__global__ void __launch_bounds__(S::kThreads, 1)
multi_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
             const __grid_constant__ CUtensorMap map_q, const Args a) {
  constexpr int N = S::N, R = S::RING, QB = S::QBUFS, TOK = S::TOK, kThreads = S::kThreads;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  static_assert(sizeof(Tail<S>) <= S::kTailBytes, "barrier block");
  Tail<S>* tail = reinterpret_cast<Tail<S>*>(smem + S::kTailOff);
  volatile int* abort_flag = &tail->abort_flag;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(kAll, tid >> 5, 0);           // uniform, and known to be
  const int set = (int)blockIdx.x / a.gs, r = (int)blockIdx.x - set * a.gs;
  const int sets = (int)gridDim.x / a.gs;

  allow_next_grid();
  if (tid == 0) {
    for (int i = 0; i < R; ++i) {
      mbar_init(&tail->full[i], 1);
      mbar_init(&tail->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tail->q_full[i], 1);
      mbar_init(&tail->q_empty[i], 1);
      mbar_init(&tail->s_full[i], 1);
      mbar_init(&tail->p_full[i], 4 * S::GROUPS);
    }
    mbar_init(&tail->o_free, 4 * S::GROUPS);
    mbar_init(&tail->drain, 1);
    tail->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&map_k);
    if (!S::SHARED) tma_prefetch_desc(&map_v);
    tma_prefetch_desc(&map_q);
  }
  if (warp == 1) {
    tmem_alloc(&tail->tmem, S::kCols);
    tmem_relinquish();
  }
  // rows of q that no copy writes
  if (a.gh * a.gn < N) {
    for (int i = tid; i < QB * S::QBYTES / 16; i += kThreads)
      reinterpret_cast<uint4*>(smem + S::kQOff)[i] = make_uint4(0, 0, 0, 0);
    fence_async_smem();
  }
  wait_prior_grid();

  // this set's window
  if (a.narrow) find_window<S, int>(a, tail, set, sets);
  else find_window<S, int64_t>(a, tail, set, sets);
  Walk<S> walk;
  walk.b = tail->start.b;
  walk.item = tail->start.item;
  walk.j = tail->start.j;
  walk.left = (int)(tail->lin[1] - tail->lin[0]);
  walk.part = 0;
  if (tid == 0 && r == 0) a.info[set] = Window{walk.b, walk.item, walk.j, walk.left};
  walk.s = Seq{};
  if (walk.left > 0) {
    bool bad;
    walk.s = seq_of<S>(a, walk.b, &bad);
  }
  const uint32_t tmem = tail->tmem, ocol = tmem + 2 * N;
  const uint32_t ring = smem_addr(smem), qb = smem_addr(smem + S::kQOff);
  Segment g;
  bool ok = true;

  if (warp == 0) {
    // ------------------------------------------------------------ block ids, TMA --
    // read again by the other column groups of the item, else once
    const uint64_t policy = a.gs > 1 ? policy_evict_last() : policy_evict_first();
    const int bs = 1 << a.bs_shift, per_tile = TOK >> a.bs_shift;
    const int outside = a.num_blocks << a.bs_shift >> 3;        // such a copy reads zeros
    int u = 0;
    while (ok && walk.next(a, r, &g)) {
      if (!g.active) continue;
      const int32_t* table = a.tables + (int64_t)g.b * a.max_blocks;
      auto id_of = [&](int j) {
        return lane < per_tile && (int64_t)j * TOK + lane * bs < g.L ? table[j * per_tile + lane]
                                                                     : -1;
      };
      int id = id_of(g.j0);
      for (int j = g.j0; j < g.j1 && ok; ++j) {
        const int nb = (min(TOK, g.L - j * TOK) + bs - 1) >> a.bs_shift;
        int group = outside;
        if (lane < nb) {
          if (id >= 0 && id < a.num_blocks) group = id << a.bs_shift >> 3;
          else report(a.status_dev, PA_ERR_BAD_BLOCK_ID);
        }
        if (j + 1 < g.j1) id = id_of(j + 1);
#pragma unroll
        for (int kv = 0; kv < (S::SHARED ? 1 : 2); ++kv) {
          const int stage = u % R;
          if (lane == 0) {
            ok = mbar_wait(&tail->empty[stage], ((u / R) & 1) ^ 1, abort_flag, kLimitNs);
            if (ok) mbar_arrive_expect_tx(&tail->full[stage], (uint32_t)((nb * bs >> 3) * S::GS));
          }
          ok = __shfl_sync(kAll, (int)ok, 0) != 0;
          if (!ok) break;
          if (lane < nb) {
            uint8_t* dst = smem + stage * S::UNIT + (lane * bs >> 3) * S::GS;
            if (S::SHARED) tma_block(dst, &map_k, &tail->full[stage], group, policy);
            else tma_block_head(dst, kv ? &map_v : &map_k, &tail->full[stage], group, g.h, policy);
          }
          ++u;
        }
        // With two tiles of shared memory a copy's time is in the way: the next tile's blocks are
        // brought to L2, from where they come in half the time (the first two tiles are asked for
        // at once).
        if (S::SHARED && j > g.j0 && id >= 0 && id < a.num_blocks &&
            (a.gs == 1 || (lane & 1) == r) && j + 1 < g.j1)
          prefetch_block(&map_k, id << a.bs_shift >> 3, policy);
      }
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      report(a.status_dev, PA_ERR_TIMEOUT);
    }
    if (*abort_flag && lane == 0) {             // copies in flight land before the CTA ends
      for (int i = max(0, u - R); i < u; ++i)
        mbar_wait_drain(&tail->full[i % R], (i / R) & 1, kLimitNs);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issue --
    // K . q of tile t, then V . p of tile t - 1, so that the softmax of a tile runs while the
    // tensor cores have the next one's scores; but where the next tile is still on its way, the
    // product goes first and frees the ring for the one behind it.
    // Descriptors are built once a tile and stepped by constants (the start-address field holds
    // address / 16), and the whole warp runs along, so that they stay uniform.
    constexpr uint32_t ab = DT == PA_BFLOAT16 ? 1u : 0u;
    constexpr uint32_t idesc_s = idesc_f16(ab, 0, 0, TOK, N);
    constexpr uint32_t idesc_o = idesc_f16(ab, 1, 1, S::VM, N);
    constexpr int PGS = S::SHARED ? S::GS : 1024;
    {
      int t = 0, seg = 0;
      bool prev_first = false;
      int prev_seg = 0;
      auto wait = [&](uint64_t* bar, int parity) -> bool {
        return __all_sync(kAll, mbar_wait(bar, parity, abort_flag, kLimitNs));
      };
      auto issue_pv = [&](int p) -> bool {
        const int u = S::SHARED ? p : 2 * p + 1, slot = p & 1;
        // the weights are there, and with them: S of tile p is read
        if ((!S::SHARED && !wait(&tail->full[u % R], (u / R) & 1)) ||
            !wait(&tail->p_full[slot], (p >> 1) & 1) ||
            (prev_first && prev_seg > 0 && !wait(&tail->o_free, (prev_seg - 1) & 1)))
          return false;
        tc_fence_after();
        const uint32_t va = ring + (u % R) * S::UNIT;
        const uint64_t vd = smem_desc_sw128(va, 1024, S::VGS);
        const uint64_t pd = smem_desc_sw128(S::SHARED ? va + (S::QS - 1) * 1024
                                                      : smem_addr(smem + S::kPOff) +
                                                            slot * S::PBYTES,
                                            1024, PGS);
        uint32_t more = !prev_first;
#pragma unroll
        for (int k = 0; k < TOK / 16; ++k)
#pragma unroll
          for (int term = 0; term < S::TERMS; ++term) {
#pragma unroll
            for (int v = 0; v < S::VT; ++v)
              mma_by_one(ocol + v * N,
                      vd + (uint64_t)((v * (S::VM / 64) * 1024 + k * 2 * S::VGS) >> 4),
                      pd + (uint64_t)((k * 2 * PGS + term * (N > 32 ? TOK * 128 : 64)) >> 4),
                      idesc_o, more);
            more = 1;
          }
        commit_by_one(&tail->empty[u % R]);
        return true;
      };
      while (ok && walk.next(a, r, &g)) {
        if (!g.active) continue;
        const int qs = seg % QB;
        for (int j = g.j0; j < g.j1 && ok; ++j) {
          const int u = S::SHARED ? t : 2 * t;
          const bool first = j == g.j0;
          bool left = t > 0;                     // the product of tile t - 1 is not issued
          // Scores of tile t go first only if the tile and q are there by now: they take
          // longer than the softmax that the product of tile t - 1 waits for.
          if (left && !(__all_sync(kAll, mbar_test(&tail->full[u % R], (u / R) & 1)) &&
                        (!first ||
                         __all_sync(kAll, mbar_test(&tail->q_full[qs], (seg / QB) & 1))))) {
            ok = issue_pv(t - 1);
            left = false;
          }
          ok = ok && wait(&tail->full[u % R], (u / R) & 1) &&
               (!first || wait(&tail->q_full[qs], (seg / QB) & 1));
          if (!ok) break;
          tc_fence_after();
          const uint64_t kd = smem_desc_sw128(ring + (u % R) * S::UNIT, 16, S::GS);
          const uint64_t qd = smem_desc_sw128(qb + qs * S::QBYTES, 16, 1024);
          const uint32_t scol = tmem + (t & 1) * N;
#pragma unroll
          for (int k = 0; k < 4 * S::QS; ++k)
            mma_by_one(scol, kd + (uint64_t)(((k >> 2) * 1024 + (k & 3) * 32) >> 4),
                    qd + (uint64_t)(((k >> 2) * (N * 128) + (k & 3) * 32) >> 4), idesc_s, k > 0);
          if (!S::SHARED) commit_by_one(&tail->empty[u % R]);
          commit_by_one(&tail->s_full[t & 1]);
          if (j + 1 == g.j1) commit_by_one(&tail->q_empty[qs]);
          if (left) ok = issue_pv(t - 1);
          prev_first = first;
          prev_seg = seg;
          ++t;
        }
        ++seg;
      }
      if (ok && t > 0) ok = issue_pv(t - 1);
      if (!ok && lane == 0) {
        *abort_flag = 1;
        report(a.status_dev, PA_ERR_TIMEOUT);
      }
      // every product and commit issued here ends before TMEM is freed
      if (t > 0) {
        commit_by_one(&tail->drain);
        mbar_wait_drain(&tail->drain, 0, kLimitNs);
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    // ----------------------------------------------------------------------- q --
    int seg = 0;
    while (ok && walk.next(a, r, &g)) {
      if (!g.active) continue;
      const int slot = seg % QB;
      if (seg >= QB) {
        ok = mbar_wait(&tail->q_empty[slot], (seg / QB - 1) & 1, abort_flag, kLimitNs);
        ok = __all_sync(kAll, ok);
        if (!ok) break;
      }
      if (lane == 0) {
        mbar_arrive_expect_tx(&tail->q_full[slot], (uint32_t)(S::QS * a.gh * a.gn * 128));
        for (int x = 0; x < S::QS; ++x)
          tma_q(smem + S::kQOff + slot * S::QBYTES + x * (N * 128), &map_q, &tail->q_full[slot],
                g.h * a.G + g.g0, g.qs + g.i0, x);
      }
      __syncwarp();
      ++seg;
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      report(a.status_dev, PA_ERR_TIMEOUT);
    }
    if (*abort_flag && lane == 0) {             // copies in flight land before the CTA ends
      for (int i = max(0, seg - QB); i < seg; ++i)
        mbar_wait_drain(&tail->q_full[i % QB], (i / QB) & 1, kLimitNs);
    }
    // sequences without work: empty ones of a step without q_start, and bad ones
    for (int b = (int)blockIdx.x; b < a.B; b += (int)gridDim.x) {
      bool bad;
      const Seq s = seq_of<S>(a, b, &bad);
      if (bad) {
        if (lane == 0) report(a.status_dev, PA_ERR_BAD_BLOCK_ID);
      } else if (!a.q_start && s.L == 0) {
        uint4* row = static_cast<uint4*>(a.out) + (int64_t)b * a.Hq * (S::DV / 8);
        for (int i = lane; i < a.Hq * (S::DV / 8); i += 32) row[i] = make_uint4(0, 0, 0, 0);
      }
    }
  } else {
    // ------------------------------------------------ softmax and output rows --
    // A group of four warps has NC columns of every tile.  A thread holds, of every eight of
    // them, two in the rows (tokens) lane / 4 + 8 i of its warp: what belongs to a column stays
    // in registers.
    constexpr int NC = S::NC, HALVES = TOK / 64, K = NC / 4;
    const int wq = warp & 3;                     // TMEM lane quarter of this warp
    const int grp = (warp - 3) >> 2, c_lo = grp * NC;
    const int st = (tid - 96) & 127;             // thread of the group
    const uint32_t quarter = (uint32_t)(wq * 32) << 16;
    const int row0 = wq * (TOK / 4) + (lane >> 2);
    const int pair = 2 * (lane & 3);
    // row of element (half, q) and column of element (i, q), k = 2 i + (q & 1)
    auto row_of = [&](int half, int q) { return row0 + 16 * half + 8 * (q >> 1); };
    auto col_of = [&](int k) { return c_lo + 8 * (k >> 1) + pair + (k & 1); };
    const float sl2 = a.scale_log2;
    // fp16 weights stand 2^7 higher: below 2^-14 they would lose bits.  A weight is at most
    // 2^kRaise times that.
    constexpr float kShift = DT == PA_BFLOAT16 ? 0.f : 7.f;
    // of the thread's columns: running maximum, what is added to a score before its power of
    // two, sum of the weights of the thread's rows
    float top[K], neg[K], l[K];
    const uint32_t flag = smem_addr(&tail->abort_flag);
    int t = 0;
    // A wait that runs out, or finds that another's has, ends the waiting and nothing else: the
    // warp goes on through the window, so that every thread meets every barrier of its group (they
    // have no limit of their own), and the window's tiles bound what follows.  Rows of out that
    // end behind that are not stored.
    auto wait_all = [&](uint64_t* bar, int parity) {
      if (!__all_sync(kAll, mbar_try_wait(bar, parity)) &&
          !__all_sync(kAll, mbar_wait_far<kLimitNs>(smem_addr(bar), parity, flag)))
        *abort_flag = 1;
    };
    // V . p of tile i, which frees its V
    auto wait_product = [&](int i) {
      const int u = S::SHARED ? i : 2 * i + 1;
      wait_all(&tail->empty[u % R], (u / R) & 1);
    };
    auto sync = [&]() { named_barrier(1 + grp, 128); };
    // a column's value in all rows of the warp, from its lanes'
    auto over_rows = [&](float x, auto&& f) -> float {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) x = f(x, __shfl_xor_sync(kAll, x, o));
      return x;
    };
    auto larger = [](float x, float y) { return fmaxf(x, y); };
    auto plus = [](float x, float y) { return x + y; };
    while (walk.next(a, r, &g)) {
      if (!g.active) continue;
      const int ctx = g.L - g.n;
      // the columns of this item (those of the one before have been read)
      sync();
      if (st < NC) {
        const int c = c_lo + st, x = c / a.gh, i = g.i0 + x, head = g.g0 + c - x * a.gh;
        const bool live = x < a.gn && i < g.n && head < a.G;
        tail->query[c] = live ? i : -1;
        tail->out_row[c] = live ? (g.qs + i) * a.Hq + g.h * a.G + head : -1;
      }
      sync();
      for (int j = g.j0; j < g.j1; ++j, ++t) {
        const bool first = j == g.j0, last = j + 1 == g.j1;
        const int u = S::SHARED ? t : 2 * t + 1;              // the tile of V
        const bool edge = (j + 1) * TOK > ctx;               // new tokens, or behind the end
        if (edge && st < NC) {
          // what a column sees of this tile: of each 32 tokens the older ones, the new ones of
          // its set, none behind the end
          const int i = tail->query[c_lo + st];
          const int32_t* set = a.mask + (int64_t)(g.qs + max(i, 0)) * a.words;
#pragma unroll
          for (int w = 0; w < TOK / 32; ++w) {
            const int lo = j * TOK + 32 * w - ctx;           // the new token of bit 0
            const int ends_at = g.L - j * TOK - 32 * w;
            uint32_t bits;
            if (a.mask) {
              // words x and x + 1 of the set, from bit lo - 32 x on
              const int x = lo >> 5;
              const uint32_t w0 = x < 0 ? kAll : (x < a.words ? (uint32_t)set[x] : 0u);
              const uint32_t w1 = x + 1 < 0 ? kAll : (x + 1 < a.words ? (uint32_t)set[x + 1] : 0u);
              bits = __funnelshift_r(w0, w1, lo & 31);
            } else {
              const int n = i + 1 - lo;                      // a chain: new tokens up to i
              bits = n <= 0 ? 0u : (n >= 32 ? kAll : (1u << n) - 1);
            }
            if (lo < 0) bits |= lo <= -32 ? kAll : (1u << -lo) - 1;
            if (ends_at < 32) bits &= ends_at <= 0 ? 0u : (1u << ends_at) - 1;
            tail->seen[c_lo + st][w] = bits;
          }
        }
        wait_all(&tail->s_full[t & 1], (t >> 1) & 1);
        tc_fence_after();
        if (edge) sync();
        float s[HALVES][NC / 8][4];
#pragma unroll
        for (int hf = 0; hf < HALVES; ++hf)
          load_scores<NC>(tmem + quarter + ((uint32_t)(16 * hf) << 16) + (t & 1) * N + c_lo, s[hf]);
        const uint64_t scale2 = f2_pack(sl2, sl2);
#pragma unroll
        for (int hf = 0; hf < HALVES; ++hf)
#pragma unroll
          for (int i = 0; i < NC / 8; ++i)
#pragma unroll
            for (int q = 0; q < 4; q += 2)
              f2_unpack(mul2(f2_pack(s[hf][i][q], s[hf][i][q + 1]), scale2), s[hf][i][q],
                        s[hf][i][q + 1]);
        if (edge) {
#pragma unroll
          for (int k = 0; k < K; ++k) {
            // the thread's rows stand in one word
            const uint32_t bits = tail->seen[col_of(k)][row0 >> 5] >> (row0 & 31);
#pragma unroll
            for (int hf = 0; hf < HALVES; ++hf) {
              if (!(bits >> (16 * hf) & 1)) s[hf][k >> 1][k & 1] = -CUDART_INF_F;
              if (!(bits >> (16 * hf + 8) & 1)) s[hf][k >> 1][2 + (k & 1)] = -CUDART_INF_F;
            }
          }
        }
        // the largest of a column in the thread's rows
        float most[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
          float m = fmaxf(s[0][k >> 1][k & 1], s[0][k >> 1][2 + (k & 1)]);
          if (HALVES == 2)
            m = fmax3(m, s[HALVES - 1][k >> 1][k & 1], s[HALVES - 1][k >> 1][2 + (k & 1)]);
          most[k] = m;
        }
        bool raise = first;
        if (!first) {
          bool over = false;
#pragma unroll
          for (int k = 0; k < K; ++k) over = over || most[k] > top[k] + kRaise;  // also of -inf
          raise = any_of(1 + grp, 128, over);
        }
        if (raise) {
#pragma unroll
          for (int k = 0; k < K; ++k) {
            const float m = over_rows(most[k], larger);
            if (lane < 4) tail->red[wq][col_of(k)] = m;
          }
          sync();
          float by[K];
#pragma unroll
          for (int k = 0; k < K; ++k) {
            const int c = col_of(k);
            const float before = first ? -CUDART_INF_F : top[k];
            top[k] = fmaxf(before, fmaxf(fmaxf(tail->red[0][c], tail->red[1][c]),
                                         fmaxf(tail->red[2][c], tail->red[3][c])));
            neg[k] = (top[k] == -CUDART_INF_F ? 0.f : -top[k]) + kShift;
            by[k] = before == -CUDART_INF_F ? 0.f : ex2_approx(before - top[k]);
            l[k] = first ? 0.f : l[k] * by[k];
          }
          if (!first) {
            if (wq == 0 && lane < 4) {
#pragma unroll
              for (int k = 0; k < K; ++k) tail->by[col_of(k)] = by[k];
            }
            sync();
            // O (complete up to the tile before; this one's product waits for its weights)
            wait_product(t - 1);
            tc_fence_after();
#pragma unroll 1
            for (int v = 0; v < S::VT; ++v)
#pragma unroll 1
              for (int c0 = c_lo; c0 < c_lo + NC; c0 += 16) {
                float o[16];
                tmem_ld16(ocol + quarter + v * N + c0, o);
                uint32_t w[16];
#pragma unroll
                for (int c = 0; c < 16; ++c) w[c] = __float_as_uint(o[c] * tail->by[c0 + c]);
                tmem_st16_nowait(ocol + quarter + v * N + c0, w);
              }
            tmem_wait_st();
          }
        }
        // weights: to shared memory as rows of 64 columns, N-major, in storage-type terms
        constexpr int PGS = S::SHARED ? S::GS : 1024;
        uint8_t* weights = S::SHARED ? smem + (u % R) * S::UNIT + (S::QS - 1) * 1024
                                     : smem + S::kPOff + (t & 1) * S::PBYTES;
#pragma unroll
        for (int hf = 0; hf < HALVES; ++hf)
#pragma unroll
          for (int q = 0; q < 4; q += 2) {
            const int row = row_of(hf, q);
            uint8_t* prow = weights + (row >> 3) * PGS + (row & 7) * 128 + (lane & 3) * 4;
#pragma unroll
            for (int i = 0; i < NC / 8; ++i) {
              float x, y;
              f2_unpack(f2_add(f2_pack(s[hf][i][q], s[hf][i][q + 1]),
                               f2_pack(neg[2 * i], neg[2 * i + 1])), x, y);
              x = ex2_approx(x);
              y = ex2_approx(y);
              l[2 * i] += x;
              l[2 * i + 1] += y;
              s[hf][i][q] = x;
              s[hf][i][q + 1] = y;
              const int chunk = (c_lo >> 3) + i;
              uint32_t* hi = reinterpret_cast<uint32_t*>(prow + ((chunk ^ (row & 7)) << 4));
              if (S::TERMS == 1) {
                *hi = pack2<DT>(x, y);
              } else {
                uint32_t* lo = reinterpret_cast<uint32_t*>(
                    N > 32 ? prow + TOK * 128 + ((chunk ^ (row & 7)) << 4)
                           : prow + (((chunk + 4) ^ (row & 7)) << 4));
                split2<DT>(x, y, hi, lo);
              }
            }
          }
        // V of tokens behind the end, and of new tokens that not every column sees.  A row's
        // slabs are shared out to the threads that look at it.
        const bool ends = (j + 1) * TOK > g.L;
        const bool fresh = (g.n > 1 || a.mask) && (j + 1) * TOK > ctx;
        bool apart = false;
        if (ends || fresh) {
          wait_all(&tail->full[u % R], (u / R) & 1);
          constexpr int SIDES = TOK == 64 ? 2 : 1, PARTS = SIDES * S::GROUPS;
          const int row = TOK == 64 ? wq * 16 + (lane & 15) : wq * 32 + lane;
          const int mine = grp * SIDES + (TOK == 64 ? lane >> 4 : 0), tok = j * TOK + row;
          uint8_t* vrow = smem + (u % R) * S::UNIT + (row >> 3) * S::VGS + (row & 7) * 128;
          // lanes side by side over the banks
          auto at = [&](int x) { return vrow + (x >> 3) * 1024 + ((x ^ row) & 7) * 16; };
          bool zero = tok >= g.L;
          if (fresh) {
            bool odd = false;
            if (tok >= ctx && tok < g.L) {
#pragma unroll 4
              for (int x = mine; x < 8 * S::VS; x += PARTS) {
                const uint4 w = *reinterpret_cast<const uint4*>(at(x));
                odd = odd || odd2<DT>(w.x) || odd2<DT>(w.y) || odd2<DT>(w.z) || odd2<DT>(w.w);
              }
            }
            const uint32_t rows = __ballot_sync(kAll, odd);
            if (lane == 0) tail->odd[grp][wq] = rows;
            apart = any_of(3, 128 * S::GROUPS, odd);
            if (apart) {
              uint32_t both = 0;
#pragma unroll
              for (int i = 0; i < S::GROUPS; ++i) both |= tail->odd[i][wq];
              if (TOK == 64) both |= both >> 16;
              zero = zero || (both >> (row & (TOK / 4 - 1)) & 1);
            }
          }
          if (zero) {
#pragma unroll 4
            for (int x = mine; x < 8 * S::VS; x += PARTS)
              *reinterpret_cast<uint4*>(at(x)) = make_uint4(0, 0, 0, 0);
          }
        }
        fence_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tail->p_full[t & 1]);
        if (apart) {
          // o += p v for each such row, where the column sees it
          wait_product(t);
          tc_fence_after();
#pragma unroll 1
          for (int w = 0; w < 4; ++w) {
            uint32_t rows = 0;
#pragma unroll
            for (int i = 0; i < S::GROUPS; ++i) rows |= tail->odd[i][w];
            if (TOK == 64) rows = (rows | rows >> 16) & 0xFFFFu;
            while (rows) {
              const int x = w * (TOK / 4) + __ffs(rows) - 1, at = j * TOK + x;
              rows &= rows - 1;
#pragma unroll
              for (int hf = 0; hf < HALVES; ++hf)
#pragma unroll
                for (int i = 0; i < NC / 8; ++i)
#pragma unroll
                  for (int q = 0; q < 4; ++q)
                    if (row_of(hf, q) == x) {
                      const int c = col_of(2 * i + (q & 1));
                      tail->share[c] = tail->seen[c][x >> 5] >> (x & 31) & 1 ? s[hf][i][q] : -1.f;
                    }
              sync();
              const int id = a.tables[(int64_t)g.b * a.max_blocks + (at >> a.bs_shift)];
              // in the pool: a bad block's are zeros, unless its copy has not come
              const int64_t slot = ((int64_t)(id >= 0 && id < a.num_blocks ? id : 0) << a.bs_shift) +
                                   (at & ((1 << a.bs_shift) - 1));
              const uint16_t* vsrc =
                  static_cast<const uint16_t*>(a.v_src) +
                  (S::SHARED ? slot * (64 * S::QS) : (slot * a.H + g.h) * S::DV);
#pragma unroll 1
              for (int v = 0; v < S::VT; ++v) {
                const int dim = v * S::VM + (S::VM == 128 ? wq * 32 + lane : wq * 16 + (lane & 15));
                const float val = widen2<DT>(vsrc[dim]).x;
#pragma unroll 1
                for (int c0 = c_lo; c0 < c_lo + NC; c0 += 16) {
                  float o[16];
                  tmem_ld16(ocol + quarter + v * N + c0, o);
                  uint32_t ow[16];
#pragma unroll
                  for (int c = 0; c < 16; ++c) {
                    const float p = tail->share[c0 + c];
                    ow[c] = __float_as_uint(p == -1.f ? o[c] : fmaf(p, val, o[c]));
                  }
                  tmem_st16_nowait(ocol + quarter + v * N + c0, ow);
                  tmem_wait_st();
                }
              }
              sync();
            }
          }
          tc_fence_before();
          named_barrier(3, 128 * S::GROUPS);     // every thread has read the rows' words
        }
        if (!last) continue;

        // ------------------------------------------------------- the segment's end --
        const bool whole = g.j0 == 0 && g.j1 == g.nt;
        const int64_t part = 2 * (int64_t)blockIdx.x + g.part;
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const float sum = over_rows(l[k], plus);
          if (lane < 4) tail->sum[wq][col_of(k)] = sum;
        }
        if (!whole && wq == 0 && lane < 4) {
#pragma unroll
          for (int k = 0; k < K; ++k) a.ws_m[part * N + col_of(k)] = top[k];
        }
        sync();
        if (st < NC) {
          const int c = c_lo + st;
          const float sum = (tail->sum[0][c] + tail->sum[1][c]) +
                            (tail->sum[2][c] + tail->sum[3][c]);
          tail->by[c] = sum == 0.f ? 0.f : 1.f / sum;
          if (!whole) a.ws_l[part * N + c] = sum;
        }
        wait_product(t);
        sync();
        tc_fence_after();
        const bool has_dim = S::VM == 128 || lane < 16;
        const bool stores = has_dim && !*abort_flag;
        const int dim0 = S::VM == 128 ? wq * 32 + lane : wq * 16 + (lane & 15);
        constexpr int CS = 16;
#pragma unroll 1
        for (int c0 = c_lo; c0 < c_lo + NC; c0 += CS) {
          if (whole) {
            // two lanes exchange halves of two columns: a store of two dims of one column
            float by[CS];
            uint16_t* to[CS / 2];
            bool none = false;                   // a column without weights: zeros
#pragma unroll
            for (int c = 0; c < CS; ++c) by[c] = tail->by[c0 + c];
#pragma unroll
            for (int c = 0; c < CS; c += 2) {
              const int row = tail->out_row[c0 + c + (lane & 1)];
              to[c / 2] = row >= 0 && stores ? static_cast<uint16_t*>(a.out) +
                                                    (int64_t)row * S::DV + (dim0 & ~1)
                                              : nullptr;
              none = none || by[c] == 0.f || by[c + 1] == 0.f;
            }
#pragma unroll 1
            for (int v = 0; v < S::VT; ++v) {
              float o[CS];
              tmem_ld16(ocol + quarter + v * N + c0, o);
#pragma unroll
              for (int c = 0; c < CS; ++c) o[c] *= by[c];
              if (none) {
#pragma unroll
                for (int c = 0; c < CS; ++c) o[c] = by[c] == 0.f ? 0.f : o[c];
              }
#pragma unroll
              for (int c = 0; c < CS; c += 2) {
                const float other = __shfl_xor_sync(kAll, lane & 1 ? o[c] : o[c + 1], 1);
                const uint32_t two =
                    pack2<DT>(lane & 1 ? other : o[c], lane & 1 ? o[c + 1] : other);
                if (to[c / 2]) *reinterpret_cast<uint32_t*>(to[c / 2] + v * S::VM) = two;
              }
            }
          } else {
            float* to = a.ws_acc + (part * N + c0) * S::DV + dim0;
#pragma unroll 1
            for (int v = 0; v < S::VT; ++v) {
              float o[CS];
              tmem_ld16(ocol + quarter + v * N + c0, o);
#pragma unroll
              for (int c = 0; c < CS; ++c)
                if (has_dim && c0 + c < a.gh * a.gn) to[c * S::DV + v * S::VM] = o[c];
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tail->o_free);
      }
    }
    if (*abort_flag && lane == 0) report(a.status_dev, PA_ERR_TIMEOUT);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kCols);
  }
}

// Joins the partials of items that window boundaries cut: CTA (c, r, z) looks at the boundary
// where window c + 1 begins, and joins its share z of the columns of column group r of its item,
// if that boundary is the item's first.  The parts: the segment of window c that ends there,
// then the first segments of the windows behind, as long as they begin inside the item.
// A thread takes four dims of a column and every PS-th part.
constexpr int kJoinThreads = 512;

template <class S, int PS>
struct Join {
  static constexpr int LANES = S::DV / 4;                          // threads of a column
  static constexpr int AT_ONCE = kJoinThreads / LANES / PS;        // columns at once
  // columns of a CTA: with few parts half of them or a quarter, all asked for at once
  static constexpr int COLS = PS > 1 ? AT_ONCE : (S::DV > 256 ? S::N / 4 : S::N / 2);
  static constexpr int ROUNDS = COLS > AT_ONCE ? COLS / AT_ONCE : 1;
};

template <class S, int DT, int PS>
__global__ void __launch_bounds__(kJoinThreads)
join_kernel(const Args a, int sets, int items) {
  using J = Join<S, PS>;
  constexpr int N = S::N, DV = S::DV, LANES = J::LANES, COLS = J::COLS, ROUNDS = J::ROUNDS;
  __shared__ float s_w[COLS][kMaxCtas + 1];
  __shared__ bool s_none[COLS];                            // no weight at all: zeros
  __shared__ float4 s_sum[PS > 1 ? PS : 1][PS > 1 ? COLS * LANES : 1];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = (int)blockIdx.y;
  allow_next_grid();
  wait_prior_grid();
  int c = (int)blockIdx.x + 1;
  bool same;
  if (PS > 1) {                                // the first boundary in item x, if any
    __shared__ int s_c;
    if (tid == 0) s_c = 0;
    __syncthreads();
    if (tid > 0 && tid < sets) {
      const Window w = a.info[tid];
      if (w.b == (int)blockIdx.x / items && w.item == (int)blockIdx.x % items &&
          first_cut(w, a.info[tid - 1], &same))
        s_c = tid;
    }
    __syncthreads();
    c = s_c;
    if (c == 0) return;
  }
  const Window at = a.info[c], before = a.info[c - 1];
  if (!first_cut(at, before, &same)) return;
  bool in = false;
  if (c + 1 + tid < sets) {
    const Window w = a.info[c + 1 + tid];
    in = w.b == at.b && w.item == at.item && w.j > 0 && w.tiles > 0;
  }
  const int parts = 2 + __syncthreads_count(in);
  bool bad;
  const Seq s = seq_of<S>(a, at.b, &bad);
  const int pairs = s.items / a.H, h = at.item / pairs;
  const int group = (at.item - h * pairs) * a.gs + r, i0 = group / a.chunks * a.gn;
  const int g0 = group % a.chunks * a.gh, c0 = (int)blockIdx.z * COLS;
  // columns of this CTA: none, for a group without columns
  const int n = min(COLS, a.gh * min(a.gn, s.n - i0) - c0);
  if (n <= 0) return;
  // row of part k in ws_m and ws_l
  auto row = [&](int k) -> int64_t {
    const int cta = (c - 1 + k) * a.gs + r;
    return (2 * (int64_t)cta + (k == 0 && !same ? 1 : 0)) * N + c0;
  };
  for (int w = warp; w < n; w += kJoinThreads / 32) {
    float top = -CUDART_INF_F, l = 0.f;
    float m0 = -CUDART_INF_F, l0 = 0.f;                    // of the lane's first part
    if (lane < parts) {
      m0 = a.ws_m[row(lane) + w];
      l0 = a.ws_l[row(lane) + w];
      top = m0;
    }
    for (int k = lane + 32; k < parts; k += 32) top = fmaxf(top, a.ws_m[row(k) + w]);
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
    for (int k = lane; k < parts; k += 32) {
      const float m = k < 32 ? m0 : a.ws_m[row(k) + w];
      const float y = top == -CUDART_INF_F ? 0.f : ex2_approx(m - top);
      s_w[w][k] = y;
      l = fmaf(y, k < 32 ? l0 : a.ws_l[row(k) + w], l);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(kAll, l, o);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int k = lane; k < parts; k += 32) s_w[w][k] *= inv;
    if (lane == 0) s_none[w] = l == 0.f;
  }
  __syncthreads();
  const int x = tid % (J::AT_ONCE * LANES), ps = tid / (J::AT_ONCE * LANES);
  const int col = x / LANES, d = (x % LANES) * 4;
  float4 sum[ROUNDS];
#pragma unroll
  for (int i = 0; i < ROUNDS; ++i) sum[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll(ROUNDS > 2 ? 2 : 8)
  for (int k = ps; k < parts; k += PS) {
    const float* acc = a.ws_acc + (row(k) + col) * DV + d;
#pragma unroll
    for (int i = 0; i < ROUNDS; ++i) {
      const int w = col + i * J::AT_ONCE;
      if (w < n) {
        const float y = s_w[w][k];
        const float4 v = *reinterpret_cast<const float4*>(acc + i * J::AT_ONCE * DV);
        sum[i].x = fmaf(y, v.x, sum[i].x);
        sum[i].y = fmaf(y, v.y, sum[i].y);
        sum[i].z = fmaf(y, v.z, sum[i].z);
        sum[i].w = fmaf(y, v.w, sum[i].w);
      }
    }
  }
  if (PS > 1) {
    s_sum[PS > 1 ? ps : 0][PS > 1 ? x : 0] = sum[0];
    __syncthreads();
    if (ps > 0) return;
#pragma unroll
    for (int i = 1; i < PS; ++i) {
      const float4 v = s_sum[i][PS > 1 ? x : 0];
      sum[0].x += v.x;
      sum[0].y += v.y;
      sum[0].z += v.z;
      sum[0].w += v.w;
    }
  }
#pragma unroll
  for (int i = 0; i < ROUNDS; ++i) {
    const int w = col + i * J::AT_ONCE;
    if (w >= n) break;
    const int x0 = (c0 + w) / a.gh, head = g0 + c0 + w - x0 * a.gh;
    const int64_t to = ((int64_t)(s.qs + i0 + x0) * a.Hq + h * a.G + head) * DV + d;
    const float4 y = s_none[w] ? make_float4(0.f, 0.f, 0.f, 0.f) : sum[i];
    if (head < a.G)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + to) =
          make_uint2(pack2<DT>(y.x, y.y), pack2<DT>(y.z, y.w));
  }
}

// ------------------------------------------------------------------ host side --

// A pool [num_blocks, bs, heads, 64 slabs] as [heads][8-token groups][slabs][8 tokens][64]; a
// box is one block of one head.  `heads` 0: of rows without heads.
inline bool encode_blocks(CUtensorMap* map, const void* pool, int dtype, int64_t num_blocks, int bs,
                          int heads, int slabs) {
  const cuuint64_t row = (cuuint64_t)(heads ? heads : 1) * slabs * 128;
  const cuuint64_t dims[5] = {64, 8, (cuuint64_t)slabs, (cuuint64_t)(num_blocks * bs / 8),
                              (cuuint64_t)heads};
  const cuuint64_t strides[4] = {row, 128, 8 * row, (cuuint64_t)slabs * 128};
  const cuuint32_t box[5] = {64, 8, (cuuint32_t)slabs, (cuuint32_t)(bs / 8), 1};
  const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
  return encode_fn()(map,
                     dtype == PA_BFLOAT16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                          : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                     heads ? 5 : 4, const_cast<void*>(pool), dims, strides, box, ones,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Queries [T, heads, 64 slabs] as [slabs][T][heads][64]; a box is a group of columns.
inline bool encode_q(CUtensorMap* map, const void* q, int dtype, int64_t rows, int heads, int slabs,
                     int gh, int gn) {
  const cuuint64_t row = (cuuint64_t)slabs * 128;
  const cuuint64_t dims[4] = {64, (cuuint64_t)heads, (cuuint64_t)rows, (cuuint64_t)slabs};
  const cuuint64_t strides[3] = {row, row * heads, 128};
  const cuuint32_t box[4] = {64, (cuuint32_t)gh, (cuuint32_t)gn, 1}, ones[4] = {1, 1, 1, 1};
  return encode_fn()(map,
                     dtype == PA_BFLOAT16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                          : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                     4, const_cast<void*>(q), dims, strides, box, ones,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How the (new token, query head) pairs of a KV head become columns, by the most new tokens of
// a sequence and the query heads of a KV head: n columns of a product (at most `widest`), of gh
// heads of gn new tokens; gs CTAs to a set.
struct Columns {
  int n, gh, gn, chunks, gs;
};

inline Columns columns_for(int most, int G, int widest = kWidest) {
  Columns c;
  const int64_t all = (int64_t)most * G;
  c.n = all <= 16 ? 16 : (all <= 32 ? 32 : widest);
  c.chunks = (G + c.n - 1) / c.n;
  c.gh = (G + c.chunks - 1) / c.chunks;
  c.gn = c.n / c.gh;
  c.gs = most > c.gn || c.chunks > 1 ? 2 : 1;
  return c;
}

struct Layout {
  size_t m_off, l_off, acc_off, total;
};

inline Layout layout_of(int n, int dv) {
  auto align = [](size_t x) { return (x + 255) & ~(size_t)255; };
  Layout y;
  const size_t rows = (size_t)2 * kMaxCtas * n;
  y.m_off = align(kMaxCtas * sizeof(Window));
  y.l_off = y.m_off + align(rows * sizeof(float));
  y.acc_off = y.l_off + align(rows * sizeof(float));
  y.total = y.acc_off + align(rows * dv * sizeof(float));
  return y;
}

template <class S, int DT>
cudaError_t launch(const CUtensorMap (&maps)[3], const Args& a, int ctas, int64_t items, bool cut,
                   int device, cudaStream_t stream) {
  static std::mutex lock;
  static uint64_t done = 0;                    // devices whose attribute is set
  {
    std::lock_guard<std::mutex> hold(lock);
    if (device >= 64 || !(done >> device & 1)) {
      const cudaError_t e = taken(cudaFuncSetAttribute(
          multi_kernel<S, DT>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem));
      if (e != cudaSuccess) return e;
      if (device < 64) done |= 1ull << device;
    }
  }
  cudaError_t e = launch_pdl(multi_kernel<S, DT>, dim3((unsigned)ctas), S::kThreads, S::kSmem,
                             stream, maps[0], maps[1], maps[2], a);
  const int sets = ctas / a.gs;
  if (e != cudaSuccess || !cut || sets < 2) return e;
  // few items of many parts: the parts of a few columns to a CTA, else half the columns
  const bool deep = items * 8 <= sets;
  const int cols = deep ? Join<S, 4>::COLS : Join<S, 1>::COLS;
  const dim3 grid((unsigned)(deep ? items : sets - 1), (unsigned)a.gs,
                  (unsigned)((S::N + cols - 1) / cols));
  return launch_pdl(deep ? join_kernel<S, DT, 4> : join_kernel<S, DT, 1>, grid, kJoinThreads, 0,
                    stream, a, sets, (int)(items / a.B));
}

// The shape of N columns.
template <template <int> class Of, int DT>
cudaError_t launch_columns(int n, const CUtensorMap (&maps)[3], const Args& a, int ctas,
                           int64_t items, bool cut, int device, cudaStream_t stream) {
  if (n == 16) return launch<Of<16>, DT>(maps, a, ctas, items, cut, device, stream);
  if (n == 32) return launch<Of<32>, DT>(maps, a, ctas, items, cut, device, stream);
  return launch<Of<64>, DT>(maps, a, ctas, items, cut, device, stream);
}

// What a call asks for, checked but for the sizes of its own cache.
struct Call {
  void* out;
  const void* q;
  const void* k_pool;
  const void* v_pool;
  const int32_t* tables;
  const int32_t* lens;
  const int32_t* q_start;
  const int32_t* mask;
  int B, total_q, Hq, H, bs, max_blocks, num_blocks, max_q, words, max_len;
  float scale;
  int dtype;                     // with PA_TWO_TERMS or without
  void* workspace;
  size_t workspace_bytes;
  int32_t* status_dev;
  cudaStream_t stream;
};

inline int storage(const Call& c) { return c.dtype & ~PA_TWO_TERMS; }
inline bool two_terms(const Call& c) { return c.dtype & PA_TWO_TERMS; }

// Host checks; PA_OK and *work false: nothing to do.
inline pa_status check(const Call& c, size_t workspace_needed, bool* work) {
  *work = false;
  if (c.B < 0 || c.total_q < 0 || c.max_blocks <= 0 || c.num_blocks <= 0 || c.max_len < 0 ||
      c.max_len >= (1 << 30) || !isfinite(c.scale) || (!c.q_start && c.total_q != c.B) ||
      (c.mask && (c.words <= 0 || (int64_t)c.words * 32 < c.max_q)) ||
      (int64_t)c.num_blocks * c.bs >= (1ll << 31) || (int64_t)c.total_q * c.Hq >= (1ll << 31))
    return PA_ERR_INVALID_ARG;
  if ((c.bs != 8 && c.bs != 16 && c.bs != 32 && c.bs != 64) ||
      (storage(c) != PA_FLOAT16 && storage(c) != PA_BFLOAT16))
    return PA_ERR_UNSUPPORTED;
  if (c.B == 0 || c.total_q == 0) return PA_OK;
  if (!c.out || !c.q || !c.k_pool || !c.v_pool || !c.tables || !c.lens) return PA_ERR_INVALID_ARG;
  if ((((uintptr_t)c.out | (uintptr_t)c.q | (uintptr_t)c.k_pool | (uintptr_t)c.v_pool) & 15u) != 0)
    return PA_ERR_INVALID_ARG;
  if (!c.workspace || ((uintptr_t)c.workspace & 255u) || c.workspace_bytes < workspace_needed)
    return PA_ERR_WORKSPACE;
  *work = true;
  return PA_OK;
}

// Launches a checked call, with at most `widest` columns of a product.  Launch: f(columns, maps,
// args, CTAs, items, cut, device).
template <class F>
pa_status run(const Call& c, int tok, int dv, int slabs, bool heads, int widest, const F& f) {
  const int max_q = c.q_start ? c.max_q : 1, G = c.Hq / c.H;
  const Columns cols = columns_for(max_q, G, widest);
  const int64_t groups =                       // pairs of column groups
      (((int64_t)max_q + cols.gn - 1) / cols.gn * cols.chunks + cols.gs - 1) / cols.gs;
  const int64_t nt = ((int64_t)c.max_len + tok - 1) / tok;
  // a factor at a time: the product of all three may pass 64 bits
  const int64_t most = 1ll << 31, heads_of_all = (int64_t)c.B * c.H;
  if (heads_of_all > most || heads_of_all * groups > most) return PA_ERR_INVALID_ARG;
  const int64_t items = heads_of_all * groups;
  int device = 0, sms = 0;
  if (!encode_fn() || taken(cudaGetDevice(&device)) != cudaSuccess ||
      taken(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device)) != cudaSuccess)
    return PA_ERR_CUDA;
  int64_t sets = (sms < kMaxCtas ? sms : kMaxCtas) / cols.gs;
  if ((items * nt) / sets >= (1ll << 30)) return PA_ERR_INVALID_ARG;
  if (items * nt < sets) sets = items * nt > 0 ? items * nt : 1;
  CUtensorMap maps[3];
  if (!encode_blocks(&maps[0], c.k_pool, storage(c), c.num_blocks, c.bs, heads ? c.H : 0, slabs) ||
      !encode_blocks(&maps[1], c.v_pool, storage(c), c.num_blocks, c.bs, heads ? c.H : 0, slabs) ||
      !encode_q(&maps[2], c.q, storage(c), c.total_q, c.Hq, slabs, cols.gh, cols.gn))
    return PA_ERR_INVALID_ARG;
  const Layout y = layout_of(cols.n, dv);
  char* ws = static_cast<char*>(c.workspace);
  Args a;
  a.out = c.out;
  a.v_src = c.v_pool;
  a.tables = c.tables;
  a.lens = c.lens;
  a.q_start = c.q_start;
  a.mask = c.mask;
  a.B = c.B;
  a.total_q = c.total_q;
  a.Hq = c.Hq;
  a.H = c.H;
  a.G = G;
  a.bs_shift = c.bs == 8 ? 3 : (c.bs == 16 ? 4 : (c.bs == 32 ? 5 : 6));
  a.max_blocks = c.max_blocks;
  a.num_blocks = c.num_blocks;
  a.max_q = max_q;
  a.words = c.words;
  a.max_len = c.max_len;
  a.gh = cols.gh;
  a.gn = cols.gn;
  a.chunks = cols.chunks;
  a.gs = cols.gs;
  a.narrow = items * (4 * nt + kEnds) < (1ll << 31);
  a.scale_log2 = (float)((double)c.scale * 1.4426950408889634);
  a.info = reinterpret_cast<Window*>(ws);
  a.ws_m = reinterpret_cast<float*>(ws + y.m_off);
  a.ws_l = reinterpret_cast<float*>(ws + y.l_off);
  a.ws_acc = reinterpret_cast<float*>(ws + y.acc_off);
  a.status_dev = c.status_dev;
  // an item of one tile is never cut
  const cudaError_t e = f(cols.n, maps, a, (int)(sets * cols.gs), items, nt > 1, device);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace multi
}  // namespace pa
