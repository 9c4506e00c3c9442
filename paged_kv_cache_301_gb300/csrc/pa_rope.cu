// Rotated cache writes: per-head RMS norm and position rotation of the new
// tokens' queries and keys, and the cache write of keys and values, in one pass.
//
//   y = x * rsqrt(mean(x^2) + eps) * w                       (where w is given)
//   (y_a, y_b) -> (y_a c - y_b s, y_b c + y_a s)             for each rotated pair
//
// pa_rope_append writes keys and values to a 16-bit pool, pa_rope_append_q8 to
// the 8-bit cache (pa_q8.cuh).  Every step is fp32; q and the 16-bit keys are
// rounded once, at the store, and 8-bit codes are rounded once from fp32.
//
// Both only move memory: each element is read once and written once, so the
// bound is bytes / HBM bandwidth for prompts and the chain of dependent loads
// (length -> table -> slot) for decode steps.  A head row is shared by D/16 lanes;
// each holds two 16-byte vectors, the two halves of its eight pairs, so that the
// rotation stays inside a lane and only the norm's sum is shuffled.
//
// Measured (GB300, 32 query and 8 KV heads of 128, graph of calls): decode step of 64
// sequences with norms 3.2-3.5 us; prompts of 18,432 tokens 75.0 us, 6.07 TB/s, 0.91 of
// a plain copy (the register kernel alone: 102 us), with norms 80.5; into the 8-bit cache:
// 18,432 tokens 73 us, with norms 81; a step of 256 sequences 3.3-4.1 us while no older
// block's scale rises, and more where one does (rope_step_q8_kernel).
#include <mutex>

#include "pa_common.cuh"
#include "pa_internal.h"
#include "pa_q8.cuh"
#include "pa_sm100.cuh"

namespace pa {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kRowThreads = 256;

struct RopeArgs {
  void* q_out;
  void* k_pool;
  void* v_pool;
  float* k_scale;        // 8-bit cache only
  float* v_scale;
  const void* q;
  const void* key;
  const void* value;
  const void* q_weight;
  const void* k_weight;
  const float* cos_sin;
  const int32_t* positions;
  const int32_t* tables;
  const int32_t* lens;
  const int32_t* q_start;
  int64_t q_stride, kv_stride;       // elements between tokens
  float eps;
  int max_position, rotary, interleaved;
  int B, total_q, Hq, H, bs, max_blocks, num_blocks;
  int32_t* status_dev;
};

// Where a token lives.  ok: its sequence is valid and the token is one of its.
struct Place {
  int b, pos, ok;
};

// The sequence of token t: the number of sequences that end at or before it
// (q_start is non-decreasing).  Called by whole warps with a uniform t; every
// round narrows 32-fold.
__device__ __forceinline__ int find_seq(const int32_t* q_start, int B, int t, int lane) {
  int lo = 0, n = B;                 // the answer is in [lo, lo + n]
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int j = lo + (lane + 1) * step;          // boundary q_start[j] ends sequence j - 1
    const bool before = j <= lo + n && q_start[j] <= t;
    const int k = __popc(__ballot_sync(kAll, before));
    lo += k * step;
    // the next boundary at lo + step (if in range) is past t
    n = min(step - 1, n - k * step);
  }
  return lo;
}

// Sequence b's token t (host bounds: b in [0, B]).  A sequence whose rows or
// length do not fit is not written at all; `bad` says to report it.
__device__ __forceinline__ Place place_of(const RopeArgs& a, int b, int t, bool* bad) {
  Place p = {b, 0, 0};
  *bad = false;
  if (b >= a.B) return p;            // behind the last sequence: left as it was
  const int L = a.lens[b];
  int s = t, n = 1;
  if (a.q_start) {
    s = a.q_start[b];
    const int e = a.q_start[b + 1];
    if (s < 0 || t < s || t >= e || e > a.total_q) {
      *bad = true;
      return p;
    }
    n = e - s;
  } else if (L == 0) {
    return p;                        // an empty sequence of a decode step
  }
  if (n > L || (int64_t)L > (int64_t)a.max_blocks * a.bs) {
    *bad = true;
    return p;
  }
  p.pos = L - n + (t - s);
  p.ok = 1;
  return p;
}

template <int DT>
__device__ __forceinline__ void widen8(const uint4& w, float (&x)[8]) {
  const float2 a = widen2<DT>(w.x), b = widen2<DT>(w.y), c = widen2<DT>(w.z),
               d = widen2<DT>(w.w);
  x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
  x[4] = c.x; x[5] = c.y; x[6] = d.x; x[7] = d.y;
}

template <int DT>
__device__ __forceinline__ uint4 narrow8(const float (&x)[8]) {
  return make_uint4(pack2<DT>(x[0], x[1]), pack2<DT>(x[2], x[3]), pack2<DT>(x[4], x[5]),
                    pack2<DT>(x[6], x[7]));
}

// A lane's 16 elements of a head row: vectors (8 elements) v0 and v1 of it.  Rotated
// lanes (li < R/16) hold pairs: with pairs (j, j + R/2) vectors li and li + R/16; with
// neighbours, and behind the rotated part, two vectors side by side.
struct Part {
  int v0, v1;
  bool turns;                  // the lane's elements are rotated
};

__device__ __forceinline__ Part part_of(int li, int R, int interleaved) {
  const bool turns = li < R / 16;
  if (turns && !interleaved) return {li, li + R / 16, true};
  return {2 * li, 2 * li + 1, turns};
}

// A position's cosines and sines of a lane's eight pairs.
struct Turn {
  float c[8], s[8];
};

// angles: the position's row of cos_sin, R/2 cosines, then R/2 sines.
__device__ __forceinline__ Turn load_turn(const float* angles, int R, int li) {
  const float4* c = reinterpret_cast<const float4*>(angles + 8 * li);
  const float4* s = reinterpret_cast<const float4*>(angles + R / 2 + 8 * li);
  const float4 c0 = c[0], c1 = c[1], s0 = s[0], s1 = s[1];
  Turn t;
  t.c[0] = c0.x; t.c[1] = c0.y; t.c[2] = c0.z; t.c[3] = c0.w;
  t.c[4] = c1.x; t.c[5] = c1.y; t.c[6] = c1.z; t.c[7] = c1.w;
  t.s[0] = s0.x; t.s[1] = s0.y; t.s[2] = s0.z; t.s[3] = s0.w;
  t.s[4] = s1.x; t.s[5] = s1.y; t.s[6] = s1.z; t.s[7] = s1.w;
  return t;
}

__device__ __forceinline__ uint4 pick(bool first, uint4 x, uint4 y) {
  return make_uint4(first ? x.x : y.x, first ? x.y : y.y, first ? x.z : y.z, first ? x.w : y.w);
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// 1 / the root mean square of a head row, over its D/16 lanes.  Called by whole warps
// (it shuffles).  Two-wide fp32 arithmetic: these kernels issue nearly as much as they
// move.
template <int D>
__device__ __forceinline__ float inv_rms(const float (&a)[8], const float (&b)[8], float eps) {
  using namespace sm100;
  uint64_t sum = 0;                            // two zeros
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const uint64_t p = f2_pack(a[i], a[i + 1]), q = f2_pack(b[i], b[i + 1]);
    sum = f2_fma(p, p, f2_fma(q, q, sum));
  }
  float s0, s1;
  f2_unpack(sum, s0, s1);
  float ss = s0 + s1;
#pragma unroll
  for (int o = D / 32; o; o >>= 1) ss += __shfl_xor_sync(kAll, ss, o);
  return rsqrtf(ss * (1.f / D) + eps);
}

// x <- x r w
__device__ __forceinline__ void scale8(float (&x)[8], float r, const float (&w)[8]) {
  using namespace sm100;
  const uint64_t r2 = f2_pack(r, r);
#pragma unroll
  for (int i = 0; i < 8; i += 2)
    f2_unpack(mul2(mul2(f2_pack(x[i], x[i + 1]), r2), f2_pack(w[i], w[i + 1])), x[i], x[i + 1]);
}

// RMS norm of a head row by w0 and w1, the weight's vectors v0 and v1; `on`: the
// group's row is normed.  Called by whole warps.
template <int DT, int D>
__device__ __forceinline__ void norm(float (&a)[8], float (&b)[8], bool on, uint4 w0,
                                     uint4 w1, float eps) {
  const float r = inv_rms<D>(a, b, eps);
  if (on) {
    float w[8];
    widen8<DT>(w0, w);
    scale8(a, r, w);
    widen8<DT>(w1, w);
    scale8(b, r, w);
  }
}

__device__ __forceinline__ void rotate(float (&a)[8], float (&b)[8], const Turn& t,
                                       int interleaved) {
  using namespace sm100;
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float p = a[2 * i], q = a[2 * i + 1], u = b[2 * i], v = b[2 * i + 1];
      a[2 * i] = p * t.c[i] - q * t.s[i];
      a[2 * i + 1] = q * t.c[i] + p * t.s[i];
      b[2 * i] = u * t.c[i + 4] - v * t.s[i + 4];
      b[2 * i + 1] = v * t.c[i + 4] + u * t.s[i + 4];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const uint64_t p = f2_pack(a[i], a[i + 1]), q = f2_pack(b[i], b[i + 1]);
      const uint64_t c = f2_pack(t.c[i], t.c[i + 1]), s = f2_pack(t.s[i], t.s[i + 1]);
      f2_unpack(f2_sub(mul2(p, c), mul2(q, s)), a[i], a[i + 1]);
      f2_unpack(f2_fma(q, c, mul2(p, s)), b[i], b[i + 1]);
    }
  }
}

// The angles of a live token, or null (no rotation, or a position outside the
// table: *ok becomes false).
__device__ __forceinline__ const float* angles_of(const RopeArgs& a, int t, int pos, bool* ok) {
  if (a.rotary == 0) return nullptr;
  if (a.positions) pos = a.positions[t];
  if (pos < 0 || pos >= a.max_position) {
    *ok = false;
    return nullptr;
  }
  return a.cos_sin + (int64_t)pos * a.rotary;
}

// All rows of token t, by one CTA (a decode step: its time is the chain of loads, so a
// CTA has one token and few rows a thread): row r < Hq is query head r; with
// KV16 the keys and values of the 16-bit cache follow.  Groups of D/16 lanes take
// rows in turn, U at a time so that their loads overlap; the first ones, and the
// norms' weights, are asked for before the token's place is looked up, and the
// token's angles once for all of a thread's rows.
template <int DT, int D, bool KV16>
__device__ __forceinline__ void token_rows(const RopeArgs& a, int t) {
  constexpr int TG = D / 16, NG = kRowThreads / TG, U = 2, RV = D / 8;
  const int lane = threadIdx.x & 31, li = threadIdx.x % TG, grp = threadIdx.x / TG;
  const Part part = part_of(li, a.rotary, a.interleaved);
  const int rows = KV16 ? a.Hq + 2 * a.H : a.Hq;
  const uint4* q = reinterpret_cast<const uint4*>(a.q) + t * (a.q_stride / 8);
  const uint4* key = reinterpret_cast<const uint4*>(a.key) + t * (a.kv_stride / 8);
  const uint4* value = reinterpret_cast<const uint4*>(a.value) + t * (a.kv_stride / 8);
  uint4 w[U][2];
  auto load_rows = [&](int r0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * NG + grp;
      const uint4* row = nullptr;
      if (r < a.Hq) row = q + r * RV;
      else if (KV16 && r < a.Hq + a.H) row = key + (r - a.Hq) * RV;
      else if (KV16 && r < rows) row = value + (r - a.Hq - a.H) * RV;
      w[u][0] = row ? row[part.v0] : make_uint4(0, 0, 0, 0);
      w[u][1] = row ? row[part.v1] : make_uint4(0, 0, 0, 0);
    }
  };
  load_rows(0);
  uint4 qw[2] = {}, kw[2] = {};
  if (a.q_weight) {
    qw[0] = reinterpret_cast<const uint4*>(a.q_weight)[part.v0];
    qw[1] = reinterpret_cast<const uint4*>(a.q_weight)[part.v1];
  }
  if (KV16 && a.k_weight) {
    kw[0] = reinterpret_cast<const uint4*>(a.k_weight)[part.v0];
    kw[1] = reinterpret_cast<const uint4*>(a.k_weight)[part.v1];
  }

  const int b = a.q_start ? find_seq(a.q_start, a.B, t, lane) : t;
  bool bad;
  const Place at = place_of(a, b, t, &bad);
  bool ok = at.ok;
  const float* angles = ok ? angles_of(a, t, at.pos, &ok) : nullptr;
  if (!ok) {
    if ((bad || at.ok) && threadIdx.x == 0) report(a.status_dev, PA_ERR_BAD_BLOCK_ID);
    return;
  }
  Turn turn = {};
  if (part.turns) turn = load_turn(angles, a.rotary, li);
  int64_t slot = -1;
  if (KV16) {
    const int32_t blk = a.tables[(int64_t)b * a.max_blocks + at.pos / a.bs];
    if (blk >= 0 && blk < a.num_blocks) slot = (int64_t)blk * a.bs + at.pos % a.bs;
    else if (threadIdx.x == 0) report(a.status_dev, PA_ERR_BAD_BLOCK_ID);
  }
  const bool any_norm = a.q_weight || (KV16 && a.k_weight);
  for (int r0 = 0;;) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * NG + grp;
      if (r - lane / TG >= rows) break;        // the warp's first row
      const bool is_q = r < a.Hq, is_k = KV16 && !is_q && r < a.Hq + a.H;
      float x[8], y[8];
      widen8<DT>(w[u][0], x);
      widen8<DT>(w[u][1], y);
      if (any_norm)
        norm<DT, D>(x, y, is_q ? a.q_weight != nullptr : is_k && a.k_weight != nullptr,
                    pick(is_q, qw[0], kw[0]), pick(is_q, qw[1], kw[1]), a.eps);
      if (part.turns) rotate(x, y, turn, a.interleaved);
      uint4* to = nullptr;
      if (is_q) to = reinterpret_cast<uint4*>(a.q_out) + ((int64_t)t * a.Hq + r) * RV;
      else if (is_k && slot >= 0)
        to = reinterpret_cast<uint4*>(a.k_pool) + (slot * a.H + (r - a.Hq)) * RV;
      if (to) {
        to[part.v0] = narrow8<DT>(x);
        to[part.v1] = narrow8<DT>(y);
      } else if (KV16 && !is_k && r < rows && slot >= 0) {
        to = reinterpret_cast<uint4*>(a.v_pool) + (slot * a.H + (r - a.Hq - a.H)) * RV;
        to[part.v0] = w[u][0];
        to[part.v1] = w[u][1];
      }
    }
    r0 += NG * U;
    if (r0 >= rows) break;
    load_rows(r0);
  }
}

// ---------------------------------------------------------------- many tokens --
// One CTA takes a run of tokens through a ring of shared-memory stages: bulk copies
// bring a few tokens' rows and angles in (one contiguous copy each for q, key, value
// and the row of cos_sin), seven warps norm and rotate them in place, bulk copies take
// them out (values without passing through registers).  The eighth warp issues all the
// copies, so that no computing warp waits for one to be read out.  Reads of later
// tokens and writes of earlier ones are in flight all the time, 150 KB of an SM, which
// the register kernel above cannot hold at the occupancy that a row's registers leave it.
// The norms' weights are widened once, to shared memory (with norms 77 us for 81).
constexpr int kMaxStages = 3;                  // 18,432 tokens: 75 us; two 101, four 85
constexpr int kComputeWarps = kRowThreads / 32 - 1;
constexpr int kRun = kRowThreads;              // tokens of a CTA at most: one thread places one
// Tokens per SM from which on it is taken (8 per SM: 10.3 us either way; 4 per SM: 6.2 us
// with the register kernel, 6.9 so; 120 per SM: 102 us and 75).
constexpr int kStreamTokens = 8;
constexpr int kMaxTogether = 8;                // tokens of a stage at most
constexpr uint64_t kStreamLimitNs = 2000000000ull;

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          sm100::smem_addr(dst)),
      "l"(src), "r"(bytes), "r"(sm100::smem_addr(bar))
      : "memory");
}

// 16 bytes to shared memory, behind the thread's back.
__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(sm100::smem_addr(dst)), "l"(src)
               : "memory");
}

__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst),
               "r"(sm100::smem_addr(src)), "r"(bytes)
               : "memory");
}

// The place of one thread's token: a binary search for its sequence.
__device__ __forceinline__ Place place_token(const RopeArgs& a, int t, bool* bad) {
  int b = t;
  if (a.q_start) {
    int lo = 0, hi = a.B;                      // the boundaries at or before t: [lo, hi]
    while (lo < hi) {
      const int mid = lo + (hi - lo) / 2;
      if (a.q_start[mid + 1] <= t) lo = mid + 1;
      else hi = mid;
    }
    b = lo;
  }
  return place_of(a, b, t, bad);
}

// Tokens [total_q cta / ctas, total_q (cta + 1) / ctas), kRun at most, `together` of
// them to a stage.
template <int DT, int D, bool KV16>
__device__ __forceinline__ void stream_rows(const RopeArgs& a, int cta, int ctas, int stages,
                                            int together, uint8_t* ring) {
  constexpr int TG = D / 16, NG = kComputeWarps * 32 / TG, RV = D / 8;
  __shared__ __align__(8) uint64_t full[kMaxStages], done[kMaxStages];
  __shared__ int64_t s_slot[kRun];             // pool row of the token (-1: none)
  __shared__ int s_pos[kRun];                  // row of cos_sin (-1: leave the token alone)
  __shared__ float4 s_weight[2][4][TG];        // of q and k, widened, by lane of a row
  __shared__ int s_abort;
  volatile int* abort_flag = &s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int li = tid % TG, grp = tid / TG;
  const bool copies = tid == kComputeWarps * 32;       // the thread that issues them
  const Part part = part_of(li, a.rotary, a.interleaved);
  const int t0 = (int)((int64_t)a.total_q * cta / ctas);
  const int n = (int)((int64_t)a.total_q * (cta + 1) / ctas) - t0;
  const int steps = (n + together - 1) / together;
  const uint32_t q_bytes = (uint32_t)(a.Hq * D * 2), kv_bytes = KV16 ? (uint32_t)(a.H * D * 2) : 0;
  const uint32_t row_bytes = q_bytes + 2 * kv_bytes, angle_bytes = (uint32_t)(a.rotary * 4);
  const uint32_t token_bytes = row_bytes + angle_bytes;
  if (copies) {
    for (int i = 0; i < stages; ++i) {
      sm100::mbar_init(&full[i], 2);           // rows, angles
      sm100::mbar_init(&done[i], kComputeWarps);
    }
    s_abort = 0;
    sm100::fence_mbar_init();
  }
  __syncthreads();
  auto stage_of = [&](int step) {
    return ring + (uint32_t)(step % stages) * ((uint32_t)together * token_bytes);
  };
  auto fetch_rows = [&](int step) {
    uint8_t* to = stage_of(step);
    uint64_t* bar = &full[step % stages];
    const int first = step * together, many = min(together, n - first);
    sm100::mbar_arrive_expect_tx(bar, many * row_bytes);
    for (int i = 0; i < many; ++i, to += token_bytes) {
      const int64_t t = t0 + first + i;
      bulk_load(to, static_cast<const uint16_t*>(a.q) + t * a.q_stride, q_bytes, bar);
      if (KV16) {
        bulk_load(to + q_bytes, static_cast<const uint16_t*>(a.key) + t * a.kv_stride, kv_bytes,
                  bar);
        bulk_load(to + q_bytes + kv_bytes, static_cast<const uint16_t*>(a.value) + t * a.kv_stride,
                  kv_bytes, bar);
      }
    }
  };
  auto fetch_angles = [&](int step) {
    uint8_t* to = stage_of(step) + row_bytes;
    uint64_t* bar = &full[step % stages];
    const int first = step * together, many = min(together, n - first);
    int live = 0;
    for (int i = 0; i < many; ++i) live += s_pos[first + i] >= 0 ? 1 : 0;
    sm100::mbar_arrive_expect_tx(bar, live * angle_bytes);
    if (a.rotary == 0) return;
    for (int i = 0; i < many; ++i) {
      const int pos = s_pos[first + i];
      if (pos >= 0)
        bulk_load(to + i * token_bytes, a.cos_sin + (int64_t)pos * a.rotary, angle_bytes, bar);
    }
  };
  int fetched = min(stages, steps);
  if (copies)
    for (int i = 0; i < fetched; ++i) fetch_rows(i);
  if (tid < 2 * TG) {
    const uint4* from = reinterpret_cast<const uint4*>(tid < TG ? a.q_weight : a.k_weight);
    if (from && (KV16 || tid < TG)) {
      float w[8];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        widen8<DT>(from[half ? part.v1 : part.v0], w);
        s_weight[tid / TG][2 * half][li] = make_float4(w[0], w[1], w[2], w[3]);
        s_weight[tid / TG][2 * half + 1][li] = make_float4(w[4], w[5], w[6], w[7]);
      }
    }
  }
  if (tid < n) {                               // every thread places a token of the run
    bool bad;
    const int t = t0 + tid;
    const Place at = place_token(a, t, &bad);
    bool ok = at.ok;
    if (ok) angles_of(a, t, at.pos, &ok);
    if (bad || (at.ok && !ok)) report(a.status_dev, PA_ERR_BAD_BLOCK_ID);
    int64_t slot = -1;
    if (KV16 && ok) {
      const int32_t blk = a.tables[(int64_t)at.b * a.max_blocks + at.pos / a.bs];
      if (blk >= 0 && blk < a.num_blocks) slot = (int64_t)blk * a.bs + at.pos % a.bs;
      else report(a.status_dev, PA_ERR_BAD_BLOCK_ID);
    }
    s_slot[tid] = slot;
    s_pos[tid] = !ok ? -1 : (a.rotary && a.positions ? a.positions[t] : at.pos);
  }
  __syncthreads();

  if (warp == kComputeWarps) {
    if (!copies) return;
    for (int i = 0; i < fetched; ++i) fetch_angles(i);
    bool ok = true;
    for (int step = 0; step < steps; ++step) {
      ok = sm100::mbar_wait(&done[step % stages], (step / stages) & 1, abort_flag, kStreamLimitNs);
      if (!ok) break;
      const uint8_t* token = stage_of(step);
      const int first = step * together, many = min(together, n - first);
      for (int i = 0; i < many; ++i, token += token_bytes) {
        if (s_pos[first + i] < 0) continue;
        bulk_store(static_cast<uint16_t*>(a.q_out) + (int64_t)(t0 + first + i) * a.Hq * D, token,
                   q_bytes);
        const int64_t slot = s_slot[first + i];
        if (KV16 && slot >= 0) {
          bulk_store(static_cast<uint16_t*>(a.k_pool) + slot * a.H * D, token + q_bytes, kv_bytes);
          bulk_store(static_cast<uint16_t*>(a.v_pool) + slot * a.H * D, token + q_bytes + kv_bytes,
                     kv_bytes);
        }
      }
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      if (step > 0 && fetched < steps) {
        // the stage of the step before has been read out: the next one comes in
        asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
        fetch_rows(fetched);
        fetch_angles(fetched++);
      }
    }
    if (!ok) {                                 // copies in flight land before the CTA ends
      *abort_flag = 1;
      report(a.status_dev, PA_ERR_TIMEOUT);
      for (int j = max(0, fetched - stages); j < fetched; ++j)
        sm100::mbar_wait_drain(&full[j % stages], (j / stages) & 1, kStreamLimitNs);
    }
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    return;
  }

  const bool any_norm = a.q_weight || (KV16 && a.k_weight);
  const int turned = KV16 ? a.Hq + a.H : a.Hq;
  for (int step = 0; step < steps; ++step) {
    const int first = step * together, many = min(together, n - first);
    if (!__all_sync(kAll, sm100::mbar_wait(&full[step % stages], (step / stages) & 1, abort_flag,
                                           kStreamLimitNs))) {
      *abort_flag = 1;
      break;
    }
    uint8_t* stage = stage_of(step);
    // (token, row) pairs in turn; a warp stays in the loop while any of it has a pair
    int i = 0, r = grp;
    for (int k = warp * (32 / TG); k < many * turned; k += NG, r += NG) {
      while (r >= turned && i < many) {
        r -= turned;
        ++i;
      }
      const int at = min(i, many - 1);         // behind the last pair: any row, not stored
      const bool live = i < many && s_pos[first + at] >= 0;
      const bool is_q = r < a.Hq;
      uint8_t* token = stage + (uint32_t)at * token_bytes;
      uint4* row = reinterpret_cast<uint4*>(token) + min(r, turned - 1) * RV;
      float x[8], y[8];
      widen8<DT>(row[part.v0], x);
      widen8<DT>(row[part.v1], y);
      if (any_norm) {
        const float r_rms = inv_rms<D>(x, y, a.eps);
        if (is_q ? a.q_weight != nullptr : a.k_weight != nullptr) {
          const float4 w0 = s_weight[!is_q][0][li], w1 = s_weight[!is_q][1][li],
                       w2 = s_weight[!is_q][2][li], w3 = s_weight[!is_q][3][li];
          scale8(x, r_rms, {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w});
          scale8(y, r_rms, {w2.x, w2.y, w2.z, w2.w, w3.x, w3.y, w3.z, w3.w});
        }
      }
      if (!live) continue;
      if (part.turns)
        rotate(x, y, load_turn(reinterpret_cast<const float*>(token + row_bytes), a.rotary, li),
               a.interleaved);
      row[part.v0] = narrow8<DT>(x);
      row[part.v1] = narrow8<DT>(y);
    }
    sm100::fence_async_smem();
    __syncwarp();
    if (lane == 0) sm100::mbar_arrive(&done[step % stages]);
  }
}

// Three CTAs of an SM leave a thread 80 registers: 8 bytes (bf16) or 40 (fp16) of it spill.
template <int DT, int D>
__global__ void __launch_bounds__(kRowThreads, 3)
rope_append_kernel(const RopeArgs a) {
  allow_next_grid();
  wait_prior_grid();
  token_rows<DT, D, true>(a, (int)blockIdx.x);
}

template <int DT, int D>
__global__ void __launch_bounds__(kRowThreads, 4)
rope_stream_kernel(const RopeArgs a, int stages, int together) {
  extern __shared__ __align__(128) uint8_t ring[];
  allow_next_grid();
  wait_prior_grid();
  stream_rows<DT, D, true>(a, (int)blockIdx.x, (int)gridDim.x, stages, together, ring);
}

// Bring older codes to a larger scale: 8 codes times `ratio`, rounded once more
// (exact for powers of two but where a code becomes subnormal).
__device__ __forceinline__ void rescale8(uint2* p, float ratio) {
  const uint2 w = *p;
  const float2 a = e4m3_widen2(w.x), b = e4m3_widen2(w.x >> 16), c = e4m3_widen2(w.y),
               d = e4m3_widen2(w.y >> 16);
  *p = make_uint2(e4m3x4(a.x * ratio, a.y * ratio, b.x * ratio, b.y * ratio),
                  e4m3x4(c.x * ratio, c.y * ratio, d.x * ratio, d.y * ratio));
}

// The largest finite magnitude of 16 elements.  A NaN is never the largest; an
// infinity, which would be, sends the lane through them again.
__device__ __forceinline__ float mag16(const float (&a)[8], const float (&b)[8]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fmaxf(fabsf(a[i]), fabsf(b[i])));
  if (__float_as_uint(m) == 0x7F800000u) {
    m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fmaxf(finite_mag(a[i]), finite_mag(b[i])));
  }
  return m;
}

// The same of 16 stored elements: their magnitudes order as their bits do, two at a
// time; from the infinity's bits on they are not finite.
template <int DT>
__device__ __forceinline__ float mag16(const uint4& a, const uint4& b) {
  constexpr uint32_t inf = DT == PA_BFLOAT16 ? 0x7F80u : 0x7C00u;
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
  m = max(m & 0xFFFFu, m >> 16);
  if (m >= inf) {
    m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t lo = w[i] & 0x7FFFu, hi = (w[i] >> 16) & 0x7FFFu;
      if (lo < inf) m = max(m, lo);
      if (hi < inf) m = max(m, hi);
    }
  }
  return widen2<DT>(m).x;
}

__device__ __forceinline__ uint2 quantise8(const float (&x)[8], float inv) {
  const uint64_t i2 = sm100::f2_pack(inv, inv);
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; i += 2)
    sm100::f2_unpack(mul2(sm100::f2_pack(x[i], x[i + 1]), i2), y[i], y[i + 1]);
  return make_uint2(e4m3x4(y[0], y[1], y[2], y[3]), e4m3x4(y[4], y[5], y[6], y[7]));
}

// How a CTA covers a block's rows: a head has kHead threads, whose groups hold rows
// g, g + NG, ...
template <int D, int BS>
struct BlockShape {
  static constexpr int TG = D / 16;
  static constexpr int kHead = BS * TG < kRowThreads ? BS * TG : kRowThreads;
  static constexpr int kHeads = kRowThreads / kHead;      // heads of a CTA
  static constexpr int NG = kHead / TG, RPT = BS / NG;    // groups, rows of each
};

constexpr int kKvStages = 3;                   // items of a CTA in flight

// Shared memory of the items in flight: every thread's elements, 64 bytes of a row.
template <int D, int BS>
constexpr int kv_bytes() {
  return kKvStages * BlockShape<D, BS>::RPT * 4 * kRowThreads * 16;
}

// A block with new rows: [r0, r0 + n), tokens t ..; older rows are below r0.
struct NewRows {
  int t, pos, n, blk;          // first token, its position, rows, physical block
};

// Keys and values of tokens [t0, t0 + n) (kRowThreads at most) to the 8-bit cache: the
// blocks whose first new token is among them, for `parts` groups of KV heads from
// `part` on.  A block and a group of heads is one item: its largest magnitudes are
// taken over the CTA, then its codes are made.  The rows of the items behind it are on
// their way to shared memory meanwhile, each thread's elements to a place of its own (no
// barrier, only its own copies to wait for); a block's angles are read once for all its
// heads.  18,432 tokens: 82 us, with the next item's rows in registers 93.  What bounds
// it in this form: an item's chain of maxima over the CTA, scale, codes, with two CTAs of an
// SM (the registers of a row); a third CTA spills.
template <int DT, int D, int BS>
__device__ __forceinline__ void store_run(const RopeArgs& a, int t0, int n, int part, int parts,
                                          uint8_t* smem) {
  using S = BlockShape<D, BS>;
  constexpr int TG = S::TG, NG = S::NG, RPT = S::RPT, NW = S::kHead / 32, RV = D / 8;
  constexpr int WARPS = kRowThreads / 32;
  __shared__ NewRows s_list[kRowThreads];
  __shared__ int s_count[WARPS];
  __shared__ float s_mag[2][WARPS][2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int mine = tid / S::kHead, li = tid % TG, grp = tid % S::kHead / TG;
  const Part el = part_of(li, a.rotary, a.interleaved);

  // every thread places a token; those that begin a block's new rows make the list
  NewRows first = {t0 + tid, 0, 0, -1};
  bool begins = false;
  if (tid < n) {
    bool bad;
    const Place at = place_token(a, first.t, &bad);
    if (at.ok) {
      const int row = at.pos % BS;
      begins = row == 0 || first.t == a.q_start[at.b];
      if (begins) {
        first.pos = at.pos;
        first.n = min(a.q_start[at.b + 1] - first.t, BS - row);
        first.blk = a.tables[(int64_t)at.b * a.max_blocks + at.pos / BS];
        if (first.blk < 0 || first.blk >= a.num_blocks) {
          if (part == 0) report(a.status_dev, PA_ERR_BAD_BLOCK_ID);
          begins = false;
        }
      }
    }
  }
  const uint32_t ballot = __ballot_sync(kAll, begins);
  if (lane == 0) s_count[warp] = __popc(ballot);
  __syncthreads();
  int before = 0, blocks = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    before += w < warp ? s_count[w] : 0;
    blocks += s_count[w];
  }
  if (begins) s_list[before + __popc(ballot & ((1u << lane) - 1))] = first;
  __syncthreads();

  uint4 wt[2] = {};
  if (a.k_weight) {
    wt[0] = reinterpret_cast<const uint4*>(a.k_weight)[el.v0];
    wt[1] = reinterpret_cast<const uint4*>(a.k_weight)[el.v1];
  }
  const int items = blocks * parts;
  auto place = [&](int item, int i) {          // 16 bytes of this thread
    return reinterpret_cast<uint4*>(smem) + (item % kKvStages * (RPT * 4) + i) * kRowThreads + tid;
  };
  auto ask = [&](int item) {
    if (item < items) {
      const NewRows at = s_list[item / parts];
      const int h = (part + item % parts) * S::kHeads + mine, r0 = at.pos % BS;
#pragma unroll
      for (int u = 0; u < RPT; ++u) {
        const int row = grp + u * NG;
        if (h < a.H && row >= r0 && row < r0 + at.n) {
          const int64_t from = (at.t + row - r0) * (a.kv_stride / 8) + h * RV;
          const uint4* k = reinterpret_cast<const uint4*>(a.key) + from;
          const uint4* v = reinterpret_cast<const uint4*>(a.value) + from;
          copy16(place(item, 4 * u), k + el.v0);
          copy16(place(item, 4 * u + 1), k + el.v1);
          copy16(place(item, 4 * u + 2), v + el.v0);
          copy16(place(item, 4 * u + 3), v + el.v1);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kKvStages - 1; ++i) ask(i);
  bool fresh[RPT];                             // a new row whose position is in range
  Turn turn[RPT];
  for (int item = 0; item < items; ++item) {
    const NewRows at = s_list[item / parts];
    const int h = (part + item % parts) * S::kHeads + mine, r0 = at.pos % BS;
    const bool in = h < a.H;
    const int64_t tile = (int64_t)at.blk * a.H + h;
    uint2* kc = static_cast<uint2*>(a.k_pool) + tile * (BS * RV);
    uint2* vc = static_cast<uint2*>(a.v_pool) + tile * (BS * RV);
    float k_old = 0.f, v_old = 0.f;
    if (in && r0 > 0) {
      k_old = a.k_scale[tile];
      v_old = a.v_scale[tile];
    }
    if (item % parts == 0) {                   // a new block
#pragma unroll
      for (int u = 0; u < RPT; ++u) {
        const int row = grp + u * NG;
        fresh[u] = row >= r0 && row < r0 + at.n;
        if (fresh[u]) {
          const float* angles = angles_of(a, at.t + row - r0, at.pos - r0 + row, &fresh[u]);
          if (!fresh[u] && li == 0) report(a.status_dev, PA_ERR_BAD_BLOCK_ID);
          if (el.turns && angles) turn[u] = load_turn(angles, a.rotary, li);
        }
      }
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(kKvStages - 2) : "memory");
    float kx[RPT][8], ky[RPT][8];
    uint4 vw[RPT][2];
    bool live[RPT], any = false;
    float km = 0.f, vm = 0.f;
#pragma unroll
    for (int u = 0; u < RPT; ++u) {
      // a row that is not live holds anything, and nobody else's values depend on it
      widen8<DT>(*place(item, 4 * u), kx[u]);
      widen8<DT>(*place(item, 4 * u + 1), ky[u]);
      vw[u][0] = *place(item, 4 * u + 2);
      vw[u][1] = *place(item, 4 * u + 3);
      live[u] = in && fresh[u];
      any |= live[u];
      if (a.k_weight) norm<DT, D>(kx[u], ky[u], true, wt[0], wt[1], a.eps);
      if (live[u]) {
        if (el.turns) rotate(kx[u], ky[u], turn[u], a.interleaved);
        km = fmaxf(km, mag16(kx[u], ky[u]));
        vm = fmaxf(vm, mag16<DT>(vw[u][0], vw[u][1]));
      }
    }
    ask(item + kKvStages - 1);                 // to the place that the item before held
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      km = fmaxf(km, __shfl_xor_sync(kAll, km, o));
      vm = fmaxf(vm, __shfl_xor_sync(kAll, vm, o));
    }
    // two sets of maxima: the set of the item before last has been read by all
    float (*mag)[2] = s_mag[item & 1];
    if (lane == 0) {
      mag[warp][0] = km;
      mag[warp][1] = vm;
    }
    if (!__syncthreads_or(any)) continue;      // no row left to write: scales stay
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      km = fmaxf(km, mag[mine * NW + w][0]);
      vm = fmaxf(vm, mag[mine * NW + w][1]);
    }
    const float ks = fmaxf(k_old, scale_for(km)), vs = fmaxf(v_old, scale_for(vm));
    const float k_inv = 1.f / ks, v_inv = 1.f / vs;
#pragma unroll
    for (int u = 0; u < RPT; ++u) {
      const int row = grp + u * NG;
      if (live[u]) {
        float x[8], y[8];
        kc[row * RV + el.v0] = quantise8(kx[u], k_inv);
        kc[row * RV + el.v1] = quantise8(ky[u], k_inv);
        widen8<DT>(vw[u][0], x);
        widen8<DT>(vw[u][1], y);
        vc[row * RV + el.v0] = quantise8(x, v_inv);
        vc[row * RV + el.v1] = quantise8(y, v_inv);
      } else if (in && row < r0) {
        if (ks > k_old) {
          rescale8(kc + row * RV + el.v0, k_old * k_inv);
          rescale8(kc + row * RV + el.v1, k_old * k_inv);
        }
        if (vs > v_old) {
          rescale8(vc + row * RV + el.v0, v_old * v_inv);
          rescale8(vc + row * RV + el.v1, v_old * v_inv);
        }
      }
    }
    if (in && tid % S::kHead == 0) {
      a.k_scale[tile] = ks;
      a.v_scale[tile] = vs;
    }
  }
}

// Prompts and chunks.  CTAs [0, kv_ctas) write keys and values: `groups` of them share a
// run of `run` tokens (0: all tokens are shared out evenly), some heads each.  The others
// hold query rows, of one token each or, with stages, a run of tokens.
template <int DT, int D, int BS>
__global__ void __launch_bounds__(kRowThreads, 2)
rope_append_q8_kernel(const RopeArgs a, int kv_ctas, int groups, int run, int stages,
                      int together) {
  extern __shared__ __align__(128) uint8_t ring[];
  allow_next_grid();
  wait_prior_grid();
  if ((int)blockIdx.x >= kv_ctas) {
    const int cta = (int)blockIdx.x - kv_ctas;
    if (stages)
      stream_rows<DT, D, false>(a, cta, (int)gridDim.x - kv_ctas, stages, together, ring);
    else
      token_rows<DT, D, false>(a, cta);
    return;
  }
  constexpr int heads = BlockShape<D, BS>::kHeads;
  const int parts = (a.H + heads - 1) / heads, per = (parts + groups - 1) / groups;
  const int c = (int)blockIdx.x / groups, runs = kv_ctas / groups;
  const int part = ((int)blockIdx.x - c * groups) * per;
  const int t0 = run ? c * run : (int)((int64_t)a.total_q * c / runs);
  const int t1 = run ? min(t0 + run, a.total_q) : (int)((int64_t)a.total_q * (c + 1) / runs);
  store_run<DT, D, BS>(a, t0, t1 - t0, part, min(per, parts - part), ring);
}

// A decode step: one new token per sequence.  CTAs [0, kv_ctas): each group of
// D/16 lanes takes the K or the V row of one (sequence, KV head); the others hold
// one token's query rows.  Bound by the chain length -> block id -> old scale, which the
// row's load and norm overlap (256 sequences, 32 / 8 heads: 3.3-4.1 us, 1.4-1.7 TB/s).
// A block's older rows are touched only when its scale rises; its group then reads, converts
// and stores them row after row, and the step lasts as long as its slowest group.  256
// sequences, 2,048 scales each of K and V, of which 2.5% rise (normal rows in blocks of 16
// raise 2.2% of them): 8.8 us with 7 older rows, 15.4 with 15, 27 with 63 in blocks of 64;
// where all rise 11, 19.5 and 66.
template <int DT, int D>
__global__ void __launch_bounds__(kRowThreads)
rope_step_q8_kernel(const RopeArgs a, int kv_ctas) {
  constexpr int TG = D / 16, NG = kRowThreads / TG, RV = D / 8;
  allow_next_grid();
  wait_prior_grid();
  if ((int)blockIdx.x >= kv_ctas) {
    token_rows<DT, D, false>(a, (int)blockIdx.x - kv_ctas);
    return;
  }
  const int li = threadIdx.x % TG;
  const Part part = part_of(li, a.rotary, a.interleaved);
  const int64_t item = (int64_t)blockIdx.x * NG + threadIdx.x / TG;
  const bool is_v = item & 1;
  const int h = (int)((item >> 1) % a.H);
  const int64_t b64 = (item >> 1) / a.H;
  const bool in = b64 < a.B;
  const int b = in ? (int)b64 : 0;
  uint4 w[2] = {}, wt[2] = {};
  if (in) {
    const uint4* from =
        reinterpret_cast<const uint4*>(is_v ? a.value : a.key) + b * (a.kv_stride / 8) + h * RV;
    w[0] = from[part.v0];
    w[1] = from[part.v1];
  }
  if (a.k_weight) {
    wt[0] = reinterpret_cast<const uint4*>(a.k_weight)[part.v0];
    wt[1] = reinterpret_cast<const uint4*>(a.k_weight)[part.v1];
  }
  bool bad = false;
  Place at = {0, 0, 0};
  if (in) at = place_of(a, b, b, &bad);
  bool ok = at.ok;
  const float* angles = ok ? angles_of(a, b, at.pos, &ok) : nullptr;
  int32_t blk = 0;
  if (ok) {
    blk = a.tables[(int64_t)b * a.max_blocks + at.pos / a.bs];
    ok = blk >= 0 && blk < a.num_blocks;
  }
  if (!ok && (bad || at.ok) && li == 0) report(a.status_dev, PA_ERR_BAD_BLOCK_ID);
  const int row = at.pos % a.bs;
  const int64_t tile = (int64_t)blk * a.H + h;
  float* scale = (is_v ? a.v_scale : a.k_scale) + tile;
  const float old = ok && row > 0 ? *scale : 0.f;
  Turn turn = {};
  const bool turns = part.turns && angles && !is_v;
  if (turns) turn = load_turn(angles, a.rotary, li);
  float x[8], y[8];
  widen8<DT>(w[0], x);
  widen8<DT>(w[1], y);
  if (a.k_weight) norm<DT, D>(x, y, !is_v, wt[0], wt[1], a.eps);
  if (turns) rotate(x, y, turn, a.interleaved);
  float m = mag16(x, y);
#pragma unroll
  for (int o = TG / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
  const float s = fmaxf(old, scale_for(m)), inv = 1.f / s;
  if (!ok) return;
  uint2* codes = static_cast<uint2*>(is_v ? a.v_pool : a.k_pool) + tile * a.bs * RV;
  codes[row * RV + part.v0] = quantise8(x, inv);
  codes[row * RV + part.v1] = quantise8(y, inv);
  if (s > old) {
    for (int r = 0; r < row; ++r) {
      rescale8(codes + r * RV + part.v0, old * inv);
      rescale8(codes + r * RV + part.v1, old * inv);
    }
    if (li == 0) *scale = s;
  }
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

bool overlap(const void* p, int64_t np, const void* q, int64_t nq) {
  const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
  return a < b + (uintptr_t)nq && b < a + (uintptr_t)np;
}

// The checks both entries share.
pa_status check_rope(const RopeArgs& a, int head_dim, int dtype) {
  if (a.B < 0 || a.total_q < 0 || a.Hq <= 0 || a.H <= 0 || a.max_blocks <= 0 || a.num_blocks <= 0)
    return PA_ERR_INVALID_ARG;
  if (!(head_dim == 64 || head_dim == 128)) return PA_ERR_UNSUPPORTED;
  if (!(a.bs == 8 || a.bs == 16 || a.bs == 32 || a.bs == 64)) return PA_ERR_UNSUPPORTED;
  if (dtype != PA_FLOAT16 && dtype != PA_BFLOAT16) return PA_ERR_UNSUPPORTED;
  if (a.rotary < 0 || a.rotary > head_dim || a.rotary % 16) return PA_ERR_INVALID_ARG;
  if (!(a.eps >= 0.f) || a.eps > 3.0e38f) return PA_ERR_INVALID_ARG;
  if (a.rotary > 0 && a.max_position <= 0) return PA_ERR_INVALID_ARG;
  const int64_t q_row = (int64_t)a.Hq * head_dim, kv_row = (int64_t)a.H * head_dim;
  if (a.q_stride < q_row || a.q_stride % 8 || a.kv_stride < kv_row || a.kv_stride % 8)
    return PA_ERR_INVALID_ARG;
  if (a.Hq > 65536 || a.H > 65536) return PA_ERR_INVALID_ARG;
  if (!a.q_start && a.total_q != a.B) return PA_ERR_INVALID_ARG;
  return PA_OK;
}

pa_status check_rope_pointers(const RopeArgs& a, int head_dim) {
  if (!a.q_out || !a.k_pool || !a.v_pool || !a.q || !a.key || !a.value || !a.tables || !a.lens)
    return PA_ERR_INVALID_ARG;
  if (a.rotary > 0 && !a.cos_sin) return PA_ERR_INVALID_ARG;
  if (!aligned16(a.q_out) || !aligned16(a.k_pool) || !aligned16(a.v_pool) || !aligned16(a.q) ||
      !aligned16(a.key) || !aligned16(a.value) || !aligned16(a.q_weight) ||
      !aligned16(a.k_weight) || !aligned16(a.cos_sin))
    return PA_ERR_INVALID_ARG;
  // in place is q_out = q with packed rows; any other overlap would read rows
  // that another CTA has already written
  const int64_t row = (int64_t)a.Hq * head_dim;
  const int64_t out_bytes = (int64_t)a.total_q * row * 2;
  const int64_t q_bytes = ((int64_t)(a.total_q - 1) * a.q_stride + row) * 2;
  const int64_t kv_bytes = ((int64_t)(a.total_q - 1) * a.kv_stride + (int64_t)a.H * head_dim) * 2;
  if (!(a.q_out == a.q && a.q_stride == row) && overlap(a.q_out, out_bytes, a.q, q_bytes))
    return PA_ERR_INVALID_ARG;
  if (overlap(a.q_out, out_bytes, a.key, kv_bytes) || overlap(a.q_out, out_bytes, a.value, kv_bytes))
    return PA_ERR_INVALID_ARG;
  return PA_OK;
}

// How tokens of `rows` head rows go through shared memory: stages of a CTA (0: the
// register kernel), tokens of a stage, bytes of all stages, CTAs; the current device.
struct Stream {
  int stages, together, bytes, ctas, device;
};

constexpr int kSmemOfSm = 227 * 1024;
constexpr int kSmemStatic = 9 * 1024;          // more than either kernel's own, and 1 KB a CTA

// `resident` CTAs of an SM at most.
pa_status plan_stream(int tokens, int rows, int head_dim, int rotary, int resident, Stream* s) {
  *s = {0, 1, 0, tokens, 0};
  int sms = 0;
  if (taken(cudaGetDevice(&s->device)) != cudaSuccess ||
      taken(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, s->device)) !=
          cudaSuccess)
    return PA_ERR_CUDA;
  if (tokens < kStreamTokens * sms) return PA_OK;
  // where two stages of each fit the SM's shared memory, else fewer
  const int64_t token = (int64_t)rows * head_dim * 2 + rotary * 4;
  for (int per_sm = resident; per_sm; --per_sm) {
    const int64_t room = kSmemOfSm / per_sm - kSmemStatic;
    if (2 * token > room) continue;
    while (s->together < kMaxTogether && 3 * 2 * s->together * token <= room) s->together *= 2;
    const int64_t stage = s->together * token;
    s->stages = (int)(room / stage < kMaxStages ? room / stage : kMaxStages);
    s->bytes = (int)(s->stages * stage);
    const int runs = (tokens - 1) / (kRun - 1) + 1;        // of fewer than kRun tokens
    const int ctas = sms * per_sm;
    s->ctas = ctas > runs ? ctas : runs;
    break;
  }
  return PA_OK;
}

// Shared memory above 48 KB has to be asked for.  The kernel's limit is a property of the
// kernel, not of a launch: it is set once per device, to the most that any plan takes, so
// that no call lowers it between another thread's setting and launch.
template <auto Kernel>
cudaError_t allow_smem(int device) {
  static std::mutex lock;
  static uint64_t done = 0;                    // devices whose limit is set
  std::lock_guard<std::mutex> hold(lock);
  if (device < 64 && (done >> device & 1)) return cudaSuccess;
  const cudaError_t e = taken(cudaFuncSetAttribute(
      Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemOfSm - kSmemStatic));
  if (e == cudaSuccess && device < 64) done |= 1ull << device;
  return e;
}

template <int DT, int D, int BS>
cudaError_t launch_blocks(const RopeArgs& a, const Stream& s, cudaStream_t stream) {
  // few tokens: short runs, whose blocks are written one after another, of about as many
  // tokens as a sequence has; many: as many CTAs as for the queries share them (82 us for
  // 18,432 tokens; 100 with one CTA of each kind on an SM at a time), of about four blocks
  // each or, where tokens are few, some of the heads of four (8,000 tokens, blocks of 32:
  // 46.6 us; 51 with all heads of 0 to 2 blocks)
  constexpr int heads = BlockShape<D, BS>::kHeads;
  const int parts = (a.H + heads - 1) / heads;
  int run = 0, groups = parts;
  int64_t runs;
  if (s.stages == 0) {
    run = BS < 32 ? BS : 32;
    while (run > 1 && (int64_t)run * a.B > a.total_q) run /= 2;
    runs = ((int64_t)a.total_q + run - 1) / run;
  } else {
    const int least = (a.total_q - 1) / (kRun - 1) + 1;    // of fewer than kRun tokens
    const int64_t wish = (int64_t)4 * BS * s.ctas / a.total_q;
    const int most = (int)(wish < 1 ? 1 : (wish < parts ? wish : parts));
    const int per = (parts + most - 1) / most;
    groups = (parts + per - 1) / per;
    runs = s.ctas / groups > least ? s.ctas / groups : least;
  }
  const int64_t kv = runs * groups;
  if (kv + s.ctas > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const int bytes = s.bytes > kv_bytes<D, BS>() ? s.bytes : kv_bytes<D, BS>();
  static_assert(kv_bytes<D, BS>() <= kSmemOfSm - kSmemStatic, "within the kernel's limit");
  const cudaError_t e = allow_smem<rope_append_q8_kernel<DT, D, BS>>(s.device);
  if (e != cudaSuccess) return e;
  return launch_pdl(rope_append_q8_kernel<DT, D, BS>, dim3((unsigned)(kv + s.ctas)), kRowThreads,
                    bytes, stream, a, (int)kv, groups, run, s.stages, s.together);
}

template <int DT, int D>
cudaError_t launch_q8(const RopeArgs& a, cudaStream_t stream) {
  if (!a.q_start) {
    const int64_t groups = (int64_t)a.B * a.H * 2, per = kRowThreads / (D / 16);
    const int64_t kv = (groups + per - 1) / per;
    if (kv + a.total_q > 0x7FFFFFFF) return cudaErrorInvalidValue;
    return launch_pdl(rope_step_q8_kernel<DT, D>, dim3((unsigned)(kv + a.total_q)), kRowThreads, 0,
                      stream, a, (int)kv);
  }
  Stream s;
  if (plan_stream(a.total_q, a.Hq, D, a.rotary, 2, &s) != PA_OK) return cudaErrorUnknown;
  switch (a.bs) {
    case 8: return launch_blocks<DT, D, 8>(a, s, stream);
    case 16: return launch_blocks<DT, D, 16>(a, s, stream);
    case 32: return launch_blocks<DT, D, 32>(a, s, stream);
    default: return launch_blocks<DT, D, 64>(a, s, stream);
  }
}

template <int DT, int D>
cudaError_t launch_16(const RopeArgs& a, cudaStream_t stream) {
  // Tokens of 12 KB and more: two CTAs of an SM with two tokens to a stage, whose rows keep
  // a CTA's warps busy (48 rows of 128, 18,432 tokens: 75 us, four CTAs 81; 96 rows: 147,
  // four 176).  Smaller ones: four CTAs (48 rows of 64: 41 us, two 44; 12 rows: 27, two 35)
  const int rows = a.Hq + 2 * a.H, per_sm = rows * D * 2 + a.rotary * 4 >= 12 * 1024 ? 2 : 4;
  Stream s;
  if (plan_stream(a.total_q, rows, D, a.rotary, per_sm, &s) != PA_OK)
    return cudaErrorUnknown;
  if (!s.stages)
    return launch_pdl(rope_append_kernel<DT, D>, dim3((unsigned)a.total_q), kRowThreads, 0, stream,
                      a);
  const cudaError_t e = allow_smem<rope_stream_kernel<DT, D>>(s.device);
  if (e != cudaSuccess) return e;
  return launch_pdl(rope_stream_kernel<DT, D>, dim3((unsigned)s.ctas), kRowThreads, s.bytes,
                    stream, a, s.stages, s.together);
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" pa_status pa_rope_append(
    void* q_out, void* k_pool, void* v_pool, const void* q, const void* key, const void* value,
    const void* q_weight, const void* k_weight, float eps, const float* cos_sin, int max_position,
    int rotary_dim, int interleaved, const int32_t* positions, const int32_t* block_tables,
    const int32_t* seq_lens, const int32_t* q_start, int num_seqs, int total_q,
    int64_t q_token_stride, int64_t kv_token_stride, int num_q_heads, int num_kv_heads,
    int head_dim, int block_size, int max_blocks, int num_blocks, int dtype, int32_t* status_dev,
    cudaStream_t stream) {
  const RopeArgs a = {q_out, k_pool, v_pool, nullptr, nullptr, q, key, value, q_weight, k_weight,
                      cos_sin, positions, block_tables, seq_lens, q_start,
                      q_token_stride ? q_token_stride : (int64_t)num_q_heads * head_dim,
                      kv_token_stride ? kv_token_stride : (int64_t)num_kv_heads * head_dim,
                      eps, max_position, rotary_dim, interleaved, num_seqs, total_q, num_q_heads,
                      num_kv_heads, block_size, max_blocks, num_blocks, status_dev};
  pa_status st = check_rope(a, head_dim, dtype);
  if (st != PA_OK) return st;
  if (num_seqs == 0 || total_q == 0) return PA_OK;
  st = check_rope_pointers(a, head_dim);
  if (st != PA_OK) return st;
  cudaError_t e;
  if (dtype == PA_BFLOAT16)
    e = head_dim == 128 ? launch_16<PA_BFLOAT16, 128>(a, stream)
                        : launch_16<PA_BFLOAT16, 64>(a, stream);
  else
    e = head_dim == 128 ? launch_16<PA_FLOAT16, 128>(a, stream)
                        : launch_16<PA_FLOAT16, 64>(a, stream);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

extern "C" pa_status pa_rope_append_q8(
    void* q_out, void* k_pool, void* v_pool, float* k_scale, float* v_scale, const void* q,
    const void* key, const void* value, const void* q_weight, const void* k_weight, float eps,
    const float* cos_sin, int max_position, int rotary_dim, int interleaved,
    const int32_t* positions, const int32_t* block_tables, const int32_t* seq_lens,
    const int32_t* q_start, int num_seqs, int total_q, int64_t q_token_stride,
    int64_t kv_token_stride, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
    int max_blocks, int num_blocks, int dtype, int32_t* status_dev, cudaStream_t stream) {
  const RopeArgs a = {q_out, k_pool, v_pool, k_scale, v_scale, q, key, value, q_weight, k_weight,
                      cos_sin, positions, block_tables, seq_lens, q_start,
                      q_token_stride ? q_token_stride : (int64_t)num_q_heads * head_dim,
                      kv_token_stride ? kv_token_stride : (int64_t)num_kv_heads * head_dim,
                      eps, max_position, rotary_dim, interleaved, num_seqs, total_q, num_q_heads,
                      num_kv_heads, block_size, max_blocks, num_blocks, status_dev};
  pa_status st = check_rope(a, head_dim, dtype);
  if (st != PA_OK) return st;
  if (num_seqs == 0 || total_q == 0) return PA_OK;
  st = check_rope_pointers(a, head_dim);
  if (st != PA_OK) return st;
  if (!k_scale || !v_scale || ((uintptr_t)k_scale & 3u) || ((uintptr_t)v_scale & 3u))
    return PA_ERR_INVALID_ARG;
  cudaError_t e;
  if (dtype == PA_BFLOAT16)
    e = head_dim == 128 ? launch_q8<PA_BFLOAT16, 128>(a, stream)
                        : launch_q8<PA_BFLOAT16, 64>(a, stream);
  else
    e = head_dim == 128 ? launch_q8<PA_FLOAT16, 128>(a, stream)
                        : launch_q8<PA_FLOAT16, 64>(a, stream);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
