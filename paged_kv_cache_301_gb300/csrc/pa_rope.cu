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
// (length -> table -> slot) for decode steps.  A head row is shared by D/8
// lanes that hold one 16-byte vector each: the norm's sum and the partner of a
// half-split pair are then shuffles inside the group.
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
    n = e - s;
    if (t < s || t >= e || e > a.total_q) {
      *bad = true;
      return p;
    }
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
  return make_uint4(narrow2<DT>(x[0], x[1]), narrow2<DT>(x[2], x[3]), narrow2<DT>(x[4], x[5]),
                    narrow2<DT>(x[6], x[7]));
}

// RMS norm of a head row of D, 8 elements to each of its group's D/8 lanes.  Called by
// whole warps (it shuffles); `on`: the group's row is normed, by weight's 8 elements.
template <int DT, int D>
__device__ __forceinline__ void norm(float (&x)[8], bool on, const uint4& weight, float eps) {
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
  for (int o = D / 16; o; o >>= 1) ss += __shfl_xor_sync(kAll, ss, o);
  if (on) {
    const float r = rsqrtf(ss * (1.f / D) + eps);
    float w[8];
    widen8<DT>(weight, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
  }
}

// A lane's part of a position's angles: cosines and sines of its 8 elements' pairs
// (4 pairs when they are neighbours).
struct Turn {
  float4 c[2], s[2];
};

// angles: the position's row of cos_sin, R/2 cosines, then R/2 sines.
__device__ __forceinline__ Turn load_turn(const float* angles, int R, int interleaved, int li) {
  Turn t = {};
  const float4* c = reinterpret_cast<const float4*>(angles);
  const float4* s = reinterpret_cast<const float4*>(angles + R / 2);
  if (interleaved) {
    if (li * 8 < R) {
      t.c[0] = c[li];
      t.s[0] = s[li];
    }
  } else if (li * 8 < R) {
    const int at = (li < R / 16 ? li : li - R / 16) * 2;
    t.c[0] = c[at];
    t.c[1] = c[at + 1];
    t.s[0] = s[at];
    t.s[1] = s[at + 1];
  }
  return t;
}

// Rotation of a group's row; called by whole warps (it shuffles); `on`: the group's
// row is rotated.
__device__ __forceinline__ void rotate(float (&x)[8], bool on, const Turn& t, int R,
                                       int interleaved, int li) {
  const float c[8] = {t.c[0].x, t.c[0].y, t.c[0].z, t.c[0].w, t.c[1].x, t.c[1].y, t.c[1].z, t.c[1].w};
  const float s[8] = {t.s[0].x, t.s[0].y, t.s[0].z, t.s[0].w, t.s[1].x, t.s[1].y, t.s[1].z, t.s[1].w};
  on = on && li * 8 < R;
  if (interleaved) {
    if (on) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p = x[2 * i], q = x[2 * i + 1];
        x[2 * i] = p * c[i] - q * s[i];
        x[2 * i + 1] = q * c[i] + p * s[i];
      }
    }
  } else if (R > 0) {
    const int half = R / 16;                     // lanes that hold half the rotated part
    const bool first = li < half;
    const int partner = li * 8 < R ? (first ? li + half : li - half) : li;
    const int base = (threadIdx.x & 31) - li;    // first lane of the group
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(kAll, x[i], base + partner);
    if (on) {
      const float sign = first ? -1.f : 1.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = x[i] * c[i] + sign * (y[i] * s[i]);
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

// All rows of token t, by one CTA: row r < Hq is query head r; with
// KV16 the keys and values of the 16-bit cache follow.  Groups of D/8 lanes take
// rows in turn, U at a time so that their loads overlap; the first ones, and the
// norms' weights, are asked for before the token's place is looked up, and the
// token's angles once for all of a thread's rows.
template <int DT, int D, bool KV16>
__device__ __forceinline__ void token_rows(const RopeArgs& a, int t) {
  constexpr int TG = D / 8, NG = kRowThreads / TG, U = 3;
  const int lane = threadIdx.x & 31, li = threadIdx.x % TG, grp = threadIdx.x / TG;
  const int rows = KV16 ? a.Hq + 2 * a.H : a.Hq;
  const uint4* q = reinterpret_cast<const uint4*>(a.q) + t * (a.q_stride / 8);
  const uint4* key = reinterpret_cast<const uint4*>(a.key) + t * (a.kv_stride / 8);
  const uint4* value = reinterpret_cast<const uint4*>(a.value) + t * (a.kv_stride / 8);
  uint4 w[U];
  auto load_rows = [&](int r0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * NG + grp;
      w[u] = make_uint4(0, 0, 0, 0);
      if (r < a.Hq) w[u] = q[r * TG + li];
      else if (KV16 && r < a.Hq + a.H) w[u] = key[(r - a.Hq) * TG + li];
      else if (KV16 && r < rows) w[u] = value[(r - a.Hq - a.H) * TG + li];
    }
  };
  load_rows(0);
  uint4 qw = make_uint4(0, 0, 0, 0), kw = qw;
  if (a.q_weight) qw = reinterpret_cast<const uint4*>(a.q_weight)[li];
  if (KV16 && a.k_weight) kw = reinterpret_cast<const uint4*>(a.k_weight)[li];

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
  if (angles) turn = load_turn(angles, a.rotary, a.interleaved, li);
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
      if (r0 + u * NG >= rows) break;
      const bool is_q = r < a.Hq, is_k = KV16 && !is_q && r < a.Hq + a.H;
      float x[8];
      widen8<DT>(w[u], x);
      if (any_norm)
        norm<DT, D>(x, is_q ? a.q_weight != nullptr : is_k && a.k_weight != nullptr, is_q ? qw : kw,
                    a.eps);
      rotate(x, is_q || is_k, turn, a.rotary, a.interleaved, li);
      if (is_q) {
        reinterpret_cast<uint4*>(a.q_out)[((int64_t)t * a.Hq + r) * TG + li] = narrow8<DT>(x);
      } else if (is_k) {
        if (slot >= 0)
          reinterpret_cast<uint4*>(a.k_pool)[(slot * a.H + (r - a.Hq)) * TG + li] = narrow8<DT>(x);
      } else if (KV16 && r < rows && slot >= 0) {
        reinterpret_cast<uint4*>(a.v_pool)[(slot * a.H + (r - a.Hq - a.H)) * TG + li] = w[u];
      }
    }
    r0 += NG * U;
    if (r0 >= rows) break;
    load_rows(r0);
  }
}

// ---------------------------------------------------------------- many tokens --
// One CTA takes a run of tokens through a ring of shared-memory stages: bulk copies
// bring a token's rows in (one contiguous copy each for q, key and value), the
// threads norm and rotate them in place, bulk copies take them out (values without
// passing through registers).  Reads of later tokens and writes of earlier ones are
// in flight all the time, which the register kernel above cannot hold at the
// occupancy its angles leave it.
constexpr int kMaxStages = 4;
constexpr int kPlaced = kRowThreads;           // tokens placed at once, one per thread
constexpr int kStreamTokens = 8;               // tokens per SM from which on it is taken
constexpr uint64_t kStreamLimitNs = 2000000000ull;

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          sm100::smem_addr(dst)),
      "l"(src), "r"(bytes), "r"(sm100::smem_addr(bar))
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

// Tokens [total_q cta / ctas, total_q (cta + 1) / ctas).
template <int DT, int D, bool KV16>
__device__ __forceinline__ void stream_rows(const RopeArgs& a, int cta, int ctas, int stages,
                                            uint8_t* ring) {
  constexpr int TG = D / 8, NG = kRowThreads / TG;
  __shared__ __align__(8) uint64_t full[kMaxStages];
  __shared__ int64_t s_slot[kPlaced];          // pool row of the token (-1: none)
  __shared__ int s_pos[kPlaced];               // row of cos_sin (-1: leave the token alone)
  const int tid = threadIdx.x, li = tid % TG, grp = tid / TG;
  const int t0 = (int)((int64_t)a.total_q * cta / ctas);
  const int n = (int)((int64_t)a.total_q * (cta + 1) / ctas) - t0;
  const uint32_t q_bytes = (uint32_t)(a.Hq * D * 2), kv_bytes = KV16 ? (uint32_t)(a.H * D * 2) : 0;
  const uint32_t stage_bytes = q_bytes + 2 * kv_bytes;
  if (tid == 0) {
    for (int i = 0; i < stages; ++i) sm100::mbar_init(&full[i], 1);
    sm100::fence_mbar_init();
  }
  __syncthreads();
  auto fetch = [&](int i) {                    // thread 0
    uint8_t* to = ring + (uint32_t)(i % stages) * stage_bytes;
    uint64_t* bar = &full[i % stages];
    const int64_t t = t0 + i;
    sm100::mbar_arrive_expect_tx(bar, stage_bytes);
    bulk_load(to, static_cast<const uint16_t*>(a.q) + t * a.q_stride, q_bytes, bar);
    if (KV16) {
      bulk_load(to + q_bytes, static_cast<const uint16_t*>(a.key) + t * a.kv_stride, kv_bytes, bar);
      bulk_load(to + q_bytes + kv_bytes, static_cast<const uint16_t*>(a.value) + t * a.kv_stride,
                kv_bytes, bar);
    }
  };
  if (tid == 0)
    for (int i = 0; i < min(stages, n); ++i) fetch(i);
  uint4 qw = make_uint4(0, 0, 0, 0), kw = qw;
  if (a.q_weight) qw = reinterpret_cast<const uint4*>(a.q_weight)[li];
  if (KV16 && a.k_weight) kw = reinterpret_cast<const uint4*>(a.k_weight)[li];
  const bool any_norm = a.q_weight || (KV16 && a.k_weight);
  const int turned = KV16 ? a.Hq + a.H : a.Hq;
  Turn turn = {}, next = {};
  auto turn_of = [&](int i) {
    const int pos = s_pos[i % kPlaced];
    if (a.rotary && pos >= 0)
      next = load_turn(a.cos_sin + (int64_t)pos * a.rotary, a.rotary, a.interleaved, li);
  };
  bool late = false;
  int fetched = min(stages, n);                // thread 0
  for (int i = 0; i < n; ++i) {
    if (i % kPlaced == 0) {                    // the next tokens' places
      if (i > 0) __syncthreads();
      const int t = t0 + i + tid;
      int64_t slot = -1;
      int pos = -1;
      if (i + tid < n) {
        bool bad;
        const Place at = place_token(a, t, &bad);
        bool ok = at.ok;
        if (ok) angles_of(a, t, at.pos, &ok);
        if (bad || (at.ok && !ok)) report(a.status_dev, PA_ERR_BAD_BLOCK_ID);
        if (ok) {
          pos = a.rotary && a.positions ? a.positions[t] : at.pos;
          if (KV16) {
            const int32_t blk = a.tables[(int64_t)at.b * a.max_blocks + at.pos / a.bs];
            if (blk >= 0 && blk < a.num_blocks) slot = (int64_t)blk * a.bs + at.pos % a.bs;
            else report(a.status_dev, PA_ERR_BAD_BLOCK_ID);
          }
        }
      }
      s_slot[tid] = slot;
      s_pos[tid] = pos;
      __syncthreads();
      turn_of(i);
    }
    turn = next;
    if (i + 1 < n && (i + 1) % kPlaced != 0) turn_of(i + 1);
    const bool live = s_pos[i % kPlaced] >= 0;
    uint8_t* stage = ring + (uint32_t)(i % stages) * stage_bytes;
    late = !sm100::mbar_try_wait(&full[i % stages], (i / stages) & 1) &&
           !sm100::mbar_wait_drain(&full[i % stages], (i / stages) & 1, kStreamLimitNs);
    if (live && !late) {
      for (int r0 = 0; r0 < turned; r0 += NG) {
        const int r = r0 + grp;
        uint4* at = reinterpret_cast<uint4*>(stage) + r * TG + li;
        const bool is_q = r < a.Hq, in = r < turned;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (in) w = *at;
        float x[8];
        widen8<DT>(w, x);
        if (any_norm)
          norm<DT, D>(x, is_q ? a.q_weight != nullptr : KV16 && a.k_weight != nullptr,
                      is_q ? qw : kw, a.eps);
        rotate(x, true, turn, a.rotary, a.interleaved, li);
        if (in) *at = narrow8<DT>(x);
      }
    }
    sm100::fence_async_smem();
    if (__syncthreads_or(late)) {
      late = true;
      break;
    }
    if (tid == 0) {
      if (live) {
        bulk_store(static_cast<uint16_t*>(a.q_out) + (int64_t)(t0 + i) * a.Hq * D, stage, q_bytes);
        const int64_t slot = s_slot[i % kPlaced];
        if (KV16 && slot >= 0) {
          bulk_store(static_cast<uint16_t*>(a.k_pool) + slot * a.H * D, stage + q_bytes, kv_bytes);
          bulk_store(static_cast<uint16_t*>(a.v_pool) + slot * a.H * D, stage + q_bytes + kv_bytes,
                     kv_bytes);
        }
      }
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      // the stage of the token before has been read out: the next one comes in
      asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
      if (i > 0 && fetched < n) fetch(fetched++);
    }
  }
  if (tid == 0) {
    if (late) {                                // copies in flight land before the CTA ends
      report(a.status_dev, PA_ERR_TIMEOUT);
      for (int j = max(0, fetched - stages); j < fetched; ++j)
        sm100::mbar_wait_drain(&full[j % stages], (j / stages) & 1, kStreamLimitNs);
    }
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
}

template <int DT, int D>
__global__ void __launch_bounds__(kRowThreads)
rope_append_kernel(const RopeArgs a) {
  allow_next_grid();
  wait_prior_grid();
  token_rows<DT, D, true>(a, (int)blockIdx.x);
}

template <int DT, int D>
__global__ void __launch_bounds__(kRowThreads, 4)
rope_stream_kernel(const RopeArgs a, int stages) {
  extern __shared__ __align__(128) uint8_t ring[];
  allow_next_grid();
  wait_prior_grid();
  stream_rows<DT, D, true>(a, (int)blockIdx.x, (int)gridDim.x, stages, ring);
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

__device__ __forceinline__ float mag8(const float (&x)[8]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, finite_mag(x[i]));
  return m;
}

__device__ __forceinline__ uint2 quantise8(const float (&x)[8], float inv) {
  return make_uint2(e4m3x4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv),
                    e4m3x4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv));
}

// The new rows [r0, r1) of block j of sequence b, tokens t0 .., for the KV heads from
// h0 on that the CTA's threads cover: a head has kHead threads, whose groups hold
// rows g, g + NG, ...  All older rows are below r0.  Keys are normed and rotated
// twice, for the largest magnitude and for the codes: the raw rows take a quarter
// of the registers.
template <int DT, int D, int BS>
struct BlockShape {
  static constexpr int TG = D / 8;
  static constexpr int kHead = BS * TG < kRowThreads ? BS * TG : kRowThreads;
  static constexpr int kHeads = kRowThreads / kHead;      // heads of a CTA
  static constexpr int NG = kHead / TG, RPT = BS / NG;    // groups, rows of each
};

template <int DT, int D, int BS>
__device__ __forceinline__ void store_block(const RopeArgs& a, int b, int j, int h0, int t0, int r0,
                                            int r1) {
  using S = BlockShape<DT, D, BS>;
  constexpr int TG = S::TG, NG = S::NG, RPT = S::RPT, NW = S::kHead / 32;
  __shared__ float s_mag[kRowThreads / 32][2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int mine = threadIdx.x / S::kHead, h = h0 + mine;
  const int li = threadIdx.x % TG, grp = threadIdx.x % S::kHead / TG;
  const int32_t blk = a.tables[(int64_t)b * a.max_blocks + j];
  if (blk < 0 || blk >= a.num_blocks) {
    if (threadIdx.x == 0) report(a.status_dev, PA_ERR_BAD_BLOCK_ID);
    return;
  }
  const bool in = h < a.H;
  const int64_t tile = (int64_t)blk * a.H + h;
  uint2* kc = static_cast<uint2*>(a.k_pool) + tile * (BS * D / 8);
  uint2* vc = static_cast<uint2*>(a.v_pool) + tile * (BS * D / 8);
  uint4 weight = make_uint4(0, 0, 0, 0), kw[RPT], vw[RPT];
  const float* angles[RPT];
  bool live[RPT], any = false;
#pragma unroll
  for (int u = 0; u < RPT; ++u) {
    const int row = grp + u * NG, t = t0 + row - r0;
    live[u] = in && row >= r0 && row < r1;
    kw[u] = vw[u] = make_uint4(0, 0, 0, 0);
    if (live[u]) {
      kw[u] = reinterpret_cast<const uint4*>(a.key)[t * (a.kv_stride / 8) + h * TG + li];
      vw[u] = reinterpret_cast<const uint4*>(a.value)[t * (a.kv_stride / 8) + h * TG + li];
    }
  }
  if (a.k_weight) weight = reinterpret_cast<const uint4*>(a.k_weight)[li];
  float k_old = 0.f, v_old = 0.f;
  if (in && r0 > 0) {
    k_old = a.k_scale[tile];
    v_old = a.v_scale[tile];
  }
#pragma unroll
  for (int u = 0; u < RPT; ++u) {
    const int row = grp + u * NG;
    angles[u] = nullptr;
    if (live[u]) {
      angles[u] = angles_of(a, t0 + row - r0, j * BS + row, &live[u]);
      if (!live[u] && li == 0) report(a.status_dev, PA_ERR_BAD_BLOCK_ID);
    }
    any |= live[u];
  }
  auto new_key = [&](int u, float (&x)[8]) {   // whole warps
    Turn turn = {};
    if (angles[u]) turn = load_turn(angles[u], a.rotary, a.interleaved, li);
    widen8<DT>(kw[u], x);
    if (a.k_weight) norm<DT, D>(x, true, weight, a.eps);
    rotate(x, true, turn, a.rotary, a.interleaved, li);
  };
  float km = 0.f, vm = 0.f;
#pragma unroll
  for (int u = 0; u < RPT; ++u) {
    float x[8], y[8];
    new_key(u, x);
    widen8<DT>(vw[u], y);
    if (live[u]) {
      km = fmaxf(km, mag8(x));
      vm = fmaxf(vm, mag8(y));
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    km = fmaxf(km, __shfl_xor_sync(kAll, km, o));
    vm = fmaxf(vm, __shfl_xor_sync(kAll, vm, o));
  }
  __syncthreads();                    // the last block's s_mag is read
  if (lane == 0) {
    s_mag[warp][0] = km;
    s_mag[warp][1] = vm;
  }
  if (!__syncthreads_or(any)) return; // no row left to write: scales stay
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    km = fmaxf(km, s_mag[mine * NW + w][0]);
    vm = fmaxf(vm, s_mag[mine * NW + w][1]);
  }
  const float ks = fmaxf(k_old, scale_for(km)), vs = fmaxf(v_old, scale_for(vm));
  const float k_inv = 1.f / ks, v_inv = 1.f / vs;
#pragma unroll
  for (int u = 0; u < RPT; ++u) {
    const int row = grp + u * NG;
    float x[8], y[8];
    new_key(u, x);
    if (live[u]) {
      widen8<DT>(vw[u], y);
      kc[row * TG + li] = quantise8(x, k_inv);
      vc[row * TG + li] = quantise8(y, v_inv);
    } else if (in && row < r0) {
      if (ks > k_old) rescale8(kc + row * TG + li, k_old * k_inv);
      if (vs > v_old) rescale8(vc + row * TG + li, v_old * v_inv);
    }
  }
  if (in && threadIdx.x % S::kHead == 0) {
    a.k_scale[tile] = ks;
    a.v_scale[tile] = vs;
  }
}

// Prompts and chunks.  CTAs [0, kv_ctas) hold a window of tokens (32 at most) and the
// KV heads their threads cover, and write the blocks whose first new token lies in
// the window; the others hold query rows, of one token each or, with stages, a run.
template <int DT, int D, int BS>
__global__ void __launch_bounds__(kRowThreads, 3)
rope_append_q8_kernel(const RopeArgs a, int kv_ctas, int window, int stages) {
  extern __shared__ __align__(128) uint8_t ring[];
  using S = BlockShape<DT, D, BS>;
  allow_next_grid();
  wait_prior_grid();
  if ((int)blockIdx.x >= kv_ctas) {
    const int cta = (int)blockIdx.x - kv_ctas;
    if (stages)
      stream_rows<DT, D, false>(a, cta, (int)gridDim.x - kv_ctas, stages, ring);
    else
      token_rows<DT, D, false>(a, cta);
    return;
  }
  const int lane = threadIdx.x & 31;
  const int parts = (a.H + S::kHeads - 1) / S::kHeads;
  const int h0 = (int)blockIdx.x % parts * S::kHeads, w0 = (int)blockIdx.x / parts * window;
  // each warp places the window's tokens, one per lane
  const int t = w0 + lane;
  const bool in_window = lane < window && t < a.total_q;
  int b = find_seq(a.q_start, a.B, w0, lane);
  for (int base = b;; base += 32) {
    // the 32 boundaries after `base`: count those at or before each lane's token
    const int j = base + 1 + lane;
    const int bound = j <= a.B ? a.q_start[j] : 0x7FFFFFFF;
    int passed = 0;
#pragma unroll
    for (int k = 0; k < 32; ++k) passed += __shfl_sync(kAll, bound, k) <= t ? 1 : 0;
    const bool more = in_window && passed == 32;
    if (b == base) b += passed;
    if (!__any_sync(kAll, more)) break;
  }
  Place at = {b, 0, 0};
  bool bad = false;
  if (in_window) at = place_of(a, b, t, &bad);
  int begins = 0, n_here = 0;
  if (at.ok) {
    const int row = at.pos % BS;
    begins = row == 0 || t == a.q_start[b];
    n_here = min(a.q_start[b + 1] - t, BS - row);   // its sequence's rows in this block
  }
  for (uint32_t todo = __ballot_sync(kAll, begins); todo; todo &= todo - 1) {
    const int src = __ffs(todo) - 1;
    const int bb = __shfl_sync(kAll, at.b, src), pos = __shfl_sync(kAll, at.pos, src);
    const int n = __shfl_sync(kAll, n_here, src);
    store_block<DT, D, BS>(a, bb, pos / BS, h0, w0 + src, pos % BS, pos % BS + n);
  }
}

// A decode step: one new token per sequence.  CTAs [0, kv_ctas): each group of
// D/8 lanes takes the K or the V row of one (sequence, KV head); the others hold
// one token's query rows.
template <int DT, int D>
__global__ void __launch_bounds__(kRowThreads)
rope_step_q8_kernel(const RopeArgs a, int kv_ctas) {
  constexpr int TG = D / 8, NG = kRowThreads / TG;
  allow_next_grid();
  wait_prior_grid();
  if ((int)blockIdx.x >= kv_ctas) {
    token_rows<DT, D, false>(a, (int)blockIdx.x - kv_ctas);
    return;
  }
  const int li = threadIdx.x % TG;
  const int64_t item = (int64_t)blockIdx.x * NG + threadIdx.x / TG;
  const bool is_v = item & 1;
  const int h = (int)((item >> 1) % a.H);
  const int64_t b64 = (item >> 1) / a.H;
  const bool in = b64 < a.B;
  const int b = in ? (int)b64 : 0;
  uint4 w = make_uint4(0, 0, 0, 0);
  if (in)
    w = reinterpret_cast<const uint4*>(is_v ? a.value : a.key)[b * (a.kv_stride / 8) + h * TG + li];
  uint4 weight = make_uint4(0, 0, 0, 0);
  if (a.k_weight) weight = reinterpret_cast<const uint4*>(a.k_weight)[li];
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
  if (angles && !is_v) turn = load_turn(angles, a.rotary, a.interleaved, li);
  float x[8];
  widen8<DT>(w, x);
  if (a.k_weight) norm<DT, D>(x, !is_v, weight, a.eps);
  rotate(x, !is_v, turn, a.rotary, a.interleaved, li);
  float m = mag8(x);
#pragma unroll
  for (int o = TG / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
  const float s = fmaxf(old, scale_for(m)), inv = 1.f / s;
  if (!ok) return;
  uint2* codes = static_cast<uint2*>(is_v ? a.v_pool : a.k_pool) + tile * a.bs * TG;
  codes[row * TG + li] = quantise8(x, inv);
  if (s > old) {
    for (int r = 0; r < row; ++r) rescale8(codes + r * TG + li, old * inv);
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
// register kernel), bytes of them, CTAs.
struct Stream {
  int stages, bytes, ctas;
};

pa_status plan_stream(int tokens, int rows, int head_dim, int most, Stream* s) {
  *s = {0, 0, tokens};
  int device = 0, sms = 0;
  if (cudaGetDevice(&device) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess)
    return PA_ERR_CUDA;
  if (tokens < kStreamTokens * sms) return PA_OK;
  // `most` CTAs of an SM where two stages of each fit its shared memory, else fewer
  const int64_t token = (int64_t)rows * head_dim * 2;
  for (int per_sm = most; per_sm; --per_sm) {
    const int64_t room = (227 * 1024) / per_sm - 5 * 1024;
    if (2 * token > room) continue;
    s->stages = (int)(room / token < kMaxStages ? room / token : kMaxStages);
    s->bytes = (int)(s->stages * token);
    s->ctas = sms * per_sm;
    break;
  }
  return PA_OK;
}

// Shared memory above 48 KB, static included, has to be asked for.
template <typename K>
cudaError_t allow_smem(K* kernel, int bytes) {
  if (bytes <= 44 * 1024) return cudaSuccess;
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <int DT, int D, int BS>
cudaError_t launch_blocks(const RopeArgs& a, const Stream& s, cudaStream_t stream) {
  // a window's blocks are written one after another: about as many tokens as a
  // sequence has, a block's at most
  int window = BS < 32 ? BS : 32;
  while (window > 1 && (int64_t)window * a.B > a.total_q) window /= 2;
  constexpr int heads = BlockShape<DT, D, BS>::kHeads;
  const int64_t kv = ((int64_t)a.total_q + window - 1) / window * ((a.H + heads - 1) / heads);
  if (kv + s.ctas > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const cudaError_t e = allow_smem(rope_append_q8_kernel<DT, D, BS>, s.bytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(rope_append_q8_kernel<DT, D, BS>, dim3((unsigned)(kv + s.ctas)), kRowThreads,
                    s.bytes, stream, a, (int)kv, window, s.stages);
}

template <int DT, int D>
cudaError_t launch_q8(const RopeArgs& a, cudaStream_t stream) {
  constexpr int TG = D / 8;
  if (!a.q_start) {
    const int64_t groups = (int64_t)a.B * a.H * 2, per = kRowThreads / TG;
    const int64_t kv = (groups + per - 1) / per;
    if (kv + a.total_q > 0x7FFFFFFF) return cudaErrorInvalidValue;
    return launch_pdl(rope_step_q8_kernel<DT, D>, dim3((unsigned)(kv + a.total_q)), kRowThreads, 0,
                      stream, a, (int)kv);
  }
  Stream s;
  if (plan_stream(a.total_q, a.Hq, D, 3, &s) != PA_OK) return cudaErrorUnknown;
  switch (a.bs) {
    case 8: return launch_blocks<DT, D, 8>(a, s, stream);
    case 16: return launch_blocks<DT, D, 16>(a, s, stream);
    case 32: return launch_blocks<DT, D, 32>(a, s, stream);
    default: return launch_blocks<DT, D, 64>(a, s, stream);
  }
}

template <int DT, int D>
cudaError_t launch_16(const RopeArgs& a, cudaStream_t stream) {
  Stream s;
  if (plan_stream(a.total_q, a.Hq + 2 * a.H, D, 4, &s) != PA_OK) return cudaErrorUnknown;
  if (!s.stages)
    return launch_pdl(rope_append_kernel<DT, D>, dim3((unsigned)a.total_q), kRowThreads, 0, stream,
                      a);
  const cudaError_t e = allow_smem(rope_stream_kernel<DT, D>, s.bytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(rope_stream_kernel<DT, D>, dim3((unsigned)s.ctas), kRowThreads, s.bytes,
                    stream, a, s.stages);
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
