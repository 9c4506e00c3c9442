// Writes and reads of the latent cache: pa_latent_append (RMS norm of the latent part,
// rotation of the shared key part and of the queries' rotated parts, cache write) and
// pa_latent_gather (rows of sequences, in order, as one matrix).
//
//   c = x * rsqrt(mean(x^2) + eps) * w,   (r_a, r_b) -> (r_a c_j - r_b s_j, r_b c_j + r_a s_j)
//
// Both only move memory: the bound is bytes / HBM bandwidth for prompts, and for steps the
// chain q_start -> length -> block id -> store.  What a warp moves is found from its token's
// number alone, so its loads are asked for before that chain begins.
//
// Measured (GB300, bf16, latent 512): append of 64 tokens with 16 heads 2.8 us; of 18,432 prompt
// tokens with 32 heads 35.2 us, 5.5 TB/s, 0.81 of a plain copy; gather of 65,536 rows 25.2 us,
// 6.0 TB/s, 0.88.
#include <math.h>

#include "pa_common.cuh"
#include "pa_internal.h"
#include "pa_q8.cuh"
#include "pa_share.h"

namespace pa {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
// Small CTAs, and little to a warp: 18,432 prompt tokens with eight warps of four groups of heads
// 38.5 us, eight of two 37.8, four of two 35.7, two of two 35.2, one of two 57 (an SM holds 32
// CTAs).
constexpr int kWarps = 2;
constexpr int kRope = 64;
constexpr int kHeads = 8;              // query heads that a warp turns at once: four lanes each
constexpr int kChunks = 2;             // such groups of heads to a warp

struct AppendArgs {
  void* pool;
  const void* latent;
  const void* key;
  const void* weight;
  const float* cos_sin;
  const int32_t* positions;
  const void* q;
  void* q_out;
  const int32_t* tables;
  const int32_t* lens;
  const int32_t* q_start;
  int64_t latent_stride, key_stride, q_stride, q_head, out_stride, out_head;
  float eps;
  int max_position, interleaved;
  int B, total_q, Hq, bs, max_blocks, num_blocks;
  int units;                           // warps of a token: its row, and its groups of heads
  int32_t* status_dev;
};

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

// Token t's sequence and its place there; ok: the token is one that is written.
struct Place {
  int b, pos;
  bool ok;
};

// Called by whole warps with a uniform t.
__device__ __forceinline__ Place place_of(const AppendArgs& a, int t, int lane) {
  Place p = {t, 0, false};
  int s = t, n = 1;
  if (a.q_start) {
    p.b = find_seq(a.q_start, a.B, t, lane);
    if (p.b >= a.B) return p;                  // behind the last sequence: left as it was
    s = a.q_start[p.b];
    n = a.q_start[p.b + 1] - s;
  }
  const int L = a.lens[p.b];
  if (!a.q_start && L == 0) return p;          // an empty sequence of a decode step
  if (s < 0 || t < s || t - s >= n || n > a.total_q - s || n > L ||
      (int64_t)L > (int64_t)a.max_blocks * a.bs) {
    if (lane == 0) report(a.status_dev, PA_ERR_BAD_BLOCK_ID);
    return p;
  }
  p.pos = L - n + (t - s);
  p.ok = true;
  return p;
}

// A lane's eight cosines and sines: those of its pairs in a head of kRope elements.
struct Turn {
  float c[8], s[8];
};

__device__ __forceinline__ Turn load_turn(const float* row, int li) {
  Turn t;
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    const float4 c = *reinterpret_cast<const float4*>(row + 8 * li + i);
    const float4 s = *reinterpret_cast<const float4*>(row + kRope / 2 + 8 * li + i);
    t.c[i] = c.x; t.c[i + 1] = c.y; t.c[i + 2] = c.z; t.c[i + 3] = c.w;
    t.s[i] = s.x; t.s[i + 1] = s.y; t.s[i + 2] = s.z; t.s[i + 3] = s.w;
  }
  return t;
}

// The two vectors of eight elements that lane li of a head holds, both halves of its pairs:
// pairs (j, j + 32) vectors li and li + 4, neighbours vectors 2 li and 2 li + 1.
__device__ __forceinline__ int first_vec(int li, int interleaved) {
  return interleaved ? 2 * li : li;
}
__device__ __forceinline__ int second_vec(int li, int interleaved) {
  return interleaved ? 2 * li + 1 : li + 4;
}

template <int DT>
__device__ __forceinline__ void turn(uint4& u, uint4& v, const Turn& t, int interleaved) {
  float x[8], y[8], p[8], q[8];
  widen8<DT>(u, x);
  widen8<DT>(v, y);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // pair i: (x_i, y_i), or neighbours of the 16 elements x, y
    const float a = interleaved ? (i < 4 ? x[2 * i & 7] : y[2 * i & 7]) : x[i];
    const float b = interleaved ? (i < 4 ? x[(2 * i + 1) & 7] : y[(2 * i + 1) & 7]) : y[i];
    p[i] = a * t.c[i] - b * t.s[i];
    q[i] = b * t.c[i] + a * t.s[i];
  }
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = p[i];
      x[2 * i + 1] = q[i];
      y[2 * i] = p[4 + i];
      y[2 * i + 1] = q[4 + i];
    }
    u = narrow8<DT>(x);
    v = narrow8<DT>(y);
  } else {
    u = narrow8<DT>(p);
    v = narrow8<DT>(q);
  }
}

template <int DT, int R>
__global__ void __launch_bounds__(32 * kWarps) latent_append_kernel(const AppendArgs a) {
  constexpr int kVecs = R / 256;               // vectors of c to a lane
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int t = (int)(unit / a.units), part = (int)(unit - (int64_t)t * a.units);
  allow_next_grid();
  wait_prior_grid();
  if (t >= a.total_q) return;
  const int li = lane & 3, v0 = first_vec(li, a.interleaved), v1 = second_vec(li, a.interleaved);
  if (part == 0) {
    const uint4* x = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.latent) +
                                                    t * a.latent_stride);
    uint4 w[kVecs], k0 = {}, k1 = {};
#pragma unroll
    for (int i = 0; i < kVecs; ++i) w[i] = x[lane + 32 * i];
    if (lane < 4) {
      const uint4* k = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.key) +
                                                      t * a.key_stride);
      k0 = k[v0];
      k1 = k[v1];
    }
    const Place p = place_of(a, t, lane);
    if (!p.ok) return;
    const int at = a.positions ? a.positions[t] : p.pos;
    const int id = a.tables[(int64_t)p.b * a.max_blocks + p.pos / a.bs];
    const bool turns = a.cos_sin != nullptr;
    if ((turns && (at < 0 || at >= a.max_position)) || id < 0 || id >= a.num_blocks) {
      if (lane == 0) report(a.status_dev, PA_ERR_BAD_BLOCK_ID);
      return;
    }
    uint4* row = reinterpret_cast<uint4*>(
        static_cast<uint16_t*>(a.pool) + ((int64_t)id * a.bs + p.pos % a.bs) * (R + kRope));
    if (turns && lane < 4) {
      const Turn c = load_turn(a.cos_sin + (int64_t)at * kRope, li);
      turn<DT>(k0, k1, c, a.interleaved);
    }
    if (a.weight) {
      float y[kVecs][8], ss = 0.f;
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        widen8<DT>(w[i], y[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(y[i][e], y[i][e], ss);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(kAll, ss, o);
      const float r = rsqrtf(ss * (1.f / R) + a.eps);
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        float g[8];
        widen8<DT>(static_cast<const uint4*>(a.weight)[lane + 32 * i], g);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[i][e] = y[i][e] * r * g[e];
        w[i] = narrow8<DT>(y[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < kVecs; ++i) row[lane + 32 * i] = w[i];
    if (lane < 4) {
      row[R / 8 + v0] = k0;
      row[R / 8 + v1] = k1;
    }
    return;
  }
  const uint16_t* q = static_cast<const uint16_t*>(a.q) + t * a.q_stride;
  uint16_t* out = static_cast<uint16_t*>(a.q_out) + t * a.out_stride;
  const int h0 = (part - 1) * kChunks * kHeads + (lane >> 2);
  uint4 x[kChunks], y[kChunks];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int h = h0 + c * kHeads;
    if (h < a.Hq) {
      const uint4* row = reinterpret_cast<const uint4*>(q + h * a.q_head);
      x[c] = row[v0];
      y[c] = row[v1];
    }
  }
  const Place p = place_of(a, t, lane);
  if (!p.ok) return;
  if (a.cos_sin) {
    const int at = a.positions ? a.positions[t] : p.pos;
    if (at < 0 || at >= a.max_position) {
      if (lane == 0) report(a.status_dev, PA_ERR_BAD_BLOCK_ID);
      return;
    }
    const Turn c = load_turn(a.cos_sin + (int64_t)at * kRope, li);
#pragma unroll
    for (int i = 0; i < kChunks; ++i) turn<DT>(x[i], y[i], c, a.interleaved);
  }
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int h = h0 + c * kHeads;
    if (h < a.Hq) {
      uint4* row = reinterpret_cast<uint4*>(out + h * a.out_head);
      row[v0] = x[c];
      row[v1] = y[c];
    }
  }
}

struct GatherArgs {
  void* out;
  const void* pool;
  const int32_t* tables;
  const int32_t* lens;
  const int32_t* kv_start;
  int64_t out_stride;
  int B, total, bs, max_blocks, num_blocks;
  int32_t* status_dev;
};

constexpr int kGatherRows = 4;         // rows to a warp (with eight, 65,536 rows 26.2 us, now 25.2)

// Four rows of out to a warp, its lanes side by side over all of them: 4.6 KB asked for at
// once at latent_dim 512.
template <int R>
__global__ void __launch_bounds__(32 * kWarps) latent_gather_kernel(const GatherArgs a) {
  constexpr int kRowVecs = (R + kRope) / 8;
  constexpr int kEach = kGatherRows * kRowVecs / 32;
  static_assert(kGatherRows * kRowVecs % 32 == 0, "whole rounds of a warp");
  const int lane = threadIdx.x & 31;
  const int64_t r0 = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * kGatherRows;
  allow_next_grid();
  wait_prior_grid();
  if (r0 >= a.total) return;
  const int first = find_seq(a.kv_start, a.B, (int)r0, lane);
  // lane i < kGatherRows: the slot of row r0 + i (-1: zeros, -2: not written)
  int64_t slot = -2;
  const int row = (int)r0 + lane;
  if (lane < kGatherRows && r0 + lane < a.total) {
    int b = first;
    while (b < a.B && a.kv_start[b + 1] <= row) ++b;
    if (b < a.B) {
      const int s = a.kv_start[b], n = a.kv_start[b + 1] - s, L = a.lens[b];
      if (s < 0 || row < s || n > a.total - s || n > L ||
          (int64_t)L > (int64_t)a.max_blocks * a.bs) {
        report(a.status_dev, PA_ERR_BAD_BLOCK_ID);
      } else {
        const int at = row - s;
        const int id = a.tables[(int64_t)b * a.max_blocks + at / a.bs];
        slot = -1;
        if (id >= 0 && id < a.num_blocks) slot = (int64_t)id * a.bs + at % a.bs;
        else report(a.status_dev, PA_ERR_BAD_BLOCK_ID);
      }
    }
  }
  const uint4* pool = static_cast<const uint4*>(a.pool);
  uint4 x[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int v = lane + 32 * i, r = v / kRowVecs;
    const int64_t from = __shfl_sync(kAll, slot, r);
    x[i] = from >= 0 ? pool[from * kRowVecs + (v - r * kRowVecs)] : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int v = lane + 32 * i, r = v / kRowVecs;
    const int64_t from = __shfl_sync(kAll, slot, r);
    if (from != -2)
      reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) +
                               (r0 + r) * a.out_stride)[v - r * kRowVecs] = x[i];
  }
}

// Bytes from the first to the last element of rows of `row` elements, `stride` apart.
int64_t span(int64_t rows, int64_t stride, int64_t row) { return 2 * ((rows - 1) * stride + row); }

// Whether n steps of `stride` elements stay within 2^40 elements, so that byte offsets and their
// sums fit 64 bits.
bool within(int64_t n, int64_t stride) {
  const int64_t most = 1ll << 40;
  return stride <= most && (n <= 0 || stride <= most / n);
}

bool known(int latent_dim, int rope_dim, int block_size, int dtype) {
  return (latent_dim == 256 || latent_dim == 512) && rope_dim == kRope &&
         (block_size == 8 || block_size == 16 || block_size == 32 || block_size == 64) &&
         (dtype == PA_FLOAT16 || dtype == PA_BFLOAT16);
}

pa_status check_append(const AppendArgs& a, int R) {
  if (a.q && (!a.q_out || a.Hq <= 0)) return PA_ERR_INVALID_ARG;
  if (!a.q && a.q_out) return PA_ERR_INVALID_ARG;
  if (!a.pool || !a.latent || !a.key || !a.tables || !a.lens) return PA_ERR_INVALID_ARG;
  if (a.cos_sin && a.max_position <= 0) return PA_ERR_INVALID_ARG;
  if ((((uintptr_t)a.pool | (uintptr_t)a.latent | (uintptr_t)a.key | (uintptr_t)a.weight |
        (uintptr_t)a.cos_sin | (uintptr_t)a.q | (uintptr_t)a.q_out) & 15u) != 0)
    return PA_ERR_INVALID_ARG;
  if (((a.latent_stride | a.key_stride) & 7) || a.latent_stride < R || a.key_stride < kRope)
    return PA_ERR_INVALID_ARG;
  if (!within(a.total_q, a.latent_stride) || !within(a.total_q, a.key_stride))
    return PA_ERR_INVALID_ARG;
  const int64_t T = a.total_q, heads = a.Hq;
  const Rows latent = rows_of(a.latent, T, a.latent_stride, 1, 0, R);
  const Rows key = rows_of(a.key, T, a.key_stride, 1, 0, kRope);
  const int64_t pool_bytes = 2 * (int64_t)a.num_blocks * a.bs * (R + kRope);
  const int64_t all = (int64_t)a.B * a.max_blocks, entries = all < 1ll << 60 ? all : 1ll << 60;
  // which rows of the pool are written only the GPU knows: none of it may be read
  auto in_pool = [&](const void* p, int64_t n) { return overlaps(a.pool, pool_bytes, p, n); };
  const struct {
    const void* p;
    int64_t n;
  } whole[] = {{a.weight, 2 * (int64_t)R},
               {a.cos_sin, 4 * (int64_t)a.max_position * kRope},
               {a.positions, 4 * T},
               {a.tables, 4 * entries},
               {a.lens, 4 * (int64_t)a.B},
               {a.q_start, 4 * ((int64_t)a.B + 1)}};
  if (in_pool(latent.base, latent.span()) || in_pool(key.base, key.span()))
    return PA_ERR_INVALID_ARG;
  for (const auto& w : whole)
    if (w.p && in_pool(w.p, w.n)) return PA_ERR_INVALID_ARG;
  if (!a.q) return PA_OK;
  if (!within(a.Hq, a.q_head) || !within(a.Hq, a.out_head) || !within(a.total_q, a.q_stride) ||
      !within(a.total_q, a.out_stride))
    return PA_ERR_INVALID_ARG;
  if (((a.q_stride | a.q_head | a.out_stride | a.out_head) & 7) || a.q_head < kRope ||
      a.out_head < kRope || a.q_stride < (a.Hq - 1) * a.q_head + kRope ||
      a.out_stride < (a.Hq - 1) * a.out_head + kRope)
    return PA_ERR_INVALID_ARG;
  const Rows in = rows_of(a.q, T, a.q_stride, heads, a.q_head, kRope);
  const Rows out = rows_of(a.q_out, T, a.out_stride, heads, a.out_head, kRope);
  if (in_pool(in.base, in.span()) || in_pool(out.base, out.span())) return PA_ERR_INVALID_ARG;
  for (const auto& w : whole)
    if (w.p && overlaps(out.base, out.span(), w.p, w.n)) return PA_ERR_INVALID_ARG;
  if (share(out, latent) || share(out, key)) return PA_ERR_INVALID_ARG;
  // in place, each element read and written by the same lane; else no byte of both
  if (a.q_out == a.q && (T == 1 || a.q_stride == a.out_stride) &&
      (heads == 1 || a.q_head == a.out_head))
    return PA_OK;
  return share(out, in) ? PA_ERR_INVALID_ARG : PA_OK;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" pa_status pa_latent_append(
    void* pool, const void* latent, const void* key_rope, const void* weight, float eps,
    const float* cos_sin, int max_position, int interleaved, const int32_t* positions,
    const void* q_rope, void* q_out, const int32_t* block_tables, const int32_t* seq_lens,
    const int32_t* q_start, int num_seqs, int total_q, int64_t latent_token_stride,
    int64_t key_token_stride, int64_t q_token_stride, int64_t q_head_stride,
    int64_t q_out_token_stride, int64_t q_out_head_stride, int num_q_heads, int latent_dim,
    int rope_dim, int block_size, int max_blocks, int num_blocks, int dtype, int32_t* status_dev,
    cudaStream_t stream) {
  if (!known(latent_dim, rope_dim, block_size, dtype)) return PA_ERR_UNSUPPORTED;
  if (num_seqs < 0 || total_q < 0 || max_blocks <= 0 || num_blocks <= 0 || !(eps >= 0.f) ||
      isinf(eps) || (!q_start && total_q != num_seqs) || latent_token_stride < 0 ||
      key_token_stride < 0 || q_token_stride < 0 || q_head_stride < 0 || q_out_token_stride < 0 ||
      q_out_head_stride < 0 || num_q_heads > (1 << 20))
    return PA_ERR_INVALID_ARG;
  if (num_seqs == 0 || total_q == 0) return PA_OK;
  AppendArgs a;
  a.pool = pool;
  a.latent = latent;
  a.key = key_rope;
  a.weight = weight;
  a.cos_sin = cos_sin;
  a.positions = positions;
  a.q = q_rope;
  a.q_out = q_out;
  a.tables = block_tables;
  a.lens = seq_lens;
  a.q_start = q_start;
  a.latent_stride = latent_token_stride ? latent_token_stride : latent_dim;
  a.key_stride = key_token_stride ? key_token_stride : rope_dim;
  a.q_head = q_head_stride ? q_head_stride : rope_dim;
  a.q_stride = q_token_stride;
  a.out_head = q_out_head_stride ? q_out_head_stride : rope_dim;
  a.out_stride = q_out_token_stride;
  a.eps = eps;
  a.max_position = max_position;
  a.interleaved = interleaved;
  a.B = num_seqs;
  a.total_q = total_q;
  a.Hq = num_q_heads;
  a.bs = block_size;
  a.max_blocks = max_blocks;
  a.num_blocks = num_blocks;
  a.units = 1 + (q_rope ? (num_q_heads + kChunks * kHeads - 1) / (kChunks * kHeads) : 0);
  a.status_dev = status_dev;
  if (within(num_q_heads, a.q_head) && within(num_q_heads, a.out_head)) {
    if (a.q_stride == 0) a.q_stride = num_q_heads * a.q_head;
    if (a.out_stride == 0) a.out_stride = num_q_heads * a.out_head;
  }
  const pa_status st = check_append(a, latent_dim);
  if (st != PA_OK) return st;
  const int64_t ctas = ((int64_t)total_q * a.units + kWarps - 1) / kWarps;
  if (ctas > 0x7FFFFFFF) return PA_ERR_INVALID_ARG;
  auto kernel = dtype == PA_BFLOAT16
                    ? (latent_dim == 512 ? latent_append_kernel<PA_BFLOAT16, 512>
                                         : latent_append_kernel<PA_BFLOAT16, 256>)
                    : (latent_dim == 512 ? latent_append_kernel<PA_FLOAT16, 512>
                                         : latent_append_kernel<PA_FLOAT16, 256>);
  return launch_pdl(kernel, dim3((unsigned)ctas), 32 * kWarps, 0, stream, a) == cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}

extern "C" pa_status pa_latent_gather(void* out, const void* pool, const int32_t* block_tables,
                                      const int32_t* seq_lens, const int32_t* kv_start,
                                      int num_seqs, int total_kv, int64_t out_token_stride,
                                      int latent_dim, int rope_dim, int block_size,
                                      int max_blocks, int num_blocks, int dtype,
                                      int32_t* status_dev, cudaStream_t stream) {
  if (!known(latent_dim, rope_dim, block_size, dtype)) return PA_ERR_UNSUPPORTED;
  const int row = latent_dim + rope_dim;
  if (out_token_stride == 0) out_token_stride = row;
  if (num_seqs < 0 || total_kv < 0 || max_blocks <= 0 || num_blocks <= 0 ||
      out_token_stride < row || (out_token_stride & 7) || !within(total_kv, out_token_stride))
    return PA_ERR_INVALID_ARG;
  if (num_seqs == 0 || total_kv == 0) return PA_OK;
  if (!out || !pool || !block_tables || !seq_lens || !kv_start ||
      (((uintptr_t)out | (uintptr_t)pool) & 15u) != 0)
    return PA_ERR_INVALID_ARG;
  if (overlaps(out, span(total_kv, out_token_stride, row), pool,
               span((int64_t)num_blocks * block_size, row, row)))
    return PA_ERR_INVALID_ARG;
  const GatherArgs a = {out,     pool,     block_tables, seq_lens,   kv_start,  out_token_stride,
                        num_seqs, total_kv, block_size,   max_blocks, num_blocks, status_dev};
  const int rows = kWarps * kGatherRows;
  auto kernel = latent_dim == 512 ? latent_gather_kernel<512> : latent_gather_kernel<256>;
  return launch_pdl(kernel, dim3((unsigned)(((int64_t)total_kv + rows - 1) / rows)), 32 * kWarps,
                    0, stream, a) == cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}
