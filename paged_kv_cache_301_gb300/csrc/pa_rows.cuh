// Attention of several query tokens per sequence on CUDA cores: one CTA to a query row
// and head.  Its warps take the visible tokens in turn, a token's key spread over the
// lanes, with a running maximum and sum each; the four are merged at the end.
#pragma once

#include <math_constants.h>

#include "pa_common.cuh"

namespace pa {

struct RowsArgs {
  void* out;
  const void* q;
  const void* k;                 // pool or expanded rows
  const void* v;
  const void* key_rope;
  const int32_t* tables;
  const int32_t* lens;
  const int32_t* q_start;
  const int32_t* kv_start;
  const int32_t* mask;
  int64_t key_stride;
  int B, total_q, total_kv, Hq, H, bs, max_blocks, num_blocks, max_q, words, max_len;
  float scale_log2;
  int32_t* status_dev;
};

constexpr int kRowsWarps = 4;

enum { kRowsTree = 0, kRowsLatent = 1, kRowsExpanded = 2 };

template <int DT, int DK, int DV, int MODE>
__global__ void __launch_bounds__(32 * kRowsWarps) rows_kernel(const RowsArgs a) {
  __shared__ float s_m[kRowsWarps], s_l[kRowsWarps], s_acc[kRowsWarps][DV];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int hq = blockIdx.y, row = blockIdx.x;
  int b = row, i = 0, n = 1;
  if (a.q_start) {
    int lo = 0, hi = a.B;
    while (lo < hi) {                            // sequences that end at or before row
      const int mid = (lo + hi) / 2;
      if (a.q_start[mid + 1] <= row) lo = mid + 1; else hi = mid;
    }
    b = lo;
    if (b >= a.B) return;
    const int qs = a.q_start[b], qe = a.q_start[b + 1];
    n = qe - qs;
    i = row - qs;
    if (qs < 0 || i < 0 || qe > a.total_q) {
      if (threadIdx.x == 0) report(a.status_dev, PA_ERR_BAD_BLOCK_ID);
      return;
    }
  }
  int L, ks = 0;
  bool bad;
  if (MODE == kRowsExpanded) {
    ks = a.kv_start[b];
    const int ke = a.kv_start[b + 1];
    L = ke - ks;
    bad = ks < 0 || ke > a.total_kv;
  } else {
    L = a.lens[b];
    bad = L < 0 || L > a.max_len || (int64_t)L > (int64_t)a.max_blocks * a.bs;
  }
  if (!a.q_start && L == 0) n = 0;
  if (bad || n > L || n > a.max_q) {
    if (threadIdx.x == 0) report(a.status_dev, PA_ERR_BAD_BLOCK_ID);
    return;
  }
  const int ctx = L - n, h = hq / (a.Hq / a.H);
  const uint32_t* qr = static_cast<const uint32_t*>(a.q) + ((int64_t)row * a.Hq + hq) * (DK / 2);
  float2 q[DK / 64];
#pragma unroll
  for (int e = 0; e < DK / 64; ++e) q[e] = widen2<DT>(qr[lane + 32 * e]);
  float m = -CUDART_INF_F, l = 0.f, acc[DV / 64][2] = {};
  for (int t = warp; t < L; t += kRowsWarps) {
    if (t >= ctx) {
      const int j = t - ctx;
      const bool sees = a.mask ? (a.mask[(int64_t)row * a.words + (j >> 5)] >> (j & 31)) & 1
                               : j <= i;
      if (!sees) continue;
    }
    const uint32_t *k1, *k2, *v;
    int split = DK / 2;                          // words of k1
    bool live = true;
    if (MODE == kRowsExpanded) {
      k1 = static_cast<const uint32_t*>(a.k) + ((int64_t)(ks + t) * a.Hq + hq) * 128;
      k2 = static_cast<const uint32_t*>(a.key_rope) + (int64_t)(ks + t) * (a.key_stride / 2) - 64;
      v = k1 + 64;
      split = 64;
    } else {
      const int id = a.tables[(int64_t)b * a.max_blocks + t / a.bs];
      live = id >= 0 && id < a.num_blocks;
      if (!live && lane == 0) report(a.status_dev, PA_ERR_BAD_BLOCK_ID);
      const int64_t slot = live ? (int64_t)id * a.bs + t % a.bs : 0;
      if (MODE == kRowsLatent) {
        k1 = k2 = v = static_cast<const uint32_t*>(a.k) + slot * (DK / 2);
      } else {
        k1 = k2 = static_cast<const uint32_t*>(a.k) + (slot * a.H + h) * (DK / 2);
        v = static_cast<const uint32_t*>(a.v) + (slot * a.H + h) * (DK / 2);
      }
    }
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < DK / 64; ++e) {
      const int w = lane + 32 * e;
      const float2 x = widen2<DT>(live ? (w < split ? k1[w] : k2[w]) : 0u);
      s = fmaf(q[e].x, x.x, fmaf(q[e].y, x.y, s));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    s *= a.scale_log2;
    const float top = fmaxf(m, s);
    const float by = m == -CUDART_INF_F ? 0.f : exp2f(m - top);
    const float p = s == -CUDART_INF_F ? 0.f : exp2f(s - top);
    m = top;
    l = fmaf(l, by, p);
#pragma unroll
    for (int e = 0; e < DV / 64; ++e) {
      const float2 x = widen2<DT>(live ? v[lane + 32 * e] : 0u);
      acc[e][0] = fmaf(acc[e][0], by, p * x.x);
      acc[e][1] = fmaf(acc[e][1], by, p * x.y);
    }
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < DV / 64; ++e) {
    s_acc[warp][2 * (lane + 32 * e)] = acc[e][0];
    s_acc[warp][2 * (lane + 32 * e) + 1] = acc[e][1];
  }
  __syncthreads();
  float top = -CUDART_INF_F, sum = 0.f, by[kRowsWarps];
  for (int w = 0; w < kRowsWarps; ++w) top = fmaxf(top, s_m[w]);
#pragma unroll
  for (int w = 0; w < kRowsWarps; ++w) {
    by[w] = s_m[w] == -CUDART_INF_F ? 0.f : exp2f(s_m[w] - top);
    sum = fmaf(by[w], s_l[w], sum);
  }
  for (int d = threadIdx.x; d < DV; d += 32 * kRowsWarps) {
    float y = 0.f;
#pragma unroll
    for (int w = 0; w < kRowsWarps; ++w)
      if (by[w] != 0.f) y = fmaf(by[w], s_acc[w][d], y);
    static_cast<uint16_t*>(a.out)[((int64_t)row * a.Hq + hq) * DV + d] =
        narrow<DT>(sum == 0.f ? 0.f : y / sum);
  }
}

template <int DK, int DV, int MODE>
cudaError_t launch_rows(const RowsArgs& a, int dtype, cudaStream_t stream) {
  const dim3 grid((unsigned)a.total_q, (unsigned)a.Hq);
  if (dtype == PA_BFLOAT16)
    rows_kernel<PA_BFLOAT16, DK, DV, MODE><<<grid, 32 * kRowsWarps, 0, stream>>>(a);
  else
    rows_kernel<PA_FLOAT16, DK, DV, MODE><<<grid, 32 * kRowsWarps, 0, stream>>>(a);
  return taken(cudaGetLastError());
}

}  // namespace pa
