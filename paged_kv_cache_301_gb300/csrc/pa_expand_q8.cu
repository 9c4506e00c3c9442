// pa_expand_blocks_q8: blocks of the 8-bit cache (pa_q8.cuh) back to blocks of a
// 16-bit pool, value = code * scale.
//
// bf16 holds every such product exactly; fp16 rounds below its normal range.
// One byte is read and two are written per element, so the bound is 3 bytes per
// element at HBM bandwidth.  The two layouts differ in order: codes are
// [head][row][dim], the 16-bit block is [row][head][dim].  Threads run in the
// order of the 16-bit block, eight codes each, so that a warp's stores are one
// contiguous 512 bytes and its loads are whole 64- or 128-byte rows (16 codes each, with
// stores 32 bytes apart: 70 us).  Four such vectors of K and of V are in flight per
// thread.  Measured: 65,536 tokens of 8 heads of 128, 403 MB, 62.7 us, 6.43 TB/s, 0.96 of
// a plain copy; a handful of blocks 2.1 us.
#include "pa_common.cuh"
#include "pa_q8.cuh"

namespace pa {
namespace {

constexpr int kExpandThreads = 256;
constexpr int kExpandVecs = 4;      // 8-code vectors per thread and pool

struct ExpandArgs {
  uint4* k_out;
  uint4* v_out;
  const uint2* k8;
  const uint2* v8;
  const float* k_scale;
  const float* v_scale;
  const int32_t* pairs;
  int H, bs, vecs, chunks;          // vecs: 8-code vectors of a block and pool
  int src_blocks, dst_blocks;
  int32_t* status_dev;
};

template <int DT>
__device__ __forceinline__ uint32_t expand2(uint32_t codes, float scale) {
  const float2 c = e4m3_widen2(codes);
  const float a = c.x * scale, b = c.y * scale;
  // past the type's largest value (the code above a magnitude near it): saturate; NaN stays
  uint32_t d;
  if (DT == PA_FLOAT16)
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
  else
    asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
  return d;
}

template <int DT, int D>
__global__ void __launch_bounds__(kExpandThreads) expand_q8_kernel(const ExpandArgs a) {
  constexpr int RV = D / 8;         // vectors of a head's row
  allow_next_grid();
  wait_prior_grid();
  const int pair = (int)blockIdx.x / a.chunks, chunk = (int)blockIdx.x - pair * a.chunks;
  const int32_t src = a.pairs[2 * (int64_t)pair], dst = a.pairs[2 * (int64_t)pair + 1];
  if (src < 0 || src >= a.src_blocks || dst < 0 || dst >= a.dst_blocks) {
    if (threadIdx.x == 0 && chunk == 0) report(a.status_dev, PA_ERR_BAD_BLOCK_ID);
    return;
  }
  const int64_t from = (int64_t)src * a.vecs, to = (int64_t)dst * a.vecs;
  const int i0 = chunk * (kExpandThreads * kExpandVecs) + (int)threadIdx.x;
  uint2 w[kExpandVecs][2];
  float s[kExpandVecs][2];
#pragma unroll
  for (int u = 0; u < kExpandVecs; ++u) {
    const int i = i0 + u * kExpandThreads;
    if (i < a.vecs) {
      const int d = i % RV, rh = i / RV, h = rh % a.H, row = rh / a.H;
      const int64_t at = from + (int64_t)(h * a.bs + row) * RV + d;
      w[u][0] = a.k8[at];
      w[u][1] = a.v8[at];
      s[u][0] = a.k_scale[(int64_t)src * a.H + h];
      s[u][1] = a.v_scale[(int64_t)src * a.H + h];
    }
  }
#pragma unroll
  for (int u = 0; u < kExpandVecs; ++u) {
    const int i = i0 + u * kExpandThreads;
    if (i < a.vecs) {
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const uint2 c = w[u][p];
        const float f = s[u][p];
        (p ? a.v_out : a.k_out)[to + i] =
            make_uint4(expand2<DT>(c.x, f), expand2<DT>(c.x >> 16, f), expand2<DT>(c.y, f),
                       expand2<DT>(c.y >> 16, f));
      }
    }
  }
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" pa_status pa_expand_blocks_q8(void* k_pool, void* v_pool, const void* k_pool8,
                                         const void* v_pool8, const float* k_scale,
                                         const float* v_scale, const int32_t* block_pairs,
                                         int num_pairs, int num_kv_heads, int head_dim,
                                         int block_size, int src_num_blocks, int dst_num_blocks,
                                         int dtype, int32_t* status_dev, cudaStream_t stream) {
  if (num_pairs < 0 || num_kv_heads <= 0 || src_num_blocks <= 0 || dst_num_blocks <= 0)
    return PA_ERR_INVALID_ARG;
  if (!(head_dim == 64 || head_dim == 128)) return PA_ERR_UNSUPPORTED;
  if (!(block_size == 8 || block_size == 16 || block_size == 32 || block_size == 64))
    return PA_ERR_UNSUPPORTED;
  if (dtype != PA_FLOAT16 && dtype != PA_BFLOAT16) return PA_ERR_UNSUPPORTED;
  if (num_pairs == 0) return PA_OK;
  if (!k_pool || !v_pool || !k_pool8 || !v_pool8 || !k_scale || !v_scale || !block_pairs)
    return PA_ERR_INVALID_ARG;
  if (!aligned16(k_pool) || !aligned16(v_pool) || !aligned16(k_pool8) || !aligned16(v_pool8) ||
      ((uintptr_t)k_scale & 3u) || ((uintptr_t)v_scale & 3u))
    return PA_ERR_INVALID_ARG;
  const int64_t vecs = (int64_t)block_size * num_kv_heads * head_dim / 8;
  if (vecs > (1 << 25)) return PA_ERR_INVALID_ARG;
  const int per = kExpandThreads * kExpandVecs;
  const int64_t chunks = (vecs + per - 1) / per;
  if (chunks * num_pairs > 0x7FFFFFFF) return PA_ERR_INVALID_ARG;
  const ExpandArgs a = {(uint4*)k_pool, (uint4*)v_pool, (const uint2*)k_pool8,
                        (const uint2*)v_pool8, k_scale, v_scale, block_pairs, num_kv_heads,
                        block_size, (int)vecs, (int)chunks, src_num_blocks, dst_num_blocks,
                        status_dev};
  const dim3 grid((unsigned)(chunks * num_pairs));
  cudaError_t e;
  if (dtype == PA_BFLOAT16)
    e = head_dim == 128
            ? launch_pdl(expand_q8_kernel<PA_BFLOAT16, 128>, grid, kExpandThreads, 0, stream, a)
            : launch_pdl(expand_q8_kernel<PA_BFLOAT16, 64>, grid, kExpandThreads, 0, stream, a);
  else
    e = head_dim == 128
            ? launch_pdl(expand_q8_kernel<PA_FLOAT16, 128>, grid, kExpandThreads, 0, stream, a)
            : launch_pdl(expand_q8_kernel<PA_FLOAT16, 64>, grid, kExpandThreads, 0, stream, a);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
