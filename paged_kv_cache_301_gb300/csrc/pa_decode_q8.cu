// pa_decode_q8: decode attention over the 8-bit cache (pa_q8.cuh).
//
//   out = sum_t p_t V_t / sum_t p_t,   p_t = 2^(s_t - m),
//   s_t = log2(e) * scale * q . K_t,   K_t = code * k_scale[block][head], V_t alike
//
// The plain kernel: one CTA per (sequence, query head) walks the sequence 512
// tokens at a time.  A thread takes a token's score, the CTA's threads share
// the running maximum and sum, then a thread takes one element of the output.
#include <math.h>
#include <math_constants.h>

#include "pa_common.cuh"
#include "pa_q8.cuh"

namespace pa {
namespace {

constexpr int kChunk = 512;
constexpr int kThreads = 128;

struct DecodeQ8Args {
  void* out;
  const void* q;
  const uint8_t* k_pool;
  const uint8_t* v_pool;
  const float* k_scale;
  const float* v_scale;
  const int32_t* tables;
  const int32_t* lens;
  int B, Hq, H, bs, max_blocks, num_blocks, max_seq_len;
  float scale_log2;
  int32_t* status_dev;
};

template <int DT, int D>
__global__ void __launch_bounds__(kThreads) decode_q8_plain_kernel(const DecodeQ8Args a) {
  __shared__ float s_q[D], s_p[kChunk], s_red[kThreads / 32];
  allow_next_grid();
  wait_prior_grid();
  const int b = blockIdx.x / a.Hq, hq = blockIdx.x % a.Hq, h = hq / (a.Hq / a.H);
  const int tid = threadIdx.x;
  const int raw = a.lens[b];
  const int L = max(0, min(raw, a.max_seq_len));
  if (L != raw && tid == 0) report(a.status_dev, PA_ERR_BAD_BLOCK_ID);
  const uint16_t* q = static_cast<const uint16_t*>(a.q) + (int64_t)blockIdx.x * D;
  for (int d = tid; d < D; d += kThreads) s_q[d] = widen2<DT>(q[d]).x * a.scale_log2;
  __syncthreads();
  float m = -CUDART_INF_F, l = 0.f, acc = 0.f;
  for (int t0 = 0; t0 < L; t0 += kChunk) {
    const int n = min(kChunk, L - t0);
    float top = -CUDART_INF_F;
    for (int i = tid; i < n; i += kThreads) {
      const int t = t0 + i;
      const int32_t blk = a.tables[(int64_t)b * a.max_blocks + t / a.bs];
      float s = 0.f;
      if (blk >= 0 && blk < a.num_blocks) {
        const int64_t tile = (int64_t)blk * a.H + h;
        const uint32_t* k =
            reinterpret_cast<const uint32_t*>(a.k_pool + (tile * a.bs + t % a.bs) * D);
        for (int d = 0; d < D / 4; ++d) {
          const uint32_t w = k[d];
          const float2 x = e4m3_widen2(w), y = e4m3_widen2(w >> 16);
          s += s_q[4 * d] * x.x + s_q[4 * d + 1] * x.y + s_q[4 * d + 2] * y.x +
               s_q[4 * d + 3] * y.y;
        }
        s *= a.k_scale[tile];
      } else {
        report(a.status_dev, PA_ERR_BAD_BLOCK_ID);
      }
      s_p[i] = s;
      top = fmaxf(top, s);
    }
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    if ((tid & 31) == 0) s_red[tid >> 5] = top;
    __syncthreads();
    for (int w = 0; w < kThreads / 32; ++w) top = fmaxf(top, s_red[w]);
    const float m_new = fmaxf(m, top), alpha = exp2f(m - m_new);
    m = m_new;
    l *= alpha;
    acc *= alpha;
    for (int i = 0; i < n; ++i) {
      const int t = t0 + i;
      const float p = exp2f(s_p[i] - m);
      l += p;
      const int32_t blk = a.tables[(int64_t)b * a.max_blocks + t / a.bs];
      if (tid < D && blk >= 0 && blk < a.num_blocks) {
        const int64_t tile = (int64_t)blk * a.H + h;
        const float v = e4m3_widen2(a.v_pool[(tile * a.bs + t % a.bs) * D + tid]).x;
        acc += p * (v * a.v_scale[tile]);
      }
    }
    __syncthreads();
  }
  if (tid < D)
    static_cast<uint16_t*>(a.out)[(int64_t)blockIdx.x * D + tid] =
        narrow<DT>(L == 0 ? 0.f : acc / l);
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
  return 256;
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
  if (!workspace || ((uintptr_t)workspace & 255u) ||
      workspace_bytes < pa_decode_q8_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                                     block_size, max_seq_len))
    return PA_ERR_WORKSPACE;
  const long long rows = (long long)num_seqs * num_q_heads;
  if (rows > 0x7FFFFFFF) return PA_ERR_INVALID_ARG;
  const DecodeQ8Args a = {out, q, (const uint8_t*)k_pool, (const uint8_t*)v_pool, k_scale, v_scale,
                          block_tables, seq_lens, num_seqs, num_q_heads, num_kv_heads, block_size,
                          max_blocks, num_blocks, max_seq_len,
                          (float)((double)scale * 1.4426950408889634), status_dev};
  const dim3 grid((unsigned)rows);
  cudaError_t e;
  if (dtype == PA_BFLOAT16)
    e = head_dim == 128
            ? launch_pdl(decode_q8_plain_kernel<PA_BFLOAT16, 128>, grid, kThreads, 0, stream, a)
            : launch_pdl(decode_q8_plain_kernel<PA_BFLOAT16, 64>, grid, kThreads, 0, stream, a);
  else
    e = head_dim == 128
            ? launch_pdl(decode_q8_plain_kernel<PA_FLOAT16, 128>, grid, kThreads, 0, stream, a)
            : launch_pdl(decode_q8_plain_kernel<PA_FLOAT16, 64>, grid, kThreads, 0, stream, a);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
