// pa_latent_prefill: causal attention in the expanded form of latent attention.
#include <math.h>

#include "pa_common.cuh"
#include "pa_internal.h"
#include "pa_rows.cuh"

using namespace pa;

extern "C" pa_status pa_latent_prefill(void* out, const void* q, const void* kv,
                                       const void* key_rope, const int32_t* q_start,
                                       const int32_t* kv_start, int num_seqs, int total_q,
                                       int total_kv, int64_t key_token_stride, int num_heads,
                                       int nope_dim, int rope_dim, int value_dim, int max_q_len,
                                       float scale, int dtype, int32_t* status_dev,
                                       cudaStream_t stream) {
  if (num_seqs < 0 || total_q < 0 || total_kv < 0 || num_heads <= 0 || max_q_len < 0 ||
      !isfinite(scale) || (int64_t)total_q * num_heads >= (1ll << 31) ||
      (int64_t)total_kv * num_heads >= (1ll << 31))
    return PA_ERR_INVALID_ARG;
  if (nope_dim != 128 || rope_dim != 64 || value_dim != 128 ||
      (dtype != PA_FLOAT16 && dtype != PA_BFLOAT16))
    return PA_ERR_UNSUPPORTED;
  if (key_token_stride == 0) key_token_stride = rope_dim;
  if (key_token_stride < rope_dim || key_token_stride % 8) return PA_ERR_INVALID_ARG;
  if (num_seqs == 0 || total_q == 0 || max_q_len == 0) return PA_OK;
  if (!out || !q || !q_start || !kv_start || (total_kv > 0 && (!kv || !key_rope)))
    return PA_ERR_INVALID_ARG;
  if ((((uintptr_t)out | (uintptr_t)q | (uintptr_t)kv | (uintptr_t)key_rope) & 15u) != 0)
    return PA_ERR_INVALID_ARG;
  RowsArgs a = {};
  a.out = out;
  a.q = q;
  a.k = kv;
  a.key_rope = key_rope;
  a.q_start = q_start;
  a.kv_start = kv_start;
  a.key_stride = key_token_stride;
  a.B = num_seqs;
  a.total_q = total_q;
  a.total_kv = total_kv;
  a.Hq = num_heads;
  a.H = num_heads;
  a.max_q = max_q_len;
  a.scale_log2 = (float)((double)scale * 1.4426950408889634);
  a.status_dev = status_dev;
  return launch_rows<192, 128, kRowsExpanded>(a, dtype, stream) == cudaSuccess ? PA_OK
                                                                               : PA_ERR_CUDA;
}
