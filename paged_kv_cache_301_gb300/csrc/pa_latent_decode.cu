// pa_latent_decode: attention in the absorbed form over the latent cache.
#include <math.h>

#include "pa_common.cuh"
#include "pa_internal.h"
#include "pa_rows.cuh"

using namespace pa;

// Host checks shared by the call and its workspace query.
static pa_status check_latent(int num_q_heads, int latent_dim, int rope_dim, int max_q_len) {
  if (num_q_heads <= 0 || max_q_len < 0 || (int64_t)max_q_len * num_q_heads > 65536)
    return PA_ERR_INVALID_ARG;
  if ((latent_dim != 256 && latent_dim != 512) || rope_dim != 64) return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

extern "C" size_t pa_latent_decode_workspace_bytes(int num_q_heads, int latent_dim, int rope_dim,
                                                   int max_q_len) {
  if (check_latent(num_q_heads, latent_dim, rope_dim, max_q_len) != PA_OK) return 0;
  return 256;
}

extern "C" pa_status pa_latent_decode(void* out, const void* q, const void* pool,
                                      const int32_t* block_tables, const int32_t* seq_lens,
                                      const int32_t* q_start, const int32_t* tree_mask,
                                      int num_seqs, int total_q, int num_q_heads, int latent_dim,
                                      int rope_dim, int block_size, int max_blocks,
                                      int num_blocks, int max_q_len, int mask_words,
                                      int max_seq_len, float scale, int dtype, void* workspace,
                                      size_t workspace_bytes, int32_t* status_dev,
                                      cudaStream_t stream) {
  const pa_status st = check_latent(num_q_heads, latent_dim, rope_dim, max_q_len);
  if (st != PA_OK) return st;
  if (num_seqs < 0 || total_q < 0 || max_blocks <= 0 || num_blocks <= 0 || max_seq_len < 0 ||
      max_seq_len >= (1 << 30) || !isfinite(scale) || (!q_start && total_q != num_seqs) ||
      (tree_mask && (mask_words <= 0 || (int64_t)mask_words * 32 < max_q_len)) ||
      (int64_t)num_blocks * block_size >= (1ll << 31) ||
      (int64_t)total_q * num_q_heads >= (1ll << 31))
    return PA_ERR_INVALID_ARG;
  if ((block_size != 8 && block_size != 16 && block_size != 32 && block_size != 64) ||
      (dtype != PA_FLOAT16 && dtype != PA_BFLOAT16))
    return PA_ERR_UNSUPPORTED;
  if (num_seqs == 0 || total_q == 0) return PA_OK;
  if (!out || !q || !pool || !pool || !block_tables || !seq_lens) return PA_ERR_INVALID_ARG;
  if ((((uintptr_t)out | (uintptr_t)q | (uintptr_t)pool | (uintptr_t)pool) & 15u) != 0)
    return PA_ERR_INVALID_ARG;
  if (!workspace || ((uintptr_t)workspace & 255u) || workspace_bytes < pa_latent_decode_workspace_bytes(num_q_heads, latent_dim, rope_dim, max_q_len))
    return PA_ERR_WORKSPACE;
  RowsArgs a = {};
  a.out = out;
  a.q = q;
  a.k = pool;
  a.v = pool;
  a.tables = block_tables;
  a.lens = seq_lens;
  a.q_start = q_start;
  a.mask = tree_mask;
  a.B = num_seqs;
  a.total_q = total_q;
  a.Hq = num_q_heads;
  a.H = 1;
  a.bs = block_size;
  a.max_blocks = max_blocks;
  a.num_blocks = num_blocks;
  a.max_q = q_start ? max_q_len : 1;
  a.words = mask_words;
  a.max_len = max_seq_len;
  a.scale_log2 = (float)((double)scale * 1.4426950408889634);
  a.status_dev = status_dev;
  const cudaError_t e = latent_dim == 512 ? launch_rows<576, 512, kRowsLatent>(a, dtype, stream)
                                          : launch_rows<320, 256, kRowsLatent>(a, dtype, stream);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
