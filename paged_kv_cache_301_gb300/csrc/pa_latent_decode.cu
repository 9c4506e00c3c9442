// pa_latent_decode: attention in the absorbed form over the latent cache (the kernel:
// pa_multi.cuh).
#include "pa_common.cuh"
#include "pa_internal.h"
#include "pa_multi.cuh"

namespace pa {
namespace {

// A tile of 64 tokens of 576 elements is 72 KB; two of them and 64 columns of q fill an SM's
// shared memory, with the weights over the tile's rotated part, which S alone needs.  Up to 32
// columns the second term of the weights costs nothing: the cache's bytes take longer.  With 64
// it has no room there, so that a caller who asks for it gets groups of 32 columns (128 heads of 64
// sequences 129 us for 77; 48 columns over eight sequences to 131,072 tokens 255 us for 138).
constexpr int kTwoTerms = 32;
template <int N>
using Latent512 = multi::Shape<64, 9, 8, true, N, N <= kTwoTerms ? 2 : 1>;
template <int N>
using Latent256 = multi::Shape<128, 5, 4, true, N, N <= kTwoTerms ? 2 : 1>;

}  // namespace
}  // namespace pa

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
  return multi::layout_of(multi::columns_for(max_q_len > 1 ? max_q_len : 1, num_q_heads).n,
                          latent_dim).total;
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
  pa_status st = check_latent(num_q_heads, latent_dim, rope_dim, max_q_len);
  if (st != PA_OK) return st;
  const multi::Call c = {out, q, pool, pool, block_tables, seq_lens, q_start, tree_mask, num_seqs,
                         total_q, num_q_heads, 1, block_size, max_blocks, num_blocks, max_q_len,
                         mask_words, max_seq_len, scale, dtype, workspace, workspace_bytes,
                         status_dev, stream};
  const bool bf16 = multi::storage(c) == PA_BFLOAT16;
  bool work;
  st = multi::check(c, pa_latent_decode_workspace_bytes(num_q_heads, latent_dim, rope_dim,
                                                        max_q_len), &work);
  if (st != PA_OK || !work) return st;
  return multi::run(c, latent_dim == 512 ? Latent512<16>::TOK : Latent256<16>::TOK, latent_dim,
                    (latent_dim + rope_dim) / 64, false,
                    multi::two_terms(c) ? kTwoTerms : multi::kWidest, [&](int n, auto&&... x) {
    if (latent_dim == 512)
      return bf16 ? multi::launch_columns<Latent512, PA_BFLOAT16>(n, x..., stream)
                  : multi::launch_columns<Latent512, PA_FLOAT16>(n, x..., stream);
    return bf16 ? multi::launch_columns<Latent256, PA_BFLOAT16>(n, x..., stream)
                : multi::launch_columns<Latent256, PA_FLOAT16>(n, x..., stream);
  });
}
