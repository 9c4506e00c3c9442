// pa_decode_tree: decode attention of several new tokens per sequence, a chain or a tree,
// over the paged cache (the kernel: pa_multi.cuh).
#include "pa_common.cuh"
#include "pa_internal.h"
#include "pa_multi.cuh"

namespace pa {
namespace {

// Up to 32 columns the second term of the weights costs nothing: the cache's bytes take longer.
// With 64 it costs 11% (16-token trees of 64 sequences, 121 us for 108) to 26% (a 60-token tree
// over 50,001 tokens, 185 us for 147), its rows shared memory that tiles are on their way to:
// there the caller chooses.
template <int N>
using Tree128 = multi::Shape<128, 2, 2, false, N, N <= 32 ? 2 : 1>;
template <int N>
using Tree64 = multi::Shape<128, 1, 1, false, N, N <= 32 ? 2 : 1>;
template <int N>
using Exact128 = multi::Shape<128, 2, 2, false, N, 2>;
template <int N>
using Exact64 = multi::Shape<128, 1, 1, false, N, 2>;

template <int DT, class... X>
cudaError_t launch_tree(const multi::Call& c, int head_dim, int n, X&&... x) {
  // up to 32 columns both are one shape
  if (head_dim == 128)
    return multi::two_terms(c) ? multi::launch_columns<Exact128, DT>(n, x...)
                               : multi::launch_columns<Tree128, DT>(n, x...);
  return multi::two_terms(c) ? multi::launch_columns<Exact64, DT>(n, x...)
                             : multi::launch_columns<Tree64, DT>(n, x...);
}

}  // namespace
}  // namespace pa

using namespace pa;

// Host checks shared by the call and its workspace query.
static pa_status check_tree(int num_q_heads, int num_kv_heads, int head_dim, int max_q_len) {
  if (num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads || max_q_len < 0 ||
      (int64_t)max_q_len * (num_q_heads / num_kv_heads) > 65536)
    return PA_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

extern "C" size_t pa_decode_tree_workspace_bytes(int num_q_heads, int num_kv_heads, int head_dim,
                                                 int max_q_len) {
  if (check_tree(num_q_heads, num_kv_heads, head_dim, max_q_len) != PA_OK) return 0;
  return multi::layout_of(
             multi::columns_for(max_q_len > 1 ? max_q_len : 1, num_q_heads / num_kv_heads).n,
             head_dim).total;
}

extern "C" pa_status pa_decode_tree(void* out, const void* q, const void* k_pool,
                                    const void* v_pool, const int32_t* block_tables,
                                    const int32_t* seq_lens, const int32_t* q_start,
                                    const int32_t* tree_mask, int num_seqs, int total_q,
                                    int num_q_heads, int num_kv_heads, int head_dim,
                                    int block_size, int max_blocks, int num_blocks, int max_q_len,
                                    int mask_words, int max_seq_len, float scale, int dtype,
                                    void* workspace, size_t workspace_bytes, int32_t* status_dev,
                                    cudaStream_t stream) {
  pa_status st = check_tree(num_q_heads, num_kv_heads, head_dim, max_q_len);
  if (st != PA_OK) return st;
  const multi::Call c = {out, q, k_pool, v_pool, block_tables, seq_lens, q_start, tree_mask,
                         num_seqs, total_q, num_q_heads, num_kv_heads, block_size, max_blocks,
                         num_blocks, max_q_len, mask_words, max_seq_len, scale, dtype, workspace,
                         workspace_bytes, status_dev, stream};
  const bool bf16 = multi::storage(c) == PA_BFLOAT16;
  bool work;
  st = multi::check(c, pa_decode_tree_workspace_bytes(num_q_heads, num_kv_heads, head_dim,
                                                      max_q_len), &work);
  if (st != PA_OK || !work) return st;
  return multi::run(c, Tree128<16>::TOK, head_dim, head_dim / 64, true, multi::kWidest,
                    [&](int n, auto&&... x) {
    return bf16 ? launch_tree<PA_BFLOAT16>(c, head_dim, n, x..., stream)
                : launch_tree<PA_FLOAT16>(c, head_dim, n, x..., stream);
  });
}
