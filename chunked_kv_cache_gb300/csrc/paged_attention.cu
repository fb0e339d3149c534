// paged_attention.cu -- the paged cache's attention: which page type's launcher a call takes.
#include "sr_paged.h"

namespace sr {

cudaError_t attn_prepare_bf16(int head_dim);
cudaError_t attn_launch_bf16(const PagedAttnParams& p, cudaStream_t st);
cudaError_t rows_launch_bf16(const PagedRowsParams& p, cudaStream_t st);
int attn_tile_tokens_bf16(int head_dim);
cudaError_t attn_prepare_e4m3(int head_dim);
cudaError_t attn_launch_e4m3(const PagedAttnParams& p, cudaStream_t st);
cudaError_t rows_launch_e4m3(const PagedRowsParams& p, cudaStream_t st);
int attn_tile_tokens_e4m3(int head_dim);
cudaError_t attn_prepare_int4(int head_dim);
cudaError_t attn_launch_int4(const PagedAttnParams& p, cudaStream_t st);
cudaError_t rows_launch_int4(const PagedRowsParams& p, cudaStream_t st);
int attn_tile_tokens_int4(int head_dim);

namespace {
template <typename F>
auto by_type(int page_type, F&& bf16, F&& e4m3, F&& int4) {
  return page_type == SR_PAGE_BF16 ? bf16 : page_type == SR_PAGE_E4M3 ? e4m3 : int4;
}
}  // namespace

size_t paged_part_floats(int rows, int head_dim) { return (static_cast<size_t>(rows) * (head_dim + 2) + 3) / 4 * 4; }
int paged_tile_tokens(int head_dim, int page_type) {
  return by_type(page_type, &attn_tile_tokens_bf16, &attn_tile_tokens_e4m3, &attn_tile_tokens_int4)(head_dim);
}
cudaError_t paged_attn_prepare(int head_dim, int page_type) {
  return by_type(page_type, &attn_prepare_bf16, &attn_prepare_e4m3, &attn_prepare_int4)(head_dim);
}
int64_t paged_score_tiles(int64_t pool_tokens, int n_seqs, int n_kv, int tile_tokens) {
  return (pool_tokens / tile_tokens + static_cast<int64_t>(n_seqs) * (1 + kPagedItemCost)) * n_kv;
}

cudaError_t launch_paged_attention(const PagedAttnParams& p, cudaStream_t st) {
  return by_type(p.c.page_type, &attn_launch_bf16, &attn_launch_e4m3, &attn_launch_int4)(p, st);
}
cudaError_t launch_paged_rows(const PagedRowsParams& p, cudaStream_t st) {
  return by_type(p.c.page_type, &rows_launch_bf16, &rows_launch_e4m3, &rows_launch_int4)(p, st);
}

}  // namespace sr
