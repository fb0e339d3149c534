// paged_attention_e4m3.cu -- the paged cache's attention over pages of this type.
#include "paged_attention.cuh"

namespace sr {

cudaError_t attn_prepare_e4m3(int head_dim) { return attn_prepare<SR_PAGE_E4M3>(head_dim); }
cudaError_t attn_launch_e4m3(const PagedAttnParams& p, cudaStream_t st) { return attn_launch<SR_PAGE_E4M3>(p, st); }
cudaError_t rows_launch_e4m3(const PagedRowsParams& p, cudaStream_t st) { return rows_launch<SR_PAGE_E4M3>(p, st); }
int attn_tile_tokens_e4m3(int head_dim) { return attn_tile_tokens<SR_PAGE_E4M3>(head_dim); }

}  // namespace sr
