// paged_attention_bf16.cu -- the paged cache's attention over pages of this type.
#include "paged_attention.cuh"

namespace sr {

cudaError_t attn_prepare_bf16(int head_dim) { return attn_prepare<SR_PAGE_BF16>(head_dim); }
cudaError_t attn_launch_bf16(const PagedAttnParams& p, cudaStream_t st) { return attn_launch<SR_PAGE_BF16>(p, st); }
cudaError_t rows_launch_bf16(const PagedRowsParams& p, cudaStream_t st) { return rows_launch<SR_PAGE_BF16>(p, st); }
int attn_tile_tokens_bf16(int head_dim) { return attn_tile_tokens<SR_PAGE_BF16>(head_dim); }

}  // namespace sr
