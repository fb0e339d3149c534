// paged_attention_int4.cu -- the paged cache's attention over pages of this type.
#include "paged_attention.cuh"

namespace sr {

cudaError_t attn_prepare_int4(int head_dim) { return attn_prepare<SR_PAGE_INT4>(head_dim); }
cudaError_t attn_launch_int4(const PagedAttnParams& p, cudaStream_t st) { return attn_launch<SR_PAGE_INT4>(p, st); }
cudaError_t rows_launch_int4(const PagedRowsParams& p, cudaStream_t st) { return rows_launch<SR_PAGE_INT4>(p, st); }
int attn_tile_tokens_int4(int head_dim) { return attn_tile_tokens<SR_PAGE_INT4>(head_dim); }

}  // namespace sr
