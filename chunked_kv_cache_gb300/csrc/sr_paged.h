// sr_paged.h -- parameter blocks and launchers of the paged token cache, shared
// by its host API (paged_api.cu) and kernels. Internal to libsr.so.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "sr.h"

namespace sr {

constexpr int kMaxPagedSeqs = SR_MAX_PAGED_SEQS;
constexpr int kPagedItemCost = 2;    // units of the line of tiles before an item's tiles (paged_attention.cuh)
constexpr int kMaxPromptCtas = 160;  // most CTAs a launch over several new tokens per sequence may have
constexpr int kMaxPagedCtas = 512;   // most CTAs an attention launch may have (partial result slots)

// The pool row of logical index `idx` of a sequence whose block table row is
// `table`: -1 when the entry is no page of the pool. 0 <= idx < cap.
__host__ __device__ __forceinline__ int64_t paged_row(const int32_t* table, int32_t idx, int32_t page_tokens,
                                                      int32_t n_pages) {
  const int32_t p = idx / page_tokens;
  const int32_t page = table[p];
  if (page < 0 || page >= n_pages) return -1;
  return static_cast<int64_t>(page) * page_tokens + (idx - p * page_tokens);
}

// Page of 16-token group g (0 <= g < 2^20) of a sequence: g / (page_tokens / 16) by
// multiplication with ceil(2^32 / d), exact because g * d < 2^32. magic 0: pages of one group.
__host__ __device__ __forceinline__ uint32_t page_magic(int32_t page_tokens) {
  const uint32_t d = static_cast<uint32_t>(page_tokens) / 16;
  return d == 1 ? 0u : 0xFFFFFFFFu / d + 1u;
}
__device__ __forceinline__ int32_t page_of_group(int32_t g, uint32_t magic) {
  return magic == 0 ? g : static_cast<int32_t>(__umulhi(static_cast<uint32_t>(g), magic));
}

// 4-bit pages: a record holds the codes and scales of 16 tokens of one key/value head.
__host__ __device__ constexpr int record_bytes(int head_dim) { return 9 * head_dim; }
// Byte offset of the record of head `h` that holds slot `slot` of page `page`.
__device__ __forceinline__ int64_t record_at(int32_t page, int32_t slot, int32_t h, int32_t n_kv, int32_t page_tokens,
                                             int32_t head_dim) {
  return ((static_cast<int64_t>(page) * n_kv + h) * (page_tokens >> 4) + (slot >> 4)) * record_bytes(head_dim);
}

struct PagedView {
  void* k_pages;
  void* v_pages;
  const int32_t* table;
  int32_t* seq_len;
  int32_t* seq_pos;
  int32_t* token_pos;
  float* token_mass;
  const int32_t* kv_exp;
  int32_t* err_word;
  int32_t n_heads, n_kv, group, head_dim;
  int32_t page_tokens, n_pages, max_pages;
  int32_t cap;             // max_pages * page_tokens
  int32_t page_type;
  uint32_t magic;          // page_magic(page_tokens)
  float scale_log2;        // softmax scale * log2(e)
};

// Workspace: counters, partial results, move lists, scores (see paged_layout).
struct PagedLayout {
  size_t counters;         // int32[kPagedCounters]
  size_t alloc;            // uint64[2]: entries of `moves` taken, sequences done
  size_t moves;            // int2[move_cap]: (from, to) logical indices
  int64_t move_cap;
  size_t items;            // int2[n][n_kv]
  size_t unit0;            // int64[kMaxPagedSeqs + 1]
  size_t parts;            // [kMaxPagedCtas][2] partial results
  size_t lse2;             // float[kMaxPagedSeqs][n_heads], log2 units; 0 for rows whose scores are all -inf
  size_t scores;           // float[score_tiles][group][tile tokens]
  int64_t score_tiles;
  size_t bytes;
};
// arrivals of an append's CTAs, then of an attention's parts and groups of parts, then an eviction's two 64-bit counters
constexpr int kPagedCounters = kMaxPagedSeqs + 3 * kMaxPagedCtas + 4;

struct PagedBatch {
  int32_t n;
  int32_t id[kMaxPagedSeqs];
};

constexpr int paged_box_rows(int page_tokens) { return page_tokens % 32 == 0 ? 32 : 16; }

struct AppendParams {
  PagedView c;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  int32_t* arrivals;               // [n] CTAs of each sequence that are done; left at zero
  int32_t n;
  int32_t rows_per_cta;
  int32_t id[kMaxPagedSeqs];
  int32_t row0[kMaxPagedSeqs + 1]; // first row of each sequence
  int32_t cta0[kMaxPagedSeqs + 1]; // first CTA of each sequence
};

struct PagedAttnParams {
  PagedView c;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;
  int2* items;             // [n][n_kv] first part and number of parts, when a launch of its own joins them; else NULL
  int64_t* unit0;          // [n + 1] first unit of each sequence on the line (see paged_attention.cuh), and its end
  int32_t* arrivals;       // [kMaxPagedCtas] parts, or groups of parts, of an item that are done; left at zero
  int32_t* group_arrivals; // [2 * kMaxPagedCtas]
  float* parts;
  int32_t part_rows;       // rows that a partial result has room for
  float* lse2;
  float* scores;
  int64_t score_tiles;
  int32_t spread;          // neighbouring key/value heads that neighbouring CTAs take side by side; divides n_kv
  int32_t spread_log2;
  // Key/value heads in memory. Where more query heads than SR_MAX_PAGED_GROUP share one, c.n_kv and c.group are those of
  // equal subgroups, each an item of its own: item head h reads head h * head_magic >> 22.
  int32_t kv_heads;
  uint32_t head_magic;
  // Stretches that end where items end (the rule stands at Geo::kWhole); all in 16ths of a unit, times the stretches
  int32_t each;            // whole items for each CTA, or
  int32_t pieces;          // pieces that an item is cut into (below 2: none)
  int64_t whole_cost;      // 16 * each * stretches
  int64_t cut_cost;        // 16 * stretches / pieces
  int64_t whole_extra;     // 16 * stretches * kWholeExtra, or kAloneExtra
  bool drop_scores;        // the weights' launch drops the scores from L2
  float mass_decay;
  PagedBatch b;
};

// Attention of a few new tokens per sequence, whose heads fit the columns of one product.
struct PagedRowsParams : PagedAttnParams {
  int32_t causal;
  uint32_t group_magic;            // r / group = r * group_magic >> 16 for r < 128
  int32_t row0[kMaxPagedSeqs + 1]; // first row of each sequence
};

struct ReadParams {
  PagedView c;
  __nv_bfloat16* k;
  __nv_bfloat16* v;
  int32_t n;
  int32_t rows_per_cta;
  int32_t id[kMaxPagedSeqs];
  int32_t first[kMaxPagedSeqs];    // first index of each sequence; negative: its last rows
  int32_t row0[kMaxPagedSeqs + 1];
  int32_t cta0[kMaxPagedSeqs + 1];
};

struct alignas(64) PromptParams {
  CUtensorMap kmap, vmap;  // bf16 pages: [n_pages * page_tokens][n_kv_heads * head_dim], boxes of 64 values of paged_box_rows() tokens
  PagedView c;             // n_kv, group: items of at most SR_MAX_PAGED_GROUP query heads, as in PagedAttnParams
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;
  int32_t kv_heads;
  uint32_t head_magic;
  int32_t* arrivals;       // [kMaxPromptCtas] parts of a block that are done; left at zero
  float* parts;            // [kMaxPromptCtas][2] partial results
  int32_t n;
  int32_t causal;
  int32_t id[kMaxPagedSeqs];
  int32_t row0[kMaxPagedSeqs + 1]; // first row of each sequence
  // set by paged_prompt_plan
  int32_t tpt;             // tokens of a tile of 128 query rows
  uint32_t group_magic;    // r / group = r * group_magic >> 16 for r < 128
  int32_t blocks;          // of query rows, over all sequences
  bool o_aligned;          // o begins on a multiple of 32 bytes
  int32_t blk0[kMaxPagedSeqs];     // first block of each sequence
};

struct EvictParams {
  PagedView c;
  int32_t budget, n_sink, n_recent;
  unsigned long long* alloc;
  int2* moves;
  int64_t move_cap;
  PagedBatch b;
};

cudaError_t launch_paged_reset(const PagedView& c, const PagedBatch& b, cudaStream_t st);
cudaError_t launch_paged_append(const AppendParams& p, cudaStream_t st);
cudaError_t launch_paged_rows(const PagedRowsParams& p, cudaStream_t st);
cudaError_t launch_paged_read(const ReadParams& p, cudaStream_t st);
cudaError_t launch_paged_prompt(const PromptParams& p, cudaStream_t st);
cudaError_t paged_prompt_prepare(int head_dim, int page_type);
bool paged_prompt_plan(PromptParams& p);                              // blocks of query rows; false: more work than a launch takes
size_t paged_prompt_floats(int head_dim);                            // floats of all partial results of a prompt's launch
cudaError_t launch_paged_attention(const PagedAttnParams& p, cudaStream_t st);
cudaError_t launch_paged_evict(const EvictParams& p, cudaStream_t st);
int paged_tile_tokens(int head_dim, int page_type);       // tokens of a tile
cudaError_t paged_evict_prepare();
cudaError_t paged_attn_prepare(int head_dim, int page_type);
int64_t paged_score_tiles(int64_t pool_tokens, int n_seqs, int n_kv, int tile_tokens);   // tiles that scores are kept for
size_t paged_part_floats(int group, int head_dim);                   // floats of one partial result
int paged_append_rows_per_cta(const PagedView& c, int64_t rows, bool read);

}  // namespace sr
