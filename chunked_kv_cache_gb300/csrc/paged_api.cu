// paged_api.cu -- the C ABI of the paged token cache (declared in include/sr.h):
// argument validation and launches. The sequences' state lives on the device, so a
// call validates only what the host knows; nothing here waits for the device.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>

#include "sr.h"
#include "sr_kernels.h"
#include "sr_paged.h"

struct sr_paged_cache {
  sr_paged_config cfg;
  sr_paged_buffers buf;
  sr::PagedView view;
  sr::PagedLayout layout;
  CUtensorMap kmap, vmap;   // bf16 pages
  bool prompts;             // the kernel of blocks of rows can be launched (a cache that never needs it does without)
  int device;
  int32_t* mark;         // [max_seqs] the last call that named a row (finds repeated rows)
  int32_t stamp;
};

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

sr_status validate(const sr_paged_config& c) {
  if (c.n_heads < 1 || c.n_kv_heads < 1 || c.page_tokens < 1 || c.n_pages < 1 || c.max_seqs < 1 ||
      c.max_seqs > 65536 || c.max_pages < 1)
    return SR_ERR_INVALID_ARG;
  if (c.head_dim != 64 && c.head_dim != 128) return SR_ERR_UNSUPPORTED;
  if (c.page_type != SR_PAGE_BF16 && c.page_type != SR_PAGE_E4M3 && c.page_type != SR_PAGE_INT4) return SR_ERR_UNSUPPORTED;
  if (c.n_heads % c.n_kv_heads != 0) return SR_ERR_INVALID_ARG;
  if (c.page_tokens % 16 != 0 || c.page_tokens > 1024) return SR_ERR_UNSUPPORTED;
  if (!std::isfinite(c.softmax_scale)) return SR_ERR_INVALID_ARG;
  if (c.n_heads > 65536 / c.head_dim) return SR_ERR_INVALID_ARG;
  if (static_cast<int64_t>(c.max_pages) * c.page_tokens > (int64_t(1) << 24)) return SR_ERR_INVALID_ARG;
  if (static_cast<int64_t>(c.n_pages) * c.page_tokens > (int64_t(1) << 31)) return SR_ERR_INVALID_ARG;
  return SR_OK;
}

// Query heads that attention takes together: the largest share of a key/value head's, at most SR_MAX_PAGED_GROUP.
int attn_group(const sr_paged_config& c) {
  const int all = c.n_heads / c.n_kv_heads;
  int parts = (all + SR_MAX_PAGED_GROUP - 1) / SR_MAX_PAGED_GROUP;
  while (all % parts) ++parts;
  return all / parts;
}

sr::PagedLayout paged_layout(const sr_paged_config& c, bool with_mass) {
  sr::PagedLayout l;
  const int group = attn_group(c), n_kv = c.n_heads / group;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t here = at;
    at += (n + 255) / 256 * 256;
    return here;
  };
  l.counters = take(sr::kPagedCounters * 4);
  l.alloc = l.counters + sr::kPagedCounters * 4 - 16;   // the last four counters
  // a sequence of length n moves at most n / 2 tokens
  l.move_cap = with_mass ? static_cast<int64_t>(c.n_pages) * c.page_tokens / 2 + sr::kMaxPagedSeqs : 0;
  l.moves = take(static_cast<size_t>(l.move_cap) * sizeof(int2));
  const size_t seqs = static_cast<size_t>(c.max_seqs < sr::kMaxPagedSeqs ? c.max_seqs : sr::kMaxPagedSeqs);
  l.items = take(seqs * n_kv * sizeof(int2));
  l.unit0 = take((sr::kMaxPagedSeqs + 1) * sizeof(int64_t));
  l.parts = take(std::max(sr::kMaxPagedCtas * 2 * sr::paged_part_floats(group, c.head_dim), sr::paged_prompt_floats(c.head_dim)) * 4);
  l.lse2 = take(seqs * c.n_heads * 4);
  // every token of the pool once, the sequences' lengths rounded up to tiles
  const int64_t tile = sr::paged_tile_tokens(c.head_dim, c.page_type);
  l.score_tiles = with_mass ? sr::paged_score_tiles(static_cast<int64_t>(c.n_pages) * c.page_tokens, static_cast<int>(seqs),
                                                    n_kv, static_cast<int>(tile)) : 0;
  l.scores = take(static_cast<size_t>(l.score_tiles) * group * tile * 4);
  l.bytes = at;
  return l;
}

sr_status on_device(const sr_paged_cache* c) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return SR_ERR_CUDA;
  return dev == c->device ? SR_OK : SR_ERR_STATE;
}

// The call's rows of the block table into id[0..n).
sr_status take_seqs(sr_paged_cache* c, const int32_t* seqs, int32_t n, int32_t* id) {
  if (n < 1 || n > SR_MAX_PAGED_SEQS || n > c->cfg.max_seqs) return SR_ERR_INVALID_ARG;
  if (!seqs) {
    for (int i = 0; i < n; ++i) id[i] = i;
    return SR_OK;
  }
  if (c->stamp == INT32_MAX) {
    std::memset(c->mark, 0, sizeof(int32_t) * static_cast<size_t>(c->cfg.max_seqs));
    c->stamp = 0;
  }
  ++c->stamp;
  for (int i = 0; i < n; ++i) {
    if (seqs[i] < 0 || seqs[i] >= c->cfg.max_seqs || c->mark[seqs[i]] == c->stamp) return SR_ERR_INVALID_ARG;
    c->mark[seqs[i]] = c->stamp;
    id[i] = seqs[i];
  }
  return SR_OK;
}

template <typename T>
T* ws_at(const sr_paged_cache* c, size_t offset) {
  return reinterpret_cast<T*>(static_cast<char*>(c->buf.workspace) + offset);
}

// The rows of a call: row0[0..n] from the sequences' counts.
sr_status take_counts(const int32_t* n_tokens, int32_t n, int32_t* row0) {
  int64_t rows = 0;
  for (int i = 0; i < n; ++i) {
    const int32_t count = n_tokens ? n_tokens[i] : 1;
    if (count < 0) return SR_ERR_INVALID_ARG;
    row0[i] = static_cast<int32_t>(rows);
    rows += count;
    if (rows > (int64_t(1) << 28)) return SR_ERR_INVALID_ARG;
  }
  row0[n] = static_cast<int32_t>(rows);
  return SR_OK;
}

// The CTAs that take them: cta0[0..n].
void share_rows(const int32_t* row0, int32_t n, int32_t rows_per_cta, int32_t* cta0) {
  int64_t ctas = 0;
  for (int i = 0; i < n; ++i) {
    cta0[i] = static_cast<int32_t>(ctas);
    ctas += (static_cast<int64_t>(row0[i + 1]) - row0[i] + rows_per_cta - 1) / rows_per_cta;
  }
  cta0[n] = static_cast<int32_t>(ctas);
}

void take_heads(const sr_paged_cache* c, sr::PagedView& v, int32_t& kv_heads, uint32_t& head_magic);
// What all attention calls of a few columns per sequence hand to their launch.
void attn_params(const sr_paged_cache* c, sr::PagedAttnParams& p, int32_t n, const void* q, void* o, float* lse) {
  p.b.n = n;
  p.c = c->view;
  take_heads(c, p.c, p.kv_heads, p.head_magic);
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.items = ws_at<int2>(c, c->layout.items);
  p.unit0 = ws_at<int64_t>(c, c->layout.unit0);
  p.arrivals = ws_at<int32_t>(c, c->layout.counters) + sr::kMaxPagedSeqs;
  p.group_arrivals = p.arrivals + sr::kMaxPagedCtas;
  p.parts = ws_at<float>(c, c->layout.parts);
  p.lse2 = ws_at<float>(c, c->layout.lse2);
  p.scores = ws_at<float>(c, c->layout.scores);
  p.score_tiles = c->layout.score_tiles;
  p.part_rows = p.c.group;
}

// The view's heads as attention takes them: items of at most SR_MAX_PAGED_GROUP query heads.
void take_heads(const sr_paged_cache* c, sr::PagedView& v, int32_t& kv_heads, uint32_t& head_magic) {
  kv_heads = c->cfg.n_kv_heads;
  v.n_kv = c->cfg.n_heads / v.group;
  const uint32_t parts = static_cast<uint32_t>(v.n_kv / kv_heads);       // of a key/value head's query heads
  head_magic = ((1u << 22) + parts - 1) / parts;                         // exact for heads and parts up to 1024
}

}  // namespace

extern "C" {

sr_status sr_paged_workspace_bytes(const sr_paged_config* cfg, int32_t with_mass, uint64_t* bytes) {
  if (!cfg || !bytes) return SR_ERR_INVALID_ARG;
  const sr_status st = validate(*cfg);
  if (st != SR_OK) return st;
  *bytes = paged_layout(*cfg, with_mass != 0).bytes;
  return SR_OK;
}

sr_status sr_paged_init(const sr_paged_config* cfg, const sr_paged_buffers* bufs, void* stream, sr_paged_cache** out) {
  if (out) *out = nullptr;
  if (!cfg || !bufs || !out) return SR_ERR_INVALID_ARG;
  const sr_status st = validate(*cfg);
  if (st != SR_OK) return st;
  const sr_paged_buffers& b = *bufs;
  if (!b.k_pages || !b.v_pages || !b.block_table || !b.seq_len || !b.seq_pos || !b.token_pos || !b.err_word ||
      !b.workspace)
    return SR_ERR_INVALID_ARG;
  if (!aligned(b.k_pages, 16) || !aligned(b.v_pages, 16) || !aligned(b.block_table, 4) || !aligned(b.seq_len, 4) ||
      !aligned(b.seq_pos, 4) || !aligned(b.token_pos, 4) || !aligned(b.token_mass, 4) || !aligned(b.kv_exp, 4) ||
      !aligned(b.err_word, 4) || !aligned(b.workspace, 256))
    return SR_ERR_ALIGN;
  sr_paged_cache* c = new (std::nothrow) sr_paged_cache;
  if (!c) return SR_ERR_INVALID_ARG;
  std::memset(c, 0, sizeof(*c));
  c->mark = new (std::nothrow) int32_t[cfg->max_seqs]();
  if (!c->mark) {
    delete c;
    return SR_ERR_INVALID_ARG;
  }
  c->cfg = *cfg;
  c->buf = b;
  c->layout = paged_layout(*cfg, b.token_mass != nullptr);
  sr::PagedView& v = c->view;
  v.k_pages = b.k_pages;
  v.v_pages = b.v_pages;
  v.table = b.block_table;
  v.seq_len = b.seq_len;
  v.seq_pos = b.seq_pos;
  v.token_pos = b.token_pos;
  v.token_mass = b.token_mass;
  v.kv_exp = cfg->page_type != SR_PAGE_BF16 ? b.kv_exp : nullptr;
  v.err_word = b.err_word;
  v.n_heads = cfg->n_heads;
  v.n_kv = cfg->n_kv_heads;
  v.group = attn_group(*cfg);
  v.head_dim = cfg->head_dim;
  v.page_tokens = cfg->page_tokens;
  v.n_pages = cfg->n_pages;
  v.max_pages = cfg->max_pages;
  v.cap = cfg->max_pages * cfg->page_tokens;
  v.page_type = cfg->page_type;
  v.magic = sr::page_magic(cfg->page_tokens);
  const float scale = cfg->softmax_scale > 0.f ? cfg->softmax_scale : 1.0f / std::sqrt(static_cast<float>(cfg->head_dim));
  v.scale_log2 = scale * 1.4426950408889634f;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaGetDevice(&c->device);
  if (e == cudaSuccess) e = sr::paged_attn_prepare(cfg->head_dim, cfg->page_type);
  if (e == cudaSuccess) e = sr::paged_evict_prepare();
  if (e == cudaSuccess) c->prompts = sr::paged_prompt_prepare(cfg->head_dim, cfg->page_type) == cudaSuccess;
  if (c->prompts && cfg->page_type == SR_PAGE_BF16) {
    const int64_t rows = static_cast<int64_t>(cfg->n_pages) * cfg->page_tokens, row = static_cast<int64_t>(cfg->n_kv_heads) * cfg->head_dim;
    const int box = sr::paged_box_rows(cfg->page_tokens);
    c->prompts = sr::encode_rows(&c->kmap, b.k_pages, rows, row, box) && sr::encode_rows(&c->vmap, b.v_pages, rows, row, box);
  }
  if (e == cudaSuccess) e = sr::launch_zero_words(b.err_word, 1, cs);
  if (e == cudaSuccess) e = sr::launch_zero_words(ws_at<int32_t>(c, c->layout.counters), sr::kPagedCounters, cs);
  if (e != cudaSuccess) {
    delete[] c->mark;
    delete c;
    return SR_ERR_CUDA;
  }
  *out = c;
  return SR_OK;
}

sr_status sr_paged_free(sr_paged_cache* c) {
  if (c) {
    delete[] c->mark;
    delete c;
  }
  return SR_OK;
}

sr_status sr_paged_reset(sr_paged_cache* c, const int32_t* seqs, int32_t n, void* stream) {
  if (!c) return SR_ERR_INVALID_ARG;
  sr::PagedBatch b;
  b.n = n;
  sr_status st = take_seqs(c, seqs, n, b.id);
  if (st == SR_OK) st = on_device(c);
  if (st != SR_OK) return st;
  return sr::launch_paged_reset(c->view, b, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SR_OK : SR_ERR_CUDA;
}

sr_status sr_paged_append(sr_paged_cache* c, const int32_t* seqs, const int32_t* n_tokens, int32_t n, const void* k,
                          const void* v, void* stream) {
  if (!c) return SR_ERR_INVALID_ARG;
  sr::AppendParams p;
  sr_status st = take_seqs(c, seqs, n, p.id);
  if (st != SR_OK) return st;
  if (!aligned(k, 16) || !aligned(v, 16)) return SR_ERR_ALIGN;
  st = take_counts(n_tokens, n, p.row0);
  if (st != SR_OK) return st;
  const int32_t rows = p.row0[n];
  st = on_device(c);
  if (st != SR_OK) return st;
  if (rows == 0) return SR_OK;
  if (!k || !v) return SR_ERR_INVALID_ARG;
  p.rows_per_cta = sr::paged_append_rows_per_cta(c->view, rows, false);
  share_rows(p.row0, n, p.rows_per_cta, p.cta0);
  p.c = c->view;
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.arrivals = ws_at<int32_t>(c, c->layout.counters);
  p.n = n;
  return sr::launch_paged_append(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SR_OK : SR_ERR_CUDA;
}

sr_status sr_paged_attention(sr_paged_cache* c, const int32_t* seqs, int32_t n, const void* q, void* o, float* lse,
                             float mass_decay, void* stream) {
  if (!c || !q || !o || !std::isfinite(mass_decay)) return SR_ERR_INVALID_ARG;
  sr::PagedAttnParams p;
  sr_status st = take_seqs(c, seqs, n, p.b.id);
  if (st != SR_OK) return st;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4)) return SR_ERR_ALIGN;
  if (mass_decay >= 0.f && !c->buf.token_mass) return SR_ERR_STATE;
  st = on_device(c);
  if (st != SR_OK) return st;
  attn_params(c, p, n, q, o, lse);
  p.mass_decay = mass_decay;
  return sr::launch_paged_attention(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SR_OK : SR_ERR_CUDA;
}

sr_status sr_paged_prompt_attention(sr_paged_cache* c, const int32_t* seqs, const int32_t* n_tokens, int32_t n,
                                    const void* q, void* o, float* lse, int32_t causal, void* stream) {
  if (!c) return SR_ERR_INVALID_ARG;
  sr::PromptParams p;
  sr_status st = take_seqs(c, seqs, n, p.id);
  if (st != SR_OK) return st;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4)) return SR_ERR_ALIGN;
  st = take_counts(n_tokens, n, p.row0);
  if (st == SR_OK) st = on_device(c);
  if (st != SR_OK) return st;
  if (p.row0[n] == 0) return SR_OK;
  if (!q || !o) return SR_ERR_INVALID_ARG;
  // A few new tokens each, whose heads are columns of one product: the kernel for single tokens, which is bound by the one
  // read of the cache, where the other fills 128 rows of a tile whatever there is.
  int32_t most = 0;
  for (int i = 0; i < n; ++i) most = std::max(most, p.row0[i + 1] - p.row0[i]);
  if (static_cast<int64_t>(most) * c->view.group <= SR_MAX_PAGED_GROUP) {
    sr::PagedRowsParams r;
    attn_params(c, r, n, q, o, lse);
    std::memcpy(r.b.id, p.id, sizeof(int32_t) * static_cast<size_t>(n));
    std::memcpy(r.row0, p.row0, sizeof(int32_t) * (static_cast<size_t>(n) + 1));
    r.part_rows = most * c->view.group;
    r.causal = causal != 0;
    r.group_magic = (65536u + static_cast<uint32_t>(r.c.group) - 1u) / static_cast<uint32_t>(r.c.group);
    r.mass_decay = -1.f;
    return sr::launch_paged_rows(r, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SR_OK : SR_ERR_CUDA;
  }
  if (!c->prompts) return SR_ERR_CUDA;
  p.n = n;
  p.causal = causal != 0;
  p.arrivals = ws_at<int32_t>(c, c->layout.counters) + sr::kMaxPagedSeqs;
  p.parts = ws_at<float>(c, c->layout.parts);
  p.kmap = c->kmap;
  p.vmap = c->vmap;
  p.c = c->view;
  take_heads(c, p.c, p.kv_heads, p.head_magic);
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  if (!sr::paged_prompt_plan(p)) return SR_ERR_INVALID_ARG;
  return sr::launch_paged_prompt(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SR_OK : SR_ERR_CUDA;
}

sr_status sr_paged_read(sr_paged_cache* c, const int32_t* seqs, const int32_t* first, const int32_t* n_tokens, int32_t n,
                        void* k, void* v, void* stream) {
  if (!c) return SR_ERR_INVALID_ARG;
  sr::ReadParams p;
  sr_status st = take_seqs(c, seqs, n, p.id);
  if (st != SR_OK) return st;
  if (!aligned(k, 16) || !aligned(v, 16)) return SR_ERR_ALIGN;
  for (int i = 0; i < n; ++i) {
    p.first[i] = first ? first[i] : -1;
    if (first && first[i] < 0) return SR_ERR_INVALID_ARG;
  }
  st = take_counts(n_tokens, n, p.row0);
  if (st == SR_OK) st = on_device(c);
  if (st != SR_OK) return st;
  if (p.row0[n] == 0) return SR_OK;
  if (!k || !v) return SR_ERR_INVALID_ARG;
  p.n = n;
  p.c = c->view;
  p.rows_per_cta = sr::paged_append_rows_per_cta(c->view, p.row0[n], true);
  share_rows(p.row0, n, p.rows_per_cta, p.cta0);
  p.k = static_cast<__nv_bfloat16*>(k);
  p.v = static_cast<__nv_bfloat16*>(v);
  return sr::launch_paged_read(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SR_OK : SR_ERR_CUDA;
}

sr_status sr_paged_evict(sr_paged_cache* c, const int32_t* seqs, int32_t n, int32_t budget, int32_t n_sink,
                         int32_t n_recent, void* stream) {
  if (!c || budget < 1 || n_sink < 0 || n_recent < 0 || static_cast<int64_t>(n_sink) + n_recent > budget)
    return SR_ERR_INVALID_ARG;
  sr::EvictParams p;
  sr_status st = take_seqs(c, seqs, n, p.b.id);
  if (st != SR_OK) return st;
  if (!c->buf.token_mass) return SR_ERR_STATE;
  st = on_device(c);
  if (st != SR_OK) return st;
  if (budget >= c->view.cap) return SR_OK;   // no sequence can hold more
  p.b.n = n;
  p.c = c->view;
  p.budget = budget;
  p.n_sink = n_sink;
  p.n_recent = n_recent;
  p.alloc = ws_at<unsigned long long>(c, c->layout.alloc);
  p.moves = ws_at<int2>(c, c->layout.moves);
  p.move_cap = c->layout.move_cap;
  return sr::launch_paged_evict(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SR_OK : SR_ERR_CUDA;
}

sr_status sr_paged_locate(const sr_paged_config* cfg, const int32_t* table_row, int64_t index, int64_t* row) {
  if (!cfg || !table_row || !row) return SR_ERR_INVALID_ARG;
  const sr_status st = validate(*cfg);
  if (st != SR_OK) return st;
  *row = index < 0 || index >= static_cast<int64_t>(cfg->max_pages) * cfg->page_tokens
             ? -1
             : sr::paged_row(table_row, static_cast<int32_t>(index), cfg->page_tokens, cfg->n_pages);
  return SR_OK;
}

}  // extern "C"
