// paged_cache.cu -- the paged token cache's state: appending tokens to pages and
// evicting them by accumulated attention weight.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "sr_device.cuh"
#include "sr_kernels.h"
#include "sr_paged.h"

namespace sr {

namespace {

__device__ __forceinline__ void note_error(const PagedView& c, int code) { atomicCAS(c.err_word, 0, code); }

// ------------------------------------------------------------------ reset
__global__ void __launch_bounds__(256) paged_reset_kernel(const PagedView c, const PagedBatch b) {
  grid_dep_wait();
  const int i = threadIdx.x;
  if (i < b.n) {
    c.seq_len[b.id[i]] = 0;
    c.seq_pos[b.id[i]] = 0;
  }
}

// ------------------------------------------------------------------ append
// A copy with a scatter of whole rows: HBM bound, reads the new rows once and
// writes them once. A CTA takes up to rows_per_cta rows of one sequence, every
// thread 16-byte vectors (8 bf16) of the keys and of the values. Each CTA first
// checks that all of the sequence's new tokens fit, so that a sequence is taken
// whole or not at all without a pass of its own; the last of a sequence's CTAs to
// finish raises its length (every CTA has read the old one by then).
constexpr int kAppendThreads = 256;

__device__ __forceinline__ uint2 to_e4m3(const uint4& x, float inv_scale) {
  const uint32_t in[4] = {x.x, x.y, x.z, x.w};
  uint16_t out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&in[i]));
    out[i] = __nv_cvt_float2_to_fp8x2(make_float2(f.x * inv_scale, f.y * inv_scale), __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(out[0] | (uint32_t(out[1]) << 16), out[2] | (uint32_t(out[3]) << 16));
}

template <int TYPE>
__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(const __grid_constant__ AppendParams p) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  const PagedView& c = p.c;
  __shared__ int bad;
  if (threadIdx.x == 0) bad = 0;
  // the CTA's sequence: the last i with cta0[i] <= blockIdx.x and rows of its own
  int lo = 0, hi = p.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (p.cta0[mid] <= static_cast<int>(blockIdx.x)) lo = mid; else hi = mid - 1;
  }
  const int i = lo;
  const int32_t seq = p.id[i];
  const int32_t count = p.row0[i + 1] - p.row0[i];
  const int32_t len = c.seq_len[seq], pos = c.seq_pos[seq];
  const int32_t* table = c.table + static_cast<int64_t>(seq) * c.max_pages;
  __syncthreads();
  if (len < 0 || pos < 0 || len > c.cap - count || pos > INT32_MAX - count) {
    if (threadIdx.x == 0) {
      bad = 1;
      note_error(c, SR_DEVERR_CACHE_FULL);
    }
  } else {
    const int32_t first = len / c.page_tokens, last = (len + count - 1) / c.page_tokens;
    for (int32_t g = first + static_cast<int32_t>(threadIdx.x); g <= last; g += kAppendThreads)
      if (table[g] < 0 || table[g] >= c.n_pages) {
        bad = 1;
        note_error(c, SR_DEVERR_BAD_PAGE);
      }
  }
  __syncthreads();
  if (!bad) {
    const int32_t r0 = (static_cast<int32_t>(blockIdx.x) - p.cta0[i]) * p.rows_per_cta;
    const int32_t rows = min(p.rows_per_cta, count - r0);
    const int vph = c.head_dim / 8;             // vectors per head
    const int vpr = c.n_kv * vph;               // vectors per row
    const uint4* ksrc = reinterpret_cast<const uint4*>(p.k) + static_cast<int64_t>(p.row0[i] + r0) * vpr;
    const uint4* vsrc = reinterpret_cast<const uint4*>(p.v) + static_cast<int64_t>(p.row0[i] + r0) * vpr;
    for (int x = threadIdx.x; x < rows * vpr; x += kAppendThreads) {
      const int r = x / vpr, col = x - r * vpr;
      const uint4 kx = ksrc[x], vx = vsrc[x];
      const int64_t at = paged_row(table, len + r0 + r, c.page_tokens, c.n_pages) * vpr + col;
      if constexpr (TYPE == SR_PAGE_BF16) {
        static_cast<uint4*>(c.k_pages)[at] = kx;
        static_cast<uint4*>(c.v_pages)[at] = vx;
      } else {
        const int head = col / vph;
        const float ki = c.kv_exp ? exp2f(-static_cast<float>(c.kv_exp[head])) : 1.f;
        const float vi = c.kv_exp ? exp2f(-static_cast<float>(c.kv_exp[c.n_kv + head])) : 1.f;
        static_cast<uint2*>(c.k_pages)[at] = to_e4m3(kx, ki);
        static_cast<uint2*>(c.v_pages)[at] = to_e4m3(vx, vi);
      }
    }
    const int64_t t0 = static_cast<int64_t>(seq) * c.cap + len + r0;
    for (int r = threadIdx.x; r < rows; r += kAppendThreads) {
      c.token_pos[t0 + r] = pos + r0 + r;
      if (c.token_mass) c.token_mass[t0 + r] = 0.f;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    const int32_t ctas = p.cta0[i + 1] - p.cta0[i];
    bool last = true;
    if (ctas > 1) {
      __threadfence();
      last = atomicAdd(p.arrivals + i, 1) == ctas - 1;
      if (last) p.arrivals[i] = 0;
    }
    if (last && !bad) {
      c.seq_len[seq] = len + count;
      c.seq_pos[seq] = pos + count;
    }
  }
}

// ------------------------------------------------------------------ evict
// Two launches. The first picks, one CTA per sequence: a radix select over the
// weights' bits finds the weight below which tokens go, then three ordered passes
// (ties, counts, lists) write the moves. The second moves the rows.
constexpr int kPickThreads = 1024;
constexpr int kPickWarps = kPickThreads / 32;

// The order of the weights as unsigned integers; protected tokens come last.
__device__ __forceinline__ uint32_t weight_key(float m) {
  if (m != m) return 0xFFFFFFFEu;
  const uint32_t b = __float_as_uint(m + 0.f);   // -0 counts as 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ uint32_t warp_incl_scan(uint32_t x, int lane) {
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, s);
    if (lane >= s) x += y;
  }
  return x;
}

__global__ void __launch_bounds__(kPickThreads) paged_pick_kernel(const __grid_constant__ EvictParams p) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  const PagedView& c = p.c;
  __shared__ uint32_t hist[256];
  __shared__ uint32_t sums[3][kPickWarps];
  __shared__ uint32_t pick[2];          // digit found, rank left
  __shared__ uint32_t n_free;
  __shared__ int64_t list0;
  const int i = blockIdx.x, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int32_t seq = p.b.id[i];
  const int32_t len = min(max(c.seq_len[seq], 0), c.cap);
  const int32_t pos_next = c.seq_pos[seq];
  if (len <= p.budget) {
    if (tid == 0) p.plan[i] = EvictPlan{0, 0, -1};
    return;
  }
  const int32_t* tpos = c.token_pos + static_cast<int64_t>(seq) * c.cap;
  const float* mass = c.token_mass + static_cast<int64_t>(seq) * c.cap;
  const int32_t recent0 = pos_next - p.n_recent;   // both >= 0
  auto key = [&](int32_t t) -> uint32_t {
    const int32_t q = tpos[t];
    return q < p.n_sink || q >= recent0 ? 0xFFFFFFFFu : weight_key(mass[t]);
  };
  // where this sequence's moves go: behind those of the sequences before it
  if (warp == 0) {
    int64_t s = 0;
    for (int j = lane; j < i; j += 32) s += min(max(c.seq_len[p.b.id[j]], 0), c.cap) / 2;
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    if (lane == 0) {
      list0 = s;
      n_free = 0;
    }
  }
  __syncthreads();
  uint32_t mine = 0;
  for (int32_t t = tid; t < len; t += kPickThreads) mine += key(t) != 0xFFFFFFFFu;
  mine = __reduce_add_sync(0xffffffffu, mine);
  if (lane == 0) atomicAdd(&n_free, mine);
  __syncthreads();
  uint32_t gone = min(static_cast<uint32_t>(len - p.budget), n_free);
  if (gone > 0 && list0 + len / 2 > p.move_cap) {
    if (tid == 0) note_error(c, SR_DEVERR_WORKSPACE);
    gone = 0;
  }
  if (gone == 0) {
    if (tid == 0) p.plan[i] = EvictPlan{0, 0, -1};
    return;
  }
  const int32_t kept = len - static_cast<int32_t>(gone);   // the new length
  // the key of rank `gone` (from 1): eight bits at a time
  uint32_t prefix = 0, rank = gone;
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    const uint32_t mask = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
    for (int32_t t = tid; t < len; t += kPickThreads) {
      const uint32_t k = key(t);
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1u);
    }
    __syncthreads();
    if (warp == 0) {
      uint32_t h[8], s = 0;
      for (int j = 0; j < 8; ++j) {
        h[j] = hist[lane * 8 + j];
        s += h[j];
      }
      uint32_t before = warp_incl_scan(s, lane) - s;
      for (int j = 0; j < 8; ++j) {
        if (before < rank && rank <= before + h[j]) {
          pick[0] = lane * 8 + j;
          pick[1] = rank - before;
        }
        before += h[j];
      }
    }
    __syncthreads();
    prefix |= pick[0] << shift;
    rank = pick[1];
    __syncthreads();
  }
  // every key below `prefix` goes, and of those equal to it the last `rank` by index
  const int32_t chunk = (len + kPickThreads - 1) / kPickThreads * 32;   // a warp's stretch of indices
  const int32_t t0 = warp * chunk, t1 = min(t0 + chunk, len);
  auto block_scan = [&](uint32_t x, uint32_t* buf, uint32_t& total) -> uint32_t {   // x: a per-warp count
    if (lane == 0) buf[warp] = x;
    __syncthreads();
    const uint32_t v = buf[lane];
    const uint32_t incl = warp_incl_scan(v, lane);
    total = __shfl_sync(0xffffffffu, incl, 31);
    return __shfl_sync(0xffffffffu, incl - v, warp);
  };
  uint32_t ties = 0;
  for (int32_t b = t0; b < t1; b += 32)
    ties += __popc(__ballot_sync(0xffffffffu, b + lane < t1 && key(b + lane) == prefix));
  uint32_t n_ties;
  const uint32_t tie0 = block_scan(ties, sums[0], n_ties);
  const uint32_t tie_keep = n_ties - rank;   // ties that stay: the first ones
  auto walk = [&](auto&& f) {
    uint32_t tie = tie0;
    for (int32_t b = t0; b < t1; b += 32) {
      const int32_t t = b + lane;
      const uint32_t k = t < t1 ? key(t) : 0xFFFFFFFFu;
      const uint32_t eq = __ballot_sync(0xffffffffu, t < t1 && k == prefix);
      const uint32_t below = __popc(eq & ((1u << lane) - 1u));
      const bool go = t < t1 && (k < prefix || (k == prefix && tie + below >= tie_keep));
      tie += __popc(eq);
      const uint32_t holes = __ballot_sync(0xffffffffu, go && t < kept);
      const uint32_t backs = __ballot_sync(0xffffffffu, t < t1 && !go && t >= kept);
      f(t, holes, backs);
    }
  };
  uint32_t nh = 0, nb = 0, n_holes, n_backs;
  walk([&](int32_t, uint32_t holes, uint32_t backs) {
    nh += __popc(holes);
    nb += __popc(backs);
  });
  uint32_t h0 = block_scan(nh, sums[1], n_holes), b0 = block_scan(nb, sums[2], n_backs);
  int2* list = p.moves + list0;
  walk([&](int32_t t, uint32_t holes, uint32_t backs) {
    const uint32_t lt = (1u << lane) - 1u;
    if (holes >> lane & 1u) list[h0 + __popc(holes & lt)].y = t;
    if (backs >> lane & 1u) list[b0 + __popc(backs & lt)].x = t;
    h0 += __popc(holes);
    b0 += __popc(backs);
  });
  // the second launch lowers the length: by then every CTA of this one has read the lengths
  if (tid == 0) p.plan[i] = EvictPlan{list0, static_cast<int32_t>(n_holes), kept};
}

// The second launch: `per` CTAs per sequence, a warp per moved token. A move reads
// at or behind the new length and writes below it, so that no move sees another.
constexpr int kMoveThreads = 256;
__global__ void __launch_bounds__(kMoveThreads) paged_move_kernel(const __grid_constant__ EvictParams p, int per) {
  grid_dep_wait();
  grid_dep_launch_dependents();
  const PagedView& c = p.c;
  const int i = blockIdx.x / per, part = blockIdx.x % per;
  const EvictPlan plan = p.plan[i];
  if (plan.new_len < 0) return;
  const int32_t seq = p.b.id[i];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int32_t* table = c.table + static_cast<int64_t>(seq) * c.max_pages;
  const int64_t t0 = static_cast<int64_t>(seq) * c.cap;
  const int vpr = c.n_kv * c.head_dim * (c.page_type == SR_PAGE_BF16 ? 2 : 1) / 16;
  for (int32_t j = part * (kMoveThreads / 32) + warp; j < plan.moves; j += per * (kMoveThreads / 32)) {
    const int2 m = p.moves[plan.list0 + j];
    const int64_t from = paged_row(table, m.x, c.page_tokens, c.n_pages);
    const int64_t to = paged_row(table, m.y, c.page_tokens, c.n_pages);
    if (from < 0 || to < 0) {
      if (lane == 0) note_error(c, SR_DEVERR_BAD_PAGE);
      continue;
    }
    for (int x = lane; x < 2 * vpr; x += 32) {
      uint4* pages = static_cast<uint4*>(x < vpr ? c.k_pages : c.v_pages);
      const int col = x < vpr ? x : x - vpr;
      pages[to * vpr + col] = pages[from * vpr + col];
    }
    if (lane == 0) {
      c.token_pos[t0 + m.y] = c.token_pos[t0 + m.x];
      c.token_mass[t0 + m.y] = c.token_mass[t0 + m.x];
    }
  }
  if (part == 0 && threadIdx.x == 0) c.seq_len[seq] = plan.new_len;
}

}  // namespace

int paged_append_rows_per_cta(int n_kv, int head_dim) {
  return std::max(1, 2048 * 8 / (n_kv * head_dim));
}

cudaError_t launch_paged_reset(const PagedView& c, const PagedBatch& b, cudaStream_t st) {
  return launch_dependent(paged_reset_kernel, 1, 256, 0, st, c, b);
}

cudaError_t launch_paged_append(const AppendParams& p, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>(p.cta0[p.n]);
  if (p.c.page_type == SR_PAGE_BF16) return launch_dependent(paged_append_kernel<SR_PAGE_BF16>, grid, kAppendThreads, 0, st, p);
  return launch_dependent(paged_append_kernel<SR_PAGE_E4M3>, grid, kAppendThreads, 0, st, p);
}

cudaError_t launch_paged_evict(const EvictParams& p, cudaStream_t st) {
  cudaError_t e = launch_dependent(paged_pick_kernel, p.b.n, kPickThreads, 0, st, p);
  if (e != cudaSuccess) return e;
  const int per = std::max(1, 2 * sm_count() / p.b.n);
  return launch_dependent(paged_move_kernel, static_cast<unsigned>(p.b.n) * per, kMoveThreads, 0, st, p, per);
}

}  // namespace sr
