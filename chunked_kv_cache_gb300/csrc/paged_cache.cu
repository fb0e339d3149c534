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
// One launch. The weights' bits, mapped to unsigned integers in the weights' order,
// are read once into shared memory. A radix select over 11, 11 and 10 bits finds the
// key at and below which tokens go; ordered counts turn the choice into moves (from,
// to); then all warps move rows, a warp per token. A move reads at or behind the new
// length and writes below it, so that no move sees another. Latency bound until the
// moves, which are HBM bound.
//
// Two kernels. paged_evict_kernel: every CTA of a sequence's cluster holds all keys and
// makes the whole choice for itself, so that they meet at one barrier only, before the
// first move. paged_evict_long_kernel: for sequences whose keys one CTA cannot hold;
// each CTA holds a stretch and the counts are added through distributed shared memory.
constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kKeyLimit = 40960;      // keys a CTA can hold; longer stretches are read again from global memory

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

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// the address of another CTA's copy of a shared variable, and loads from it
__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ uint32_t peer_load(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint4 peer_load4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}


// A warp moves one token: its rows, position and weight.
__device__ __forceinline__ void move_token(const PagedView& c, const int32_t* table, int32_t* tpos, float* mass, int2 m,
                                           int vpr, int lane) {
  const int64_t from = paged_row(table, m.x, c.page_tokens, c.n_pages);
  const int64_t to = paged_row(table, m.y, c.page_tokens, c.n_pages);
  if (from < 0 || to < 0) {
    if (lane == 0) note_error(c, SR_DEVERR_BAD_PAGE);
    return;
  }
  if (lane == 0) {
    tpos[m.y] = tpos[m.x];
    mass[m.y] = mass[m.x];
  }
  const uint4* ks = static_cast<const uint4*>(c.k_pages) + from * vpr;
  const uint4* vs = static_cast<const uint4*>(c.v_pages) + from * vpr;
  uint4* kd = static_cast<uint4*>(c.k_pages) + to * vpr;
  uint4* vd = static_cast<uint4*>(c.v_pages) + to * vpr;
  for (int x0 = lane; x0 < vpr; x0 += 128) {      // eight loads in flight per lane
    uint4 a[4], b[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (x0 + 32 * k < vpr) {
        a[k] = __ldcs(ks + x0 + 32 * k);
        b[k] = __ldcs(vs + x0 + 32 * k);
      }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (x0 + 32 * k < vpr) {
        kd[x0 + 32 * k] = a[k];
        vd[x0 + 32 * k] = b[k];
      }
  }
}

// Scans over a block of WARPS warps of a per-warp count: those before this warp, and all.
template <int WARPS>
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t* buf, int warp, int lane, uint32_t& total) {
  if (lane == 0) buf[warp] = x;
  __syncthreads();
  const uint32_t v = lane < WARPS ? buf[lane] : 0;
  const uint32_t incl = warp_incl_scan(v, lane);
  total = __shfl_sync(0xffffffffu, incl, 31);
  return __shfl_sync(0xffffffffu, incl - v, warp);
}

constexpr int kPickThreads = 1024;
constexpr int kPickWarps = kPickThreads / 32;
constexpr int kPickLimit = 40960;     // keys a CTA holds

__global__ void __launch_bounds__(kPickThreads, 1) paged_evict_kernel(const __grid_constant__ EvictParams p, int key_cap) {
  extern __shared__ __align__(16) uint32_t keys[];   // [key_cap], then this CTA's moves
  __shared__ uint32_t hist[3][kBins];
  __shared__ uint32_t sums[4][kPickWarps];
  __shared__ uint32_t found[3][3];                   // per pass: digit, rank in it, its keys
  const uint32_t C = cluster_size(), me = cluster_rank();
  const int i = blockIdx.x / C, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  int2* list = reinterpret_cast<int2*>(keys + key_cap);
  for (int x = tid; x < 3 * kBins; x += kPickThreads) (&hist[0][0])[x] = 0;
  grid_dep_launch_dependents();
  grid_dep_wait();
  const PagedView& c = p.c;
  const int32_t seq = p.b.id[i];
  const int32_t len = min(max(c.seq_len[seq], 0), c.cap);
  const int64_t recent0 = static_cast<int64_t>(c.seq_pos[seq]) - p.n_recent;
  if (len <= p.budget) return;                       // as in every CTA of the cluster
  int32_t* tpos = c.token_pos + static_cast<int64_t>(seq) * c.cap;
  float* mass = c.token_mass + static_cast<int64_t>(seq) * c.cap;
#pragma unroll 4
  for (int32_t t = tid; t < len; t += kPickThreads) {
    const int32_t q = tpos[t];
    const float m = mass[t];
    keys[t] = q < p.n_sink || q >= recent0 ? 0xFFFFFFFFu : weight_key(m);
  }
  __syncthreads();
  // a warp's stretch of indices, a multiple of 32
  const int32_t seg = (len + kPickThreads - 1) / kPickThreads * 32;
  const int32_t w0 = min(warp * seg, len), w1 = min(w0 + seg, len);

  // ---- the key of rank `gone` (from 1) among those that may go
  uint32_t limit = 0, rank = 0, ties = 0;            // keys below `limit` go; of those equal to it the last `rank`
  int32_t gone = 0;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, above = pass == 1 ? 21 : 10;
    const uint32_t digits = pass == 2 ? 1023 : 2047;
#pragma unroll 4
    for (int32_t x0 = w0; x0 < w1; x0 += 32) {
      const uint32_t k = x0 + lane < w1 ? keys[x0 + lane] : 0xFFFFFFFFu;
      const bool in = k != 0xFFFFFFFFu && (pass == 0 || k >> above == limit >> above);
      const uint32_t digit = k >> shift & digits;
      // equal weights would queue on one counter: the warp adds them at once
      const uint32_t act = __ballot_sync(0xffffffffu, in);
      const uint32_t d0 = __shfl_sync(0xffffffffu, digit, __ffs(act) - 1 & 31);
      if (__all_sync(0xffffffffu, !in || digit == d0)) {
        if (lane == 0 && act) atomicAdd(&hist[pass][d0], __popc(act));
      } else if (in) {
        atomicAdd(&hist[pass][digit], 1u);
      }
    }
    __syncthreads();
    const uint2 h = reinterpret_cast<const uint2*>(hist[pass])[tid];   // two digits per thread
    const uint32_t incl = warp_incl_scan(h.x + h.y, lane);
    const uint32_t warp_all = __shfl_sync(0xffffffffu, incl, 31);
    uint32_t total;
    uint32_t before = block_scan<kPickWarps>(warp_all, sums[pass], warp, lane, total) + incl - h.x - h.y;
    if (pass == 0) {
      gone = static_cast<int32_t>(min(static_cast<uint32_t>(len - p.budget), total));
      rank = static_cast<uint32_t>(gone);
    }
    if (before < rank && rank <= before + h.x + h.y) {
      const bool second = rank > before + h.x;
      found[pass][0] = tid * 2 + second;
      found[pass][1] = rank - before - (second ? h.x : 0);
      found[pass][2] = second ? h.y : h.x;
    }
    __syncthreads();
    if (gone == 0) return;                           // every token is protected; as in every CTA of the cluster
    limit |= found[pass][0] << shift;
    rank = found[pass][1];
    ties = found[pass][2];
    if (rank == ties) {                              // all keys of this digit go: no need to look further
      limit = min(limit | ((1u << shift) - 1u), 0xFFFFFFFEu);   // never the protected ones
      break;
    }
  }
  const int32_t kept = len - gone;                   // the new length

  // ---- the moves: the j-th index below `kept` that goes, the j-th at or behind it that stays
  uint32_t tie0 = 0, unused;
  const bool split = rank != ties;                   // some of the keys equal to `limit` stay: the first ones
  if (split) {
    uint32_t eq = 0;
    for (int32_t x0 = w0; x0 < w1; x0 += 32)
      eq += __popc(__ballot_sync(0xffffffffu, x0 + lane < w1 && keys[x0 + lane] == limit));
    tie0 = block_scan<kPickWarps>(eq, sums[3], warp, lane, unused);
    __syncthreads();
  }
  const uint32_t tie_keep = ties - rank, lt = (1u << lane) - 1u;
  auto walk = [&](auto&& f) {
    uint32_t tie = tie0;
#pragma unroll 4
    for (int32_t x0 = w0; x0 < w1; x0 += 32) {
      const int32_t t = x0 + lane;
      const uint32_t k = t < w1 ? keys[t] : 0xFFFFFFFFu;
      bool go = k <= limit;                          // never a protected one, nor one past the stretch
      if (split) {
        const uint32_t eq = __ballot_sync(0xffffffffu, k == limit);
        if (k == limit && tie + __popc(eq & lt) < tie_keep) go = false;
        tie += __popc(eq);
      }
      f(t, __ballot_sync(0xffffffffu, go && t < kept), __ballot_sync(0xffffffffu, t < w1 && !go && t >= kept));
    }
  };
  uint32_t nh = 0, nb = 0, moves, n_backs;
  walk([&](int32_t, uint32_t holes, uint32_t backs) {
    nh += __popc(holes);
    nb += __popc(backs);
  });
  // a count of each kind fits 16 bits: kPickLimit keys
  const uint32_t both = block_scan<kPickWarps>(nh | nb << 16, sums[3], warp, lane, moves);
  uint32_t h0 = both & 0xFFFFu, b0 = both >> 16;
  n_backs = moves >> 16;
  moves &= 0xFFFFu;
  walk([&](int32_t t, uint32_t holes, uint32_t backs) {
    const uint32_t h = h0 + __popc(holes & lt), b = b0 + __popc(backs & lt);
    if ((holes >> lane & 1u) && h % C == me) list[h / C].y = t;
    if ((backs >> lane & 1u) && b % C == me) list[b / C].x = t;
    h0 += __popc(holes);
    b0 += __popc(backs);
  });
  __syncthreads();
  if (C > 1) cluster_sync();   // every CTA has read the weights and positions: they may change
  if (me == 0 && tid == 0) c.seq_len[seq] = kept;
  const int32_t* table = c.table + static_cast<int64_t>(seq) * c.max_pages;
  const int vpr = c.n_kv * c.head_dim * (c.page_type == SR_PAGE_BF16 ? 2 : 1) / 16;
  for (uint32_t j = warp; j * C + me < moves; j += kPickWarps) move_token(c, table, tpos, mass, list[j], vpr, lane);
}

__global__ void __launch_bounds__(kEvictThreads, 1) paged_evict_long_kernel(const __grid_constant__ EvictParams p, int key_cap) {
  extern __shared__ uint32_t keys[];              // [key_cap]
  __shared__ __align__(16) uint32_t hist[2][kBins];
  __shared__ uint32_t sums[kEvictWarps];
  __shared__ uint32_t found[3];                   // digit, rank left, keys counted
  __shared__ uint32_t pub[4];                     // what the other CTAs read: ties, holes, kept tokens behind; first move (low half)
  __shared__ uint32_t pub_hi;
  const uint32_t C = cluster_size(), rank_c = cluster_rank();
  const int i = blockIdx.x / C, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  for (int x = tid; x < 2 * kBins; x += kEvictThreads) (&hist[0][0])[x] = 0;
  grid_dep_launch_dependents();
  grid_dep_wait();
  const PagedView& c = p.c;
  const int32_t seq = p.b.id[i];
  const int32_t len = min(max(c.seq_len[seq], 0), c.cap);
  // the last sequence to be done clears the list's counters for the next call
  auto done = [&] {
    if (rank_c == 0 && tid == 0 && atomicAdd(p.alloc + 1, 1ull) == static_cast<unsigned long long>(p.b.n) - 1) {
      p.alloc[0] = 0;
      p.alloc[1] = 0;
    }
  };
  if (len <= p.budget) {
    done();
    return;
  }
  int32_t* tpos = c.token_pos + static_cast<int64_t>(seq) * c.cap;
  float* mass = c.token_mass + static_cast<int64_t>(seq) * c.cap;
  const int64_t recent0 = static_cast<int64_t>(c.seq_pos[seq]) - p.n_recent;
  auto key_of = [&](int32_t q, float m) { return q < p.n_sink || q >= recent0 ? 0xFFFFFFFFu : weight_key(m); };
  // this CTA's stretch of indices: a multiple of 32 for each of its warps
  const int32_t chunk = static_cast<int32_t>((len + C * kEvictThreads - 1) / (C * kEvictThreads)) * kEvictThreads;
  const int32_t first = min(static_cast<int32_t>(rank_c) * chunk, len), count = min(chunk, len - first);
  const bool held = chunk <= key_cap;
  if (held) {
#pragma unroll 4
    for (int32_t x = tid; x < count; x += kEvictThreads) keys[x] = key_of(tpos[first + x], mass[first + x]);
  }
  __syncthreads();
  auto key = [&](int32_t x) { return held ? keys[x] : key_of(tpos[first + x], mass[first + x]); };

  // ---- the key of rank `gone` (from 1) among those that may go
  uint32_t prefix = 0, rank = 0;
  int32_t gone = 0;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t bins = pass == 2 ? 1024 : 2048;
    uint32_t* h = hist[pass & 1];
    for (int32_t x0 = warp * 32; x0 < count; x0 += kEvictThreads) {
      const int32_t x = x0 + lane;
      const uint32_t k = x < count ? key(x) : 0xFFFFFFFFu;
      const bool in = k != 0xFFFFFFFFu && (pass == 0 || k >> (pass == 1 ? 21 : 10) == prefix >> (pass == 1 ? 21 : 10));
      const uint32_t digit = (k >> shift) & (bins - 1);
      const uint32_t act = __ballot_sync(0xffffffffu, in);
      if (act == 0) continue;
      // equal weights would queue on one counter: the warp adds them at once
      const uint32_t d0 = __shfl_sync(0xffffffffu, digit, __ffs(act) - 1);
      if (__all_sync(0xffffffffu, !in || digit == d0)) {
        if (lane == 0) atomicAdd(&h[d0], __popc(act));
      } else if (in) {
        atomicAdd(&h[digit], 1u);
      }
    }
    __syncthreads();
    if (C > 1) cluster_sync();
    // every CTA adds all counts, four digits per thread, and finds the same digit
    uint4 s = make_uint4(0, 0, 0, 0);
    if (tid * 4 < static_cast<int>(bins)) {
      if (C == 1) {
        s = *reinterpret_cast<const uint4*>(h + tid * 4);
      } else {
#pragma unroll
        for (uint32_t r = 0; r < kMaxCluster; ++r)
          if (r < C) {
            const uint4 v = peer_load4(peer_addr(h + tid * 4, r));
            s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
          }
      }
    }
    const uint32_t mine = s.x + s.y + s.z + s.w;
    const uint32_t incl = warp_incl_scan(mine, lane);
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    const uint32_t ws = lane < kEvictWarps ? sums[lane] : 0;
    const uint32_t wi = warp_incl_scan(ws, lane);
    uint32_t before = incl - mine + __shfl_sync(0xffffffffu, wi - ws, warp);
    if (pass == 0) {
      const uint32_t total = __shfl_sync(0xffffffffu, wi, 31);   // tokens that may go
      gone = static_cast<int32_t>(min(static_cast<uint32_t>(len - p.budget), total));
      rank = static_cast<uint32_t>(gone);
    }
    const uint32_t v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (before < rank && rank <= before + v[j]) {
        found[0] = tid * 4 + j;
        found[1] = rank - before;
      }
      before += v[j];
    }
    __syncthreads();
    if (gone == 0) break;
    prefix |= found[0] << shift;
    rank = found[1];
    // the other buffer was read before this pass's barrier: clear it for the pass after the next
    uint32_t* other = hist[(pass + 1) & 1];
    if (pass == 1)
      for (int x = tid; x < kBins; x += kEvictThreads) other[x] = 0;
    __syncthreads();
  }
  if (gone == 0) {            // every token is protected; as in all CTAs of the cluster
    if (C > 1) cluster_sync();   // the others may still be reading this CTA's counts
    done();
    return;
  }
  const int32_t kept = len - gone;   // the new length

  // ---- every key below `prefix` goes, and of those equal to it the last `rank` by index
  const int32_t w0 = min(warp * (chunk / kEvictWarps), count), w1 = min(w0 + chunk / kEvictWarps, count);
  auto scan = [&](uint32_t x, uint32_t& total) {
    __syncthreads();
    return block_scan<kEvictWarps>(x, sums, warp, lane, total);
  };
  // counts of the CTAs before this one, and of all
  auto across = [&](int which, uint32_t& all) -> uint32_t {
    const uint32_t v = lane < static_cast<int>(C) ? (C == 1 ? pub[which] : peer_load(peer_addr(&pub[which], lane))) : 0;
    const uint32_t incl = warp_incl_scan(v, lane);
    all = __shfl_sync(0xffffffffu, incl, 31);
    return __shfl_sync(0xffffffffu, incl - v, static_cast<int>(rank_c));
  };
  uint32_t ties = 0, cta_total, n_ties;
  for (int32_t b = w0; b < w1; b += 32) ties += __popc(__ballot_sync(0xffffffffu, b + lane < w1 && key(b + lane) == prefix));
  uint32_t tie0 = scan(ties, cta_total);
  if (tid == 0) {
    pub[0] = cta_total;
    if (rank_c == 0) {        // room in the list for as many moves as there can be
      const unsigned long long at = atomicAdd(p.alloc, static_cast<unsigned long long>(min(gone, kept)));
      pub[3] = static_cast<uint32_t>(at);
      pub_hi = static_cast<uint32_t>(at >> 32);
    }
  }
  __syncthreads();
  if (C > 1) cluster_sync();
  tie0 += across(0, n_ties);
  const uint32_t tie_keep = n_ties - rank;   // ties that stay: the first ones
  const int64_t list0 = C == 1 ? static_cast<int64_t>(pub_hi) << 32 | pub[3]
                               : static_cast<int64_t>(peer_load(peer_addr(&pub_hi, 0))) << 32 | peer_load(peer_addr(&pub[3], 0));
  const bool room = list0 + min(gone, kept) <= p.move_cap;
  auto walk = [&](auto&& f) {
    uint32_t tie = tie0;
    for (int32_t b = w0; b < w1; b += 32) {
      const int32_t x = b + lane, t = first + x;
      const uint32_t k = x < w1 ? key(x) : 0xFFFFFFFFu;
      const uint32_t eq = __ballot_sync(0xffffffffu, x < w1 && k == prefix);
      const uint32_t below = __popc(eq & ((1u << lane) - 1u));
      const bool go = x < w1 && (k < prefix || (k == prefix && tie + below >= tie_keep));
      tie += __popc(eq);
      const uint32_t holes = __ballot_sync(0xffffffffu, go && t < kept);
      const uint32_t backs = __ballot_sync(0xffffffffu, x < w1 && !go && t >= kept);
      f(t, holes, backs);
    }
  };
  uint32_t nh = 0, nb = 0;
  walk([&](int32_t, uint32_t holes, uint32_t backs) {
    nh += __popc(holes);
    nb += __popc(backs);
  });
  uint32_t h0 = scan(nh, cta_total);
  if (tid == 0) pub[1] = cta_total;
  uint32_t b0 = scan(nb, cta_total);
  if (tid == 0) pub[2] = cta_total;
  __syncthreads();
  if (C > 1) cluster_sync();
  uint32_t moves, n_backs;
  h0 += across(1, moves);
  b0 += across(2, n_backs);
  int2* list = p.moves + list0;
  if (room)
    walk([&](int32_t t, uint32_t holes, uint32_t backs) {
      const uint32_t lt = (1u << lane) - 1u;
      if (holes >> lane & 1u) list[h0 + __popc(holes & lt)].y = t;
      if (backs >> lane & 1u) list[b0 + __popc(backs & lt)].x = t;
      h0 += __popc(holes);
      b0 += __popc(backs);
    });
  __syncthreads();
  if (C > 1) cluster_sync();   // the list is whole, and nobody reads another CTA's shared memory any more
  done();
  if (!room) {                 // sequences that share pages: more tokens than the pool has
    if (tid == 0) note_error(c, SR_DEVERR_WORKSPACE);
    return;
  }

  // ---- move
  if (rank_c == 0 && tid == 0) c.seq_len[seq] = kept;
  const int32_t* table = c.table + static_cast<int64_t>(seq) * c.max_pages;
  const int vpr = c.n_kv * c.head_dim * (c.page_type == SR_PAGE_BF16 ? 2 : 1) / 16;
  for (uint32_t j = warp * C + rank_c; j < moves; j += C * kEvictWarps) {
    const int2 m = __ldcg(list + j);
    move_token(c, table, tpos, mass, m, vpr, lane);
  }
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

// Shared memory of the small form: the keys, and this CTA's share of the moves.
static size_t pick_bytes(int32_t cap, int32_t most, unsigned C) {
  return static_cast<size_t>((cap + 3) / 4 * 4) * 4 + (static_cast<size_t>(most) / C + 1) * sizeof(int2);
}

cudaError_t paged_evict_prepare() {
  const cudaError_t e = cudaFuncSetAttribute(paged_evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(pick_bytes(kPickLimit, kPickLimit / 2, kMaxCluster)));
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(paged_evict_long_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kKeyLimit * 4);
}

// CTAs per sequence: one where there are few tokens to move (no barrier across CTAs
// then), else a whole cluster.
cudaError_t launch_paged_evict(const EvictParams& p, cudaStream_t st) {
  // a move fills an index that goes with a token that stays: at most so many
  const int32_t cap = p.c.cap, most = std::min(cap / 2, cap - p.budget);
  const bool small = cap <= kPickLimit;
  const unsigned C = small && most <= 64 ? 1 : kMaxCluster;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.b.n) * C);
  cfg.blockDim = dim3(small ? kPickThreads : kEvictThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (small) {
    cfg.dynamicSmemBytes = pick_bytes(cap, most, C);
    return cudaLaunchKernelEx(&cfg, paged_evict_kernel, p, static_cast<int>((cap + 3) / 4 * 4));
  }
  const int32_t per = static_cast<int32_t>(C) * kEvictThreads;
  const int key_cap = std::min((cap + per - 1) / per * kEvictThreads, kKeyLimit);
  cfg.dynamicSmemBytes = static_cast<size_t>(key_cap) * 4;
  return cudaLaunchKernelEx(&cfg, paged_evict_long_kernel, p, key_cap);
}

}  // namespace sr
