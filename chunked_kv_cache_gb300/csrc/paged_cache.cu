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
// finish raises its length (every CTA has read the old one by then). 42,684 rows of 1024
// values: 58.8 us for 350 MB (5.9 TB/s, 88 % of the copy rate), to e4m3 47.8 us for 262 MB
// (81 %); one sequence of 64 rows: 3.2 us of the GPU, less than the call costs the host.
constexpr int kAppendThreads = 256;
constexpr int kAppendUnroll = 4;      // vectors of each tensor in flight per thread

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
    const int vpr = c.n_kv * c.head_dim / 8;    // vectors per row
    const uint4* ksrc = reinterpret_cast<const uint4*>(p.k) + static_cast<int64_t>(p.row0[i] + r0) * vpr;
    const uint4* vsrc = reinterpret_cast<const uint4*>(p.v) + static_cast<int64_t>(p.row0[i] + r0) * vpr;
    const int head_shift = c.head_dim == 128 ? 4 : 3;
    auto put = [&](int r, int col, const uint4& kx, const uint4& vx) {
      const int32_t t = len + r0 + r;
      const int32_t pg = page_of_group(t >> 4, c.magic);
      const int64_t at = (static_cast<int64_t>(table[pg]) * c.page_tokens + (t - pg * c.page_tokens)) * vpr + col;
      if constexpr (TYPE == SR_PAGE_BF16) {
        static_cast<uint4*>(c.k_pages)[at] = kx;
        static_cast<uint4*>(c.v_pages)[at] = vx;
      } else {
        const int head = col >> head_shift;
        const float ki = c.kv_exp ? exp2f(-static_cast<float>(c.kv_exp[head])) : 1.f;
        const float vi = c.kv_exp ? exp2f(-static_cast<float>(c.kv_exp[c.n_kv + head])) : 1.f;
        static_cast<uint2*>(c.k_pages)[at] = to_e4m3(kx, ki);
        static_cast<uint2*>(c.v_pages)[at] = to_e4m3(vx, vi);
      }
    };
    // row and vector of it, advanced by the block's size without a division
    const int step_r = kAppendThreads / vpr, step_c = kAppendThreads - step_r * vpr;
    int r = static_cast<int>(threadIdx.x) / vpr, col = static_cast<int>(threadIdx.x) - r * vpr;
    for (int x0 = threadIdx.x; x0 < rows * vpr; x0 += kAppendUnroll * kAppendThreads) {
      uint4 kx[kAppendUnroll], vx[kAppendUnroll];
#pragma unroll
      for (int u = 0; u < kAppendUnroll; ++u)
        if (x0 + u * kAppendThreads < rows * vpr) {
          kx[u] = __ldcs(ksrc + x0 + u * kAppendThreads);
          vx[u] = __ldcs(vsrc + x0 + u * kAppendThreads);
        }
#pragma unroll
      for (int u = 0; u < kAppendUnroll; ++u) {
        if (x0 + u * kAppendThreads < rows * vpr) put(r, col, kx[u], vx[u]);
        r += step_r;
        col += step_c;
        if (col >= vpr) {
          col -= vpr;
          ++r;
        }
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
// One launch, a cluster of CTAs per sequence, each with a stretch of its indices. The
// weights' bits, mapped to unsigned integers in the weights' order, are read once into
// shared memory. A radix select (11, 11 and 10 bits, the CTAs' counts added through
// distributed shared memory) narrows the keys down to those that share the digits of
// the last key to go; as soon as these are few every CTA gathers them, one per thread, and
// goes on by itself with digits of the key, then of the index, which settles ties. The
// result is a cut: a token goes if its key lies below the cut's, or equals it at an index at
// or behind the cut's. Ordered counts turn that into moves (from, to), and all warps move
// rows, a warp per token. A move reads at or behind the new length and writes below it, so
// that no move sees another.
// Latency bound (barriers, dependent loads, code that runs once) until the moves, which are
// HBM bound: 512 of 16896 tokens go from each of 16 sequences, 1024 values to a row, in
// 30 us, where the 70 MB alone would take 10 us. One token of a sequence (the least weight, no
// digits) goes in 4 us of the GPU from 8 sequences of 1025 tokens, 5 us from 32 of 4097.
constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
// Up to here the first CTA of a cluster looks for the one lightest token by itself (with an append, by itself and by
// the cluster: 8 sequences of 1025 tokens 5.9, 7.2 us, of 4097 6.8, 7.3 us, of 8001 7.2, 7.3 us; 16 of 4601 7.4, 7.5 us,
// of 6001 7.7, 7.4 us; 32 of 4097 7.7, 7.9 us, of 4601 7.9, 7.9 us, of 8001 8.4, 7.9 us).
constexpr int32_t kAlone = 4608;
constexpr int kCandidates = 512;      // keys gathered to find the cut among them
constexpr int kKeyLimit = 45056;      // keys a CTA can hold; longer stretches are read again from global memory
static_assert(kCandidates <= kEvictThreads, "a thread holds one candidate");

// The order of the weights as unsigned integers; protected tokens come last.
constexpr uint32_t kProtected = 0xFFFFFFFFu;
__device__ __forceinline__ uint32_t weight_key(float m) {
  if (m != m) return kProtected - 1;
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
// The cluster's barrier; a block's where there is one CTA.
__device__ __forceinline__ void cluster_sync(uint32_t C) {
  if (C == 1)
    __syncthreads();
  else
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the address of a CTA's copy of a shared variable, and loads from it
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
__device__ __forceinline__ uint2 peer_load2(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared::cluster.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint4 peer_load4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}

// What the CTAs of a cluster read of one another.
struct EvictShared {
  uint32_t hist[2][kBins];
  uint2 cand[kCandidates];          // (key, index) of this CTA's candidates
  uint32_t n_cand, n_ties, n_holes, n_backs, cut_index;
  unsigned long long list0;         // rank 0: the sequence's first entry in the list of moves
  unsigned long long lightest;      // one token to go: the smallest (key, complement of the index)
};

// A warp moves one token's rows.
__device__ __forceinline__ void move_rows(const PagedView& c, int64_t from, int64_t to, int vpr, int lane) {
  const uint4* ks = static_cast<const uint4*>(c.k_pages) + from * vpr;
  const uint4* vs = static_cast<const uint4*>(c.v_pages) + from * vpr;
  uint4* kd = static_cast<uint4*>(c.k_pages) + to * vpr;
  uint4* vd = static_cast<uint4*>(c.v_pages) + to * vpr;
  for (int x0 = lane; x0 < vpr; x0 += 128) {     // eight loads in flight per lane
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

__global__ void __launch_bounds__(kEvictThreads, 2) paged_evict_kernel(const __grid_constant__ EvictParams p, int key_cap) {
  extern __shared__ uint32_t keys[];              // [key_cap]
  __shared__ __align__(16) EvictShared sh;
  __shared__ uint32_t sums[2][kEvictWarps];
  __shared__ uint32_t found[3];                   // digit, rank in it, its keys
  __shared__ uint2 cut_at;
  uint32_t C = cluster_size();
  const uint32_t me = cluster_rank();
  const int i = blockIdx.x / C, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  for (int x = tid; x < 2 * kBins; x += kEvictThreads) (&sh.hist[0][0])[x] = 0;
  if (tid == 0) sh.n_cand = 0;
  grid_dep_launch_dependents();
  grid_dep_wait();
  const PagedView& c = p.c;
  const int32_t seq = p.b.id[i];
  const int32_t len = min(max(c.seq_len[seq], 0), c.cap);
  const int64_t recent0 = static_cast<int64_t>(c.seq_pos[seq]) - p.n_recent;
  // the last sequence to be done clears the list's counters for the next call
  auto done = [&] {
    if (me == 0 && tid == 0 && atomicAdd(p.alloc + 1, 1ull) == static_cast<unsigned long long>(p.b.n) - 1) {
      p.alloc[0] = 0;
      p.alloc[1] = 0;
    }
  };
  if (len <= p.budget) {                          // as in every CTA of the cluster
    done();
    return;
  }
  const bool one = len - p.budget == 1;           // token too many
  if (one && len <= kAlone) {
    if (me != 0) return;
    C = 1;
  }
  int32_t* tpos = c.token_pos + static_cast<int64_t>(seq) * c.cap;
  float* mass = c.token_mass + static_cast<int64_t>(seq) * c.cap;
  auto key_of = [&](int32_t q, float m) { return q < p.n_sink || q >= recent0 ? kProtected : weight_key(m); };
  // this CTA's stretch of indices, and a warp's: a multiple of 32
  const int32_t chunk = static_cast<int32_t>((len + C * kEvictThreads - 1) / (C * kEvictThreads)) * kEvictThreads;
  const int32_t first = min(static_cast<int32_t>(me) * chunk, len), count = min(chunk, len - first);
  const int32_t w0 = min(warp * (chunk / kEvictWarps), count), w1 = min(w0 + chunk / kEvictWarps, count);
  // f(x, key) for this warp's indices, eight loads of each array in flight, short stretches' as well
  auto load_keys = [&](auto&& f) {
    constexpr int kBatch = 8;
    for (int32_t x0 = w0 + lane; x0 < w1; x0 += 32 * kBatch) {
      int32_t q[kBatch];
      float m[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (x0 + 32 * k < w1) {
          q[k] = tpos[first + x0 + 32 * k];
          m[k] = mass[first + x0 + 32 * k];
        }
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (x0 + 32 * k < w1) f(x0 + 32 * k, key_of(q[k], m[k]));
    }
  };
  const bool held = !one && chunk <= key_cap;
  if (held) load_keys([&](int32_t x, uint32_t k) { keys[x] = k; });   // a warp reads the keys that it wrote
  const int32_t* table = c.table + static_cast<int64_t>(seq) * c.max_pages;
  const int vpr = c.n_kv * c.head_dim * (c.page_type == SR_PAGE_BF16 ? 2 : 1) / 16;
  if (one) {
    // ---- one token too many, as in serving token by token: the lightest goes, and the last
    // index's token takes its place
    unsigned long long best = ~0ull;
    load_keys([&](int32_t x, uint32_t k) {
      if (k != kProtected)
        best = min(best, static_cast<unsigned long long>(k) << 32 | static_cast<uint32_t>(~(first + x)));
    });
    auto warp_min = [](unsigned long long v) {
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) v = min(v, __shfl_xor_sync(0xffffffffu, v, s));
      return v;
    };
    best = warp_min(best);
    unsigned long long* mins = reinterpret_cast<unsigned long long*>(sh.cand);
    if (lane == 0) mins[warp] = best;
    __syncthreads();
    if (warp == 0) {
      best = warp_min(lane < kEvictWarps ? mins[lane] : ~0ull);
      if (lane == 0) sh.lightest = best;
    }
    cluster_sync(C);
    if (me == 0 && warp == 0) {
      if (C > 1) {
        best = ~0ull;
        if (lane < static_cast<int>(C)) {
          const uint2 v = peer_load2(peer_addr(&sh.lightest, lane));
          best = static_cast<unsigned long long>(v.y) << 32 | v.x;
        }
        best = warp_min(best);
      }
      best = __shfl_sync(0xffffffffu, best, 0);
      const int32_t at = static_cast<int32_t>(~static_cast<uint32_t>(best)), last = len - 1;
      if (best != ~0ull) {
        bool whole = true;                        // nothing to move, or both ends have a page
        if (at != last) {
          const int64_t from = paged_row(table, last, c.page_tokens, c.n_pages);
          const int64_t to = paged_row(table, at, c.page_tokens, c.n_pages);
          whole = from >= 0 && to >= 0;
          if (whole) {
            if (lane == 0) {
              tpos[at] = tpos[last];
              mass[at] = mass[last];
            }
            move_rows(c, from, to, vpr, lane);
          } else if (lane == 0) {
            note_error(c, SR_DEVERR_BAD_PAGE);
          }
        }
        if (whole && lane == 0) c.seq_len[seq] = last;
      }
    }
    if (C > 1) cluster_sync(C);   // this CTA's lightest has been read
    done();
    return;
  }

  auto key = [&](int32_t x) { return x >= w1 ? kProtected : held ? keys[x] : key_of(tpos[first + x], mass[first + x]); };
  __syncthreads();


  // ---- the key of rank `rank` (from 1) among those that may go
  uint32_t prefix = 0, rank = 0;
  uint32_t cut_key = 0, cut_index = 0;
  int32_t gone = 0;
  int pass = 0;
  unsigned long long list_at = 0;
  // Equal digits queue on one counter (weights share their leading bits): a warp adds those of its first lane
  // at once. 2 sequences of 105000 tokens, 5000 to go: 40.8 us where it did so only if all were equal, 34.4 us
  // so, 44.5 us with up to four rounds of it, 46.5 us with the warp's lanes matched among each other.
  auto tally = [&](uint32_t* h, bool in, uint32_t digit) {
    const uint32_t act = __ballot_sync(0xffffffffu, in);
    if (act == 0) return;
    const uint32_t d0 = __shfl_sync(0xffffffffu, digit, __ffs(act) - 1);
    const uint32_t same = __ballot_sync(0xffffffffu, in && digit == d0);
    if (lane == 0) atomicAdd(&h[d0], __popc(same));
    if (in && digit != d0) atomicAdd(&h[digit], 1u);
  };
  // the keys before this thread's four digits, of which it has s; all of them in `total`
  auto keys_before = [&](const uint4& s, uint32_t& total) {
    const uint32_t mine = s.x + s.y + s.z + s.w;
    const uint32_t incl = warp_incl_scan(mine, lane);
    if (lane == 31) sums[0][warp] = incl;
    __syncthreads();
    const uint32_t ws = lane < kEvictWarps ? sums[0][lane] : 0;
    const uint32_t wi = warp_incl_scan(ws, lane);
    total = __shfl_sync(0xffffffffu, wi, 31);
    return incl - mine + __shfl_sync(0xffffffffu, wi - ws, warp);
  };
  // the digit of the rank-th key
  auto find = [&](const uint4& s, uint32_t before) {
    const uint32_t v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (before < rank && rank <= before + v[j]) {
        found[0] = tid * 4 + j;
        found[1] = rank - before;
        found[2] = v[j];
      }
      before += v[j];
    }
    __syncthreads();
  };
#pragma unroll 1
  for (;; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, above = pass == 1 ? 21 : 10;
    const uint32_t digits = pass == 2 ? 1023 : 2047;
    uint32_t* h = sh.hist[pass & 1];
    for (int32_t x0 = w0; x0 < w1; x0 += 32) {
      const uint32_t k = key(x0 + lane);
      const bool in = k != kProtected && (pass == 0 || k >> above == prefix >> above);
      tally(h, in, k >> shift & digits);
    }
    cluster_sync(C);
    // every CTA adds all counts, four digits per thread, and finds the same digit
    uint4 s = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (uint32_t r = 0; r < kMaxCluster; ++r)
      if (r < C) {
        const uint4 v = C == 1 ? *reinterpret_cast<const uint4*>(h + tid * 4) : peer_load4(peer_addr(h + tid * 4, r));
        s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
      }
    uint32_t total;
    const uint32_t before = keys_before(s, total);
    if (pass == 0) {
      gone = static_cast<int32_t>(min(static_cast<uint32_t>(len - p.budget), total));   // of those that may go
      rank = static_cast<uint32_t>(gone);
      // the sequence's place in the list of moves, long before it is needed
      if (me == 0 && tid == 31) list_at = atomicAdd(p.alloc, static_cast<unsigned long long>(min(gone, len - gone)));
    }
    find(s, before);
    if (gone == 0) {          // every token is protected; as in every CTA of the cluster
      cluster_sync(C);        // the others may still be reading this CTA's counts
      done();
      return;
    }
    prefix |= found[0] << shift;
    rank = found[1];
    const uint32_t n = found[2];
    if (rank == n) {                              // all of this digit's keys go
      cut_key = min(prefix | ((1u << shift) - 1u), kProtected - 1);
      cut_index = 0;
      break;
    }
    if (n <= kCandidates) {
      // gather these keys and rank them: lighter first, of equal ones the last index
      for (int32_t x0 = w0; x0 < w1; x0 += 32) {
        const uint32_t k = key(x0 + lane);
        const bool in = k != kProtected && k >> shift == prefix >> shift;
        const uint32_t act = __ballot_sync(0xffffffffu, in);
        if (act == 0) continue;
        uint32_t at = 0;
        if (lane == 0) at = atomicAdd(&sh.n_cand, __popc(act));
        at = __shfl_sync(0xffffffffu, at, 0);
        if (in) sh.cand[at + __popc(act & ((1u << lane) - 1u))] = make_uint2(k, static_cast<uint32_t>(first + x0 + lane));
      }
      cluster_sync(C);
      uint2 my = make_uint2(0, 0);
      uint32_t m[kMaxCluster], from = 0, place = 0, owner = 0;   // candidates of each CTA: n in all
#pragma unroll
      for (uint32_t r = 0; r < kMaxCluster; ++r)
        m[r] = r >= C ? 0 : C == 1 ? sh.n_cand : peer_load(peer_addr(&sh.n_cand, r));
#pragma unroll
      for (uint32_t r = 0; r < kMaxCluster; ++r) {
        const uint32_t at = static_cast<uint32_t>(tid) - from;
        if (at < m[r]) {
          place = at;
          owner = r;
        }
        from += m[r];
      }
      bool alive = static_cast<uint32_t>(tid) < n;
      if (alive) my = C == 1 ? sh.cand[place] : peer_load2(peer_addr(&sh.cand[place], owner));
      // The rank-th of n <= 512 distinct values, one per thread, by digits of this CTA's own until one is left.
      // (The others have read this CTA's counts before the barrier above.)
      const unsigned long long v = static_cast<unsigned long long>(my.x & ((1u << shift) - 1u)) << 24 | (~my.y & 0xFFFFFFu);
      uint32_t* own = sh.hist[0];
      for (int top = shift + 24;;) {
        const int low = max(top - 11, 0);
        reinterpret_cast<uint4*>(own)[tid] = make_uint4(0, 0, 0, 0);
        __syncthreads();
        const uint32_t digit = static_cast<uint32_t>(v >> low) & ((1u << (top - low)) - 1u);
        tally(own, alive, digit);
        __syncthreads();
        const uint4 mine = reinterpret_cast<uint4*>(own)[tid];
        uint32_t all;
        find(mine, keys_before(mine, all));
        alive = alive && digit == found[0];
        rank = found[1];
        top = low;
        if (found[2] == 1 || low == 0) break;
      }
      if (alive) cut_at = my;
      __syncthreads();
      cut_key = cut_at.x;
      cut_index = cut_at.y;
      break;
    }
    if (pass == 2) {
      // more equal keys than that: the cut is the tie before which n - rank ties stay
      uint32_t ties = 0;
      for (int32_t x0 = w0; x0 < w1; x0 += 32) ties += __popc(__ballot_sync(0xffffffffu, key(x0 + lane) == prefix));
      if (lane == 0) sums[1][warp] = ties;
      __syncthreads();
      const uint32_t tv = lane < kEvictWarps ? sums[1][lane] : 0;
      const uint32_t ti = warp_incl_scan(tv, lane);
      if (tid == 31) sh.n_ties = ti;
      cluster_sync(C);
      const uint32_t pv = lane < static_cast<int>(C) ? (C == 1 ? sh.n_ties : peer_load(peer_addr(&sh.n_ties, lane))) : 0;
      const uint32_t pi = warp_incl_scan(pv, lane);
      uint32_t tie = __shfl_sync(0xffffffffu, pi - pv, static_cast<int>(me)) + __shfl_sync(0xffffffffu, ti - tv, warp);
      if (tid == 0) sh.cut_index = 0xFFFFFFFFu;
      __syncthreads();
      for (int32_t x0 = w0; x0 < w1; x0 += 32) {
        const bool eq = key(x0 + lane) == prefix;
        const uint32_t act = __ballot_sync(0xffffffffu, eq);
        if (eq && tie + __popc(act & ((1u << lane) - 1u)) == n - rank) sh.cut_index = first + x0 + lane;
        tie += __popc(act);
      }
      cluster_sync(C);
      uint32_t ci = lane < static_cast<int>(C) ? (C == 1 ? sh.cut_index : peer_load(peer_addr(&sh.cut_index, lane))) : 0xFFFFFFFFu;
      cut_index = __reduce_min_sync(0xffffffffu, ci);
      cut_key = prefix;
      break;
    }
    // the first buffer, read by all before this pass's barrier, serves the third pass
    if (pass == 1)
      for (int x = tid; x < kBins; x += kEvictThreads) sh.hist[0][x] = 0;
    __syncthreads();
  }
  const int32_t kept = len - gone;   // the new length

  // ---- the moves: the j-th index below `kept` that goes, the j-th at or behind it that stays
  auto walk = [&](auto&& f) {
    for (int32_t x0 = w0; x0 < w1; x0 += 32) {
      const int32_t x = x0 + lane, t = first + x;
      const uint32_t k = key(x);
      const bool go = k < cut_key || (k == cut_key && static_cast<uint32_t>(t) >= cut_index);
      f(t, __ballot_sync(0xffffffffu, go && t < kept), __ballot_sync(0xffffffffu, x < w1 && !go && t >= kept));
    }
  };
  // A sequence is evicted from whole or not at all: one with an end of a move on no page of the pool stays as it
  // is. The counts carry that in their top bit, so that all CTAs of the cluster know before anything is written.
  constexpr uint32_t kNoPage = 1u << 31;
  uint32_t nh = 0, nb = 0;
  bool off = false;
  walk([&](int32_t t, uint32_t holes, uint32_t backs) {
    nh += __popc(holes);
    nb += __popc(backs);
    if ((holes | backs) >> lane & 1u) off |= static_cast<uint32_t>(table[page_of_group(t >> 4, c.magic)]) >= static_cast<uint32_t>(c.n_pages);
  });
  if (__any_sync(0xffffffffu, off)) nh |= kNoPage;
  __syncthreads();
  if (lane == 0) {
    sums[0][warp] = nh;
    sums[1][warp] = nb;
  }
  __syncthreads();
  uint32_t hv = lane < kEvictWarps ? sums[0][lane] : 0;
  const uint32_t bv = lane < kEvictWarps ? sums[1][lane] : 0;
  const uint32_t off_here = __any_sync(0xffffffffu, hv & kNoPage) ? kNoPage : 0;
  hv &= ~kNoPage;
  const uint32_t hi = warp_incl_scan(hv, lane), bi = warp_incl_scan(bv, lane);
  const uint32_t most = static_cast<uint32_t>(min(gone, kept));   // moves there can be
  if (tid == 31) {
    sh.n_holes = hi | off_here;
    sh.n_backs = bi;
    sh.list0 = list_at;        // of the first CTA
  }
  cluster_sync(C);
  const uint2 l2 = C == 1 ? *reinterpret_cast<const uint2*>(&sh.list0) : peer_load2(peer_addr(&sh.list0, 0));
  uint32_t ph = 0, pb = 0;
  if (lane < static_cast<int>(C)) {
    ph = C == 1 ? sh.n_holes : peer_load(peer_addr(&sh.n_holes, lane));
    pb = C == 1 ? sh.n_backs : peer_load(peer_addr(&sh.n_backs, lane));
  }
  const bool paged = !__any_sync(0xffffffffu, ph & kNoPage);
  ph &= ~kNoPage;
  const uint32_t phi = warp_incl_scan(ph, lane), pbi = warp_incl_scan(pb, lane);
  const uint32_t moves = __shfl_sync(0xffffffffu, phi, 31);
  uint32_t h0 = __shfl_sync(0xffffffffu, phi - ph, static_cast<int>(me)) + __shfl_sync(0xffffffffu, hi - hv, warp);
  uint32_t b0 = __shfl_sync(0xffffffffu, pbi - pb, static_cast<int>(me)) + __shfl_sync(0xffffffffu, bi - bv, warp);
  const int64_t list0 = static_cast<int64_t>(l2.y) << 32 | l2.x;
  const bool room = list0 + most <= p.move_cap;
  int2* list = p.moves + list0;
  if (room && paged)
    walk([&](int32_t t, uint32_t holes, uint32_t backs) {
      const uint32_t lt = (1u << lane) - 1u;
      if (holes >> lane & 1u) list[h0 + __popc(holes & lt)].y = t;
      if (backs >> lane & 1u) list[b0 + __popc(backs & lt)].x = t;
      h0 += __popc(holes);
      b0 += __popc(backs);
    });
  cluster_sync(C);             // the list is whole; nobody reads another CTA's shared memory, or a weight, any more
  done();
  if (!room || !paged) {       // no room: sequences that share pages, more tokens than the pool has
    if (tid == 0) note_error(c, paged ? SR_DEVERR_WORKSPACE : SR_DEVERR_BAD_PAGE);
    return;
  }

  // ---- move: a warp looks up 32 of its moves at once, then takes them one by one
  if (me == 0 && tid == 0) c.seq_len[seq] = kept;
  const uint32_t step = C * kEvictWarps;
  for (uint32_t j0 = warp * C + me; j0 < moves; j0 += 32 * step) {
    const uint32_t j = j0 + lane * step;
    int64_t from = -1, to = -1;
    if (j < moves) {
      const int2 m = __ldcg(list + j);
      from = paged_row(table, m.x, c.page_tokens, c.n_pages);
      to = paged_row(table, m.y, c.page_tokens, c.n_pages);
      tpos[m.y] = tpos[m.x];
      mass[m.y] = mass[m.x];
    }
    const int n = static_cast<int>(min((moves - j0 + step - 1) / step, 32u));
    for (int q = 0; q < n; ++q) {
      const int64_t f = __shfl_sync(0xffffffffu, from, q), g = __shfl_sync(0xffffffffu, to, q);
      if ((f | g) < 0) continue;      // an entry that the caller changed during the call
      move_rows(c, f, g, vpr, lane);
    }
  }
}

}  // namespace

// One wave of the four CTAs that an SM holds, but at least a vector of each tensor per thread; two
// waves where a thread would have more than 16 (42,700 rows of 1024 values: 61.3 us in one, 58.9 us in
// two; 4,000 rows: 7.5 us, 9.1 us).
int paged_append_rows_per_cta(int n_kv, int head_dim, int64_t rows) {
  const int64_t vectors = static_cast<int64_t>(n_kv) * head_dim / 8;     // of a row
  const int64_t wave = 4ll * sm_count();
  const int64_t ctas = rows * vectors > 16 * wave * kAppendThreads ? 2 * wave : wave;
  return static_cast<int>(std::max((kAppendThreads + vectors - 1) / vectors, (rows + ctas - 1) / ctas));
}

cudaError_t launch_paged_reset(const PagedView& c, const PagedBatch& b, cudaStream_t st) {
  return launch_dependent(paged_reset_kernel, 1, 256, 0, st, c, b);
}

cudaError_t launch_paged_append(const AppendParams& p, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>(p.cta0[p.n]);
  if (p.c.page_type == SR_PAGE_BF16) return launch_dependent(paged_append_kernel<SR_PAGE_BF16>, grid, kAppendThreads, 0, st, p);
  return launch_dependent(paged_append_kernel<SR_PAGE_E4M3>, grid, kAppendThreads, 0, st, p);
}

cudaError_t paged_evict_prepare() {
  return cudaFuncSetAttribute(paged_evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kKeyLimit * 4);
}

cudaError_t launch_paged_evict(const EvictParams& p, cudaStream_t st) {
  // CTAs per sequence: a whole cluster while every CTA has an SM to itself, fewer in larger
  // batches (32 sequences of 4160 tokens, 64 to move, with an append: 18.4 us with 4, 21.5 us with 8; 64 of
  // 576, 64 to move: 22.9 us with 2, 37.2 us with 8; 16 of 16896, 512 to move: 51.0 us with 4, 41.3 us with 8).
  const int32_t cap = p.c.cap;
  const unsigned room = static_cast<unsigned>(std::max(1, sm_count() / p.b.n));
  unsigned C = kMaxCluster;
  while (C > room) C /= 2;
  const int32_t per = static_cast<int32_t>(C) * kEvictThreads;
  const int key_cap = std::min((cap + per - 1) / per * kEvictThreads, kKeyLimit);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.b.n) * C);
  cfg.blockDim = dim3(kEvictThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(key_cap) * 4;
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
  return cudaLaunchKernelEx(&cfg, paged_evict_kernel, p, key_cap);
}

}  // namespace sr
