// paged_attention.cuh -- attention of one new token per sequence over the paged
// token cache, and the attention weight that each cached token draws.
//
//   x_h(t) = scale * q_h . k(t),  o_h = sum_t e^(x_h(t) - lse_h) v(t),
//   lse_h = ln sum_t e^x_h(t),    mass(t) <- decay * mass(t) + sum_h e^(x_h(t) - lse_h).
//
// With up to 16 query heads per key/value head it is bound by the one read of the cache, and
// every choice below serves that stream. More query heads of one key head are taken in equal
// parts of at most 16, each an item that reads the head for itself; parts lie side by side, so
// that most of the reads end in L2, as far as 2, 4 or 8 divides the number of items per token.
// That form is bound by the parts' own copies and products: 32 sequences of 4096 tokens and one
// key head of 128 (10 us of bytes) take 19.7 us with 16 query heads, 27.2 us with 32, 45.5 us
// with 64, 69.6 us with 128. Shares without large divisors up to 16 come in many parts and are
// slow: 18 heads (2 parts of 9) 25.6 us, but 17 (17 of one) and 34 (17 of 2) 110.8 us; 72 (6 of
// 12) 56.9 us, but 71 (71 of one) 426.6 us, with a head dim of 64 256.2 us.
//
// Work split. A sequence and key/value head (an item) is cut into tiles of CT
// tokens; the launch's tiles, item after item, form one line, and every CTA takes an
// equal stretch of it, whatever the lengths: a batch of unequal sequences and a
// single long one both occupy the whole GPU, and the lengths, which only the device
// knows, never reach the host. Where items are nearly equal, or small, the stretches end
// where items end (the rule stands at kWhole). A CTA that covers an item whole writes its
// output; of an item cut between CTAs each writes its partial result (fp32 sums, maximum and
// sum of the softmax), and the last of them to arrive joins the parts in the order of the
// line, so that results do not depend on timing. More than kJoin parts are joined in two
// levels (kJoin neighbours first), so that no CTA reads many of them by itself. Many rows of
// many parts are joined by a launch of their own (the rule stands at the launch).
//
// Inside a CTA each of four warps owns a quarter of every tile and runs by itself: it
// copies its tokens' keys and values into its own three shared-memory stages (4-bit pages of 128 dims: two)
// (cp.async, 16-byte chunks, rows past the length filled with zeros; 4-bit pages: bulk copies) and computes on
// the oldest stage. The copies run ahead across items, so that the stream does not pause
// where one item ends.
//
// The products are transposed: scores = keys (16 rows) x queries (8 columns), sums =
// values^T (16 dims) x weights (8 columns), so that a group of up to 8 query heads wastes
// nothing that 16 rows of queries would (64 sequences of 4096 tokens, e4m3: 94.3 us with queries as rows, 89.5 us so). The
// weights turn from the one product's result into the other's operand by an 8x8
// transposition between registers and never leave them. Warp-level products fit here: the
// rows that a tcgen05 tile would need (128) are not there, and the tensor pipe is idle for
// more than half of the time. The merge of the four warps' sums uses the stages just read.
//
// What bounds it: the stream, at 6.5 - 6.9 TB/s once it runs, and about 7 us per call before
// and after it (lengths, the first copies, merge, join); with e4m3 pages and head dim 64 the
// arithmetic too, since a scheduler has two warps. 8 sessions of 2072 .. 11432 tokens with 40
// heads of 128: 144 us for 963 MB (6.7 TB/s, 99 % of the copy rate); one of 131071, 8 heads: 84 us for
// 537 MB (95 %); 32 of 4001 .. 32768, e4m3: 144 us for 935 MB (96 %); 64 of 1 .. 16384: 87 us for
// 522 MB (89 %); 16 of 1000 .. 8192 with weights: 50 us for 232 MB (69 %).
//
// 4-bit pages: a warp's records come by bulk copies, one for each 16 tokens' keys or values, and their codes become fp16 in
// registers: the matrix load that brings a word of eight codes (16-bit units of four, transposed for the values) leaves
// just the pairs that five instructions of logic and four fused products and sums turn into eight operands, scale and all.
// That decoding is what bounds it: 355 instructions for 16 tokens of 128 dims (255 of 64), of which two warps a scheduler issue
// 2.2 a cycle and SM, waiting for one another's results (no pipe is above 52 %; at four a cycle the stream would bound). 32
// sequences of 4001 .. 32768 tokens, 8 key heads: 124.7 us for 526 MB (4.2 TB/s, 62 % of the copy rate; e4m3, 935 MB: 144
// us); one of 131071: 41 us for 151 MB; 64 of 1 .. 16384, 64 dims: 35 us for 75 MB, 49 us with weights, of which storing the
// scores is 1 us and the second launch the rest. Written with the masks and their bits as constants the compiler made two instructions of each: 149 us for
// the first of these.
//
// A few new tokens per sequence (drafts to verify), whose heads fit the 16 columns: columns are (token, head) pairs, and the
// last tokens' scores are masked by column. 4 tokens of 16 sequences of 1000 .. 8192, 32 heads, 8 key heads, 4 bits: 35 us (e4m3
// 37, bf16 50), where blocks of 128 rows (paged_prompt.cu) took 64 us; 8 tokens, which go there: 83, 70 and 59 us.
//
// Precision. Scores, softmax statistics and sums are fp32. bf16 pages: a weight meets the
// values as two bf16 numbers, itself rounded and what that leaves (2^-15 of it at most is lost):
// the second product costs under 1 % of the time (85.4 us and 84.8 us for 16 sequences of 8192
// tokens), and without it outputs were 0.0023 off in the mean instead of 0.0017, of which 0.0017
// is the rounding of the output itself. e4m3 and 4-bit pages: keys and values become fp16 exactly, the
// weights are scaled by 2^6 and rounded to fp16 (2^-11), and a head's query is scaled by a
// power of two to a largest element in [1, 2), so that fp16's ten fraction bits hold bf16's
// seven exactly over 2^14 of range and to 2^-24 of the largest element below that.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <type_traits>

#include "sr_device.cuh"
#include "sr_kernels.h"
#include "sr_paged.h"
#include "sr_paged_device.cuh"

namespace sr {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
// Two CTAs of three stages per warp fill an SM's shared memory with 128 KB of copies in flight; three
// CTAs of two stages have 96 KB and were slower (one sequence of 131071 tokens: 87 us, 100 us) or no faster.
constexpr float kLn2 = 0.69314718055994531f;

template <int D, int TYPE>
struct Geo {
  static constexpr bool kRecords = TYPE == SR_PAGE_INT4;
  static constexpr int kRowBytes = D * (TYPE == SR_PAGE_BF16 ? 2 : 1);   // a token's keys (or values) of one head
  static constexpr int kChunks = kRowBytes / 16;
  // tokens per warp and tile: 4 KB of keys, 4 KB of values; 64 tokens of records
  static constexpr int KT = kRecords ? 64 : 4096 / kRowBytes;
  // Records are bound by their decoding: more warps (rows of 64 values), fewer stages (two CTAs, 64 tokens, of 128 values: 3
  // stages 127.4 us for 32 sequences of 4001 .. 32768 tokens, 2 stages 125.6 us; 32 tokens, 5 stages 148.3 us).
  static constexpr int kCtasPerSm = kRecords && D == 64 ? 3 : 2;
  static constexpr int kStages = kRecords && D == 128 ? 2 : 3;
  static constexpr int CT = kWarps * KT;           // tokens per tile
  static constexpr int kGroups = KT / 16;          // 16-token groups: a group never crosses a page
  // Whether the warps take their tiles in step. Nothing in them depends on it, but warps that drift apart
  // read DRAM in shorter runs: 32 sequences of 4001 .. 32768 tokens, e4m3: 160 us without, 152 us in
  // step; 8 sessions, bf16: 152 us, 148 us. Rows of 64 bytes have more arithmetic than that gains
  // (64 sequences of 8192: 95 us, 98 us in step).
  static constexpr bool kInStep = kRowBytes > 64;
  // Stretches end where items end (so many whole items each, or an item in so many pieces), where the largest,
  // in units of the line, is not above kWhole / 16 of an even one or so many units more: fewer parts to join, and
  // none twice. The ratio: DRAM serves the CTAs that are left faster (even stretches, whole items: 32 sequences of
  // 4096 tokens, 1.19 times an even one, 85.3 us, 80.1 us; 32 of 3500 .. 4096, 1.27, 79.9 us, 77.9 us; 32 of
  // 3000 .. 4096, 1.36, 74.1 us, 75.4 us), but arithmetic does not get faster (64 of 8192, rows of 64 bytes,
  // 1.19: 93.2 us, 98.8 us). The units: a join costs as much as a few tiles. Where CTAs are left for pieces, these
  // are the better choice from kWholeExtra on (even, whole, pieces: 16 of 512, 5.8 units more: 11.5, 10.9, 11.0 us;
  // 16 of 640, 6.9: 12.9, 13.0, 12.2 us; rows of 64 bytes, 8 of 768, 3.9: 9.2, 8.2, 8.5 us; 16 of 1536, 4.6: 12.7,
  // 12.6, 11.4 us); where there are none, whole items are, up to kAloneExtra (24 of 1280, 8.1: 26.8, 24.9 us; rows of
  // 64 bytes, 24 of 2560, 4.4: 20.1, 19.0 us; 24 of 4096, 6.6: 25.7, 27.6 us). Where the rule tries pieces in vain the
  // trial costs 0.1 us.
  static constexpr int kWhole = kInStep ? 21 : 18;
  static constexpr int kWholeExtra = kInStep ? 6 : 4;
  static constexpr int kAloneExtra = kInStep ? 9 : 6;
  static constexpr int kHalfBytes = kRecords ? KT / 16 * record_bytes(D) : 4096;   // a stage's keys, or its values
  static constexpr int kStageBytes = 2 * kHalfBytes;
  static constexpr int kStageArea = kWarps * kStages * kStageBytes;
  // A warp's 8 rows of D sums while the warps merge, in its free stage: rows four floats apart in
  // banks beyond a multiple of 32, so that stores and loads spread over all of them.
  static constexpr int kMergeRow = D + 4;
  static_assert(8 * kMergeRow * 4 <= kStageBytes, "the merge does not fit a stage");
};

// Shared-memory position of 16-byte chunk c of row r, permuted so that eight rows'
// equal chunks (what one matrix load reads) lie in different banks.
template <int CHUNKS>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  if constexpr (CHUNKS >= 8) return static_cast<uint32_t>(r * CHUNKS + (c ^ (r & 7))) * 16u;
  return static_cast<uint32_t>(r * CHUNKS + (c ^ ((r >> 1) & 3))) * 16u;
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(policy) : "memory");
}
__device__ __forceinline__ void copy16_or_zero(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void store_hinted(float* dst, float x, uint64_t policy) {
  asm volatile("st.global.L2::cache_hint.f32 [%0], %1, %2;" ::"l"(dst), "f"(x), "l"(policy) : "memory");
}
// Drops 128 bytes from L2 without writing them to memory: they hold nothing until they are written again.
__device__ __forceinline__ void discard_line(const void* line) {
  asm volatile("discard.global.L2 [%0], 128;" ::"l"(line) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// transposes an 8x8 matrix of 16-bit elements spread over the warp
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <int TYPE>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if constexpr (TYPE == SR_PAGE_BF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ void copy_bulk(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar, uint64_t policy) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
               : "memory");
}
constexpr uint64_t kCopyTimeoutNs = 2000000000ull;

// N neighbouring words of shared memory
template <int N>
__device__ __forceinline__ void load_words(uint32_t (&r)[N], uint32_t addr) {
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr) : "memory");
  else
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r[0]) : "r"(addr) : "memory");
}
// Releases what this thread has seen written, and acquires what earlier such additions released.
__device__ __forceinline__ int32_t add_acq_rel(int32_t* p, int32_t x) {
  int32_t old;
  asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(x) : "memory");
  return old;
}

struct SharedHead {
  int64_t cum[kMaxPagedSeqs + 1];       // units before each sequence of the batch
  int32_t len[kMaxPagedSeqs];
  int32_t longest;                      // units of the longest item
  float ml[kWarps][8][2];               // each warp's maximum and sum of eight heads, while warps merge
  int last;                             // this CTA is the last of its item's to arrive
  int abort;                            // a copy never came: err_word tells, the outputs are void
  uint64_t full[kWarps][8];             // 4-bit pages: a stage's copies have landed
};

// A place on the line of tiles. Each item takes kItemCost units before its tiles:
// what changing items costs a CTA, in tiles (with 1, 2, 3: 16 sequences of 300 .. 3000 tokens of 64 13.9, 12.2,
// 12.9 us; 16 of 1000 .. 8192 with 40 heads 43.8, 42.2, 43.0 us; 32 of 100 .. 2000 21.3, 20.7, 22.1 us; slower: 64 of
// 1 .. 16384 80.3, 80.7, 80.6 us; 64 of 100 .. 600 20.5, 20.7, 20.9 us).
constexpr int kItemCost = kPagedItemCost;
// Up to kSpread neighbouring heads are read side by side by neighbouring CTAs, so that a
// token's row, whole in memory, is read at about one time. Rows of 64 bytes per head need
// it, because DRAM delivers twice that (8 heads, 64 sequences of 8192 tokens, head dim 64,
// e4m3: 178 us one by one, 127 us side by side); longer ones gain up to 10 %.
constexpr int kSpreadLog2 = 3, kSpread = 1 << kSpreadLog2;
struct Cursor {
  int i, h;            // sequence of the batch, key/value head
  int32_t tile, tiles; // tile of the item, tiles it has
  int32_t len;
};

template <int CT>
__device__ __forceinline__ int64_t seq_units(int32_t len, int n_kv) {
  return len > 0 ? static_cast<int64_t>((len + CT - 1) / CT + kItemCost) * n_kv : 0;
}
template <int CT>
__device__ __forceinline__ void cursor_seq(Cursor& c, const SharedHead& s) {
  while (s.len[c.i] == 0) ++c.i;        // the line holds a tile here: some sequence has one
  c.len = s.len[c.i];
  c.tiles = (c.len + CT - 1) / CT;
}
template <int CT>
__device__ __forceinline__ void cursor_next(Cursor& c, const SharedHead& s, int n_kv, int32_t& left) {
  // left: units of this CTA's stretch from the cursor's tile on
  --left;
  if (++c.tile < c.tiles) return;
  c.tile = 0;
  left -= kItemCost;
  if (left <= 0 || ++c.h < n_kv) return;
  c.h = 0;
  ++c.i;
  cursor_seq<CT>(c, s);
}

__device__ __forceinline__ int64_t div_pos(int64_t a, int64_t b) {   // a >= 0, b > 0; mostly short numbers
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// What the weights' launch subtracts from a row's scores: where all of them are -inf, 0 leaves weights of 0, as in the
// output, and -inf would leave NaN.
__device__ __forceinline__ float weight_reference(float lse2) { return lse2 == -INFINITY ? 0.f : lse2; }

// ---- joining partial results
constexpr int kJoin = 48;

// What a launch does beyond the outputs of one new token per sequence.
constexpr int kPlain = 0, kMass = 1, kRows = 2;      // nothing; the tokens' weights; a few new tokens per sequence
template <int MODE>
using Params = std::conditional_t<MODE == kRows, PagedRowsParams, PagedAttnParams>;
// Columns of the products: the heads of the item's group, or those of each of the sequence's new tokens.
template <int MODE>
__device__ __forceinline__ int columns_of(const Params<MODE>& p, int i) {
  if constexpr (MODE == kRows) return (p.row0[i + 1] - p.row0[i]) * p.c.group;
  return p.c.group;
}
// The output (or query) row of column r of sequence i and item head h.
template <int MODE>
__device__ __forceinline__ int64_t row_of(const Params<MODE>& p, int i, int h, int r) {
  if constexpr (MODE == kRows) {
    const int j = static_cast<int>(static_cast<uint32_t>(r) * p.group_magic >> 16);
    return static_cast<int64_t>(p.row0[i] + j) * p.c.n_heads + h * p.c.group + (r - j * p.c.group);
  }
  return static_cast<int64_t>(i) * p.c.n_heads + h * p.c.group + r;
}

// Partial result of a CTA: slot 0 for an item that began before its stretch, 1 for one
// that begins in it. [group][D] sums, then (maximum, sum) per row.
__host__ __device__ __forceinline__ int64_t part_floats(int group, int D) { return (group * (D + 2) + 3) / 4 * 4; }
template <int D>
__device__ __forceinline__ float* part_at(const PagedAttnParams& p, int cta, int slot) {
  return p.parts + (static_cast<int64_t>(cta) * 2 + slot) * part_floats(p.part_rows, D);
}

// Joins n parts: the one at first, slot s0, and those of every step-th CTA after it, slot
// 0. The result is another part (dst) or the output. Each warp takes query rows, its lanes
// the head dimension; sixteen parts at a time, all their loads in flight together.
constexpr int kJoinBatch = 16;
template <int D, int MODE>
__device__ __noinline__ void join_parts(const Params<MODE>& p, int first, int s0, int step, int n, float* dst, int item_i,
                                        int item_h, int warp, int lane) {
  constexpr int kCols = D / 32;
  const int ml = p.part_rows * D, columns = columns_of<MODE>(p, item_i);
  for (int r = warp; r < columns; r += kWarps) {
    float top = -INFINITY, sum = 0.f, a[kCols];
#pragma unroll
    for (int x = 0; x < kCols; ++x) a[x] = 0.f;
#pragma unroll 1
    for (int k0 = 0; k0 < n; k0 += kJoinBatch) {
      float v[kJoinBatch][kCols];
#pragma unroll
      for (int k = 0; k < kJoinBatch; ++k) {
        const int kk = min(k0 + k, n - 1);     // one past the end repeats the last, with no weight
        const float* src = part_at<D>(p, first + kk * step, kk == 0 ? s0 : 0) + r * D + lane * kCols;
        if constexpr (kCols == 4) {
          const float4 x = __ldcg(reinterpret_cast<const float4*>(src));
          v[k][0] = x.x; v[k][1] = x.y; v[k][2] = x.z; v[k][3] = x.w;
        } else {
          const float2 x = __ldcg(reinterpret_cast<const float2*>(src));
          v[k][0] = x.x; v[k][1] = x.y;
        }
      }
      float mk = -INFINITY, lk = 0.f;
      if (lane < kJoinBatch && k0 + lane < n) {
        const float2 x = __ldcg(reinterpret_cast<const float2*>(
                                    part_at<D>(p, first + (k0 + lane) * step, k0 + lane == 0 ? s0 : 0) + ml) + r);
        mk = x.x;
        lk = x.y;
      }
      float t = mk;
#pragma unroll
      for (int s = 8; s > 0; s >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, s));
      t = fmaxf(__shfl_sync(0xffffffffu, t, 0), top);
      // a first batch has nothing to rescale; a maximum of -inf stands for no token, or NaN alone
      const float f = top == -INFINITY ? 1.f : ex2_approx(top - t);
      const float w = mk == -INFINITY ? 0.f : ex2_approx(mk - t);
      top = t;
      float s1 = w * lk;
#pragma unroll
      for (int s = 8; s > 0; s >>= 1) s1 += __shfl_xor_sync(0xffffffffu, s1, s);
      sum = sum * f + __shfl_sync(0xffffffffu, s1, 0);
#pragma unroll
      for (int x = 0; x < kCols; ++x) a[x] *= f;
#pragma unroll
      for (int k = 0; k < kJoinBatch; ++k) {
        const float wk = __shfl_sync(0xffffffffu, w, k);
        if (k0 + k < n)
#pragma unroll
          for (int x = 0; x < kCols; ++x) a[x] = fmaf(wk, v[k][x], a[x]);
      }
    }
    if (dst) {
      // in place over its own first part: this warp alone reads and writes row r
#pragma unroll
      for (int x = 0; x < kCols; ++x) dst[r * D + lane * kCols + x] = a[x];
      if (lane == 0) reinterpret_cast<float2*>(dst + ml)[r] = make_float2(top, sum);
    } else {
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const int64_t out = row_of<MODE>(p, item_i, item_h, r);
      uint32_t* o = reinterpret_cast<uint32_t*>(p.o + out * D + lane * kCols);
      auto of = [&](int x) { return sum == 0.f ? 0.f : a[x] * inv; };      // no weight: 0, whatever the values are
      o[0] = pack_bf16x2(of(0), of(1));
      if constexpr (kCols == 4) o[1] = pack_bf16x2(of(2), of(3));
      if (lane == 0) {
        const float lse2 = sum == 0.f ? -INFINITY : top + log2f(sum);
        if (p.lse) p.lse[out] = lse2 * kLn2;
        if constexpr (MODE != kRows) p.lse2[out] = weight_reference(lse2);
      }
    }
  }
}

// ---- values that are no finite numbers, among new tokens that some columns do not see (a weight of zero times such a value
// is none either): they leave the stage before the products, and are added to the columns that do see them.
// Takes them out of rows first .. last - 1 of a warp's values; a bit for each row (of at most 32) that had some.
template <int D, int TYPE>
__device__ __noinline__ uint32_t take_odd(uint32_t vs, int first, int last, int lane) {
  using G = Geo<D, TYPE>;
  uint32_t odd = 0;
#pragma unroll 1
  for (int r = first; r < last; ++r) {
    bool any = false;
    if constexpr (G::kRecords) {
      if (lane < D / 16) {
        const uint32_t at = vs + r / 16 * record_bytes(D) + 8 * D + r % 16 * (D / 16) + lane;
        uint32_t b;
        asm volatile("ld.shared.u8 %0, [%1];" : "=r"(b) : "r"(at) : "memory");
        any = b == 255;
        if (any) asm volatile("st.shared.u8 [%0], %1;" ::"r"(at), "r"(0) : "memory");
      }
    } else if (lane < G::kChunks) {
      const uint32_t at = vs + chunk_at<G::kChunks>(r, lane);
      uint32_t x[4];
      load_words(x, at);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < (TYPE == SR_PAGE_BF16 ? 2 : 4); ++k) {
          const uint32_t mask = TYPE == SR_PAGE_BF16 ? 0x7F80u << (16 * k) : 0x7Fu << (8 * k);
          if ((x[i] & mask) == mask) {
            any = true;
            x[i] &= ~((TYPE == SR_PAGE_BF16 ? 0xFFFFu : 0xFFu) << ((TYPE == SR_PAGE_BF16 ? 16 : 8) * k));
          }
        }
      if (any) asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]) : "memory");
    }
    if (__any_sync(0xffffffffu, any)) odd |= 1u << (r - first);
  }
  if constexpr (G::kRecords) fence_proxy_async_smem();
  __syncwarp();
  return odd;
}
// The weight of token t for query row `row`, computed again: 2^(scale * q . k - m).
template <int D, int TYPE>
__device__ __noinline__ float weight_again(const PagedRowsParams& p, int32_t seq, int32_t t, int head, int64_t row, float scale, float m) {
  float x = 0.f;
  for (int d = 0; d < D; ++d)
    x = fmaf(__bfloat162float(p.q[row * D + d]), page_value<D, TYPE>(p.c, p.kv_heads, p.c.k_pages, seq, t, head, d), x);
  return ex2_approx(x * scale - (m == -INFINITY ? 0.f : m));
}

template <int D, int TYPE, int NT, int MODE>
__global__ void __launch_bounds__(kThreads, Geo<D, TYPE>::kCtasPerSm) paged_attn_kernel(const __grid_constant__ Params<MODE> p) {
  using G = Geo<D, TYPE>;
  constexpr bool MASS = MODE == kMass;
  constexpr int kStages = G::kStages;
  static_assert(kStages <= 8, "more stages than barriers");
  extern __shared__ __align__(128) uint8_t smem[];
  SharedHead& sh = *reinterpret_cast<SharedHead*>(smem + G::kStageArea);
  grid_dep_launch_dependents();
  const PagedView& c = p.c;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int n = p.b.n, group = c.group;
  // this lane's sequences, read from the parameters ahead of the wait (32 addresses of them at a
  // time are slow: 256 sequences of 16 tokens 18.3 us behind it, 16.9 us so)
  int32_t id[kMaxPagedSeqs / 32];
  if (warp == 0) {
#pragma unroll
    for (int k = 0; k < kMaxPagedSeqs / 32; ++k) {
      id[k] = p.b.id[lane * (kMaxPagedSeqs / 32) + k];
      asm volatile("" : "+r"(id[k]));
    }
  }
  const WaitCtx wc{&sh.abort, c.err_word, kCopyTimeoutNs};
  if constexpr (G::kRecords) {          // the first barrier below makes them visible
    if (threadIdx.x == 0) sh.abort = 0;
    if (lane < kStages) mbar_init(&sh.full[warp][lane], 1);
    mbar_fence_init();
  }
  grid_dep_wait();
  // S neighbouring CTAs take the same stretch for S neighbouring key/value heads
  const int S = p.spread, sub = static_cast<int>(blockIdx.x) & (S - 1), me = static_cast<int>(blockIdx.x) >> p.spread_log2;
  const int n_kv = c.n_kv >> p.spread_log2;        // heads on the line

  // ---- the line of tiles
  if (warp == 0) {
    int64_t mine = 0;
    int32_t len[kMaxPagedSeqs / 32];
#pragma unroll
    for (int k = 0; k < kMaxPagedSeqs / 32; ++k) {
      const int i = lane * (kMaxPagedSeqs / 32) + k;
      len[k] = i < n ? min(max(c.seq_len[id[k]], 0), c.cap) : 0;
      if constexpr (MODE == kRows)
        if (i < n && p.row0[i + 1] == p.row0[i]) len[k] = 0;      // nothing asked of it
      mine += seq_units<G::CT>(len[k], n_kv);
    }
    int64_t incl = mine;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, incl, s);
      if (lane >= s) incl += y;
    }
    int64_t at = incl - mine;
#pragma unroll
    for (int k = 0; k < kMaxPagedSeqs / 32; ++k) {
      const int i = lane * (kMaxPagedSeqs / 32) + k;
      sh.len[i] = len[k];
      sh.cum[i] = at;
      at += seq_units<G::CT>(len[k], n_kv);
    }
    if (lane == 31) sh.cum[kMaxPagedSeqs] = at;
    int32_t longest = len[0];
#pragma unroll
    for (int k = 1; k < kMaxPagedSeqs / 32; ++k) longest = max(longest, len[k]);
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (lane == 0) sh.longest = (longest + G::CT - 1) / G::CT + kItemCost;
  }
  __syncthreads();
  // sequences without a token: nothing to attend to
  for (int i = blockIdx.x; i < n; i += gridDim.x)
    if (sh.len[i] == 0) {
      int64_t row = i, rows = 1;
      if constexpr (MODE == kRows) {
        row = p.row0[i];
        rows = p.row0[i + 1] - row;
      }
      for (int x = threadIdx.x; x < rows * c.n_heads * (D / 8); x += kThreads)
        reinterpret_cast<uint4*>(p.o + row * c.n_heads * D)[x] = make_uint4(0, 0, 0, 0);
      for (int h = threadIdx.x; h < rows * c.n_heads; h += kThreads)
        if (p.lse) p.lse[row * c.n_heads + h] = -INFINITY;
      if (p.items)
        for (int h = threadIdx.x; h < c.n_kv; h += kThreads) p.items[i * c.n_kv + h] = make_int2(0, 1);
    }
  const int64_t T = sh.cum[n];
  if (MASS && blockIdx.x == 0)
    for (int i = threadIdx.x; i <= n; i += kThreads) p.unit0[i] = sh.cum[i];
  if (T == 0) return;
  int64_t u0, left64, share = 0, rest = 0;   // first unit and units of the stretch
  int cut = 0;                             // pieces of each item of the stretch, where all have as many
  const int64_t bound = max(T * G::kWhole, T * 16 + p.whole_extra);
  if (sh.longest * p.whole_cost <= bound) {
    // whole items; left64 == 0: none but empty ones
    auto start = [&](int item) {
      const int i = item / n_kv;
      return i < n ? sh.cum[i] + (item - i * n_kv) * seq_units<G::CT>(sh.len[i], 1) : T;
    };
    u0 = start(me * p.each);
    left64 = start((me + 1) * p.each) - u0;
    if (left64 == 0) return;
  } else if (p.pieces > 1 && (sh.longest + 2 * p.pieces) * p.cut_cost <= bound) {
    // one of `pieces` equal pieces of an item, as far as it has tiles
    const int item = me / p.pieces, i = item / n_kv;
    if (i >= n) return;
    const int32_t tiles = (sh.len[i] + G::CT - 1) / G::CT;
    cut = min(p.pieces, tiles);
    const int x = me - item * p.pieces;
    if (x >= cut) return;
    const int32_t t0 = x * tiles / cut;
    u0 = sh.cum[i] + (item - i * n_kv) * static_cast<int64_t>(tiles + kItemCost) + kItemCost + t0;
    left64 = (x + 1) * tiles / cut - t0;
  } else {
    // CTAs that work: each gets one unit at least, so that all between an item's first and last have a part of it
    const int64_t ctas = min(static_cast<int64_t>(gridDim.x >> p.spread_log2), T);
    if (me >= ctas) return;
    // equal stretches, the first `rest` one unit longer
    share = div_pos(T, ctas);
    rest = T - share * ctas;
    u0 = me * share + min(static_cast<int64_t>(me), rest);
    left64 = share + (me < rest ? 1 : 0);
  }
  Cursor comp;
  {
    int lo = 0, hi = n - 1;   // the last sequence that starts at or before u0
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (sh.cum[mid] <= u0) lo = mid; else hi = mid - 1;
    }
    comp.i = lo;
    cursor_seq<G::CT>(comp, sh);
    const int64_t within = u0 - sh.cum[comp.i];
    const int32_t units = comp.tiles + kItemCost;
    comp.h = static_cast<int>(div_pos(within, units));
    const int32_t unit = static_cast<int32_t>(within - static_cast<int64_t>(comp.h) * units);
    comp.tile = max(unit - kItemCost, 0);
    left64 -= max(kItemCost - unit, 0);
  }
  // of at most 2^36 units (256 sequences of 2^24 tokens, 1024 heads) a CTA's stretch has fewer than 2^31
  int32_t left = static_cast<int32_t>(left64);
  if (left <= 0) return;    // nothing but the units before an item
  Cursor load = comp;
  int32_t left_load = left;
  const uint32_t stage0 = smem_u32(smem) + warp * kStages * G::kStageBytes;
  uint32_t bad = 0;       // bit stage * kGroups + group: the group's page is none of the pool's
  const int64_t row_pitch = static_cast<int64_t>(p.kv_heads) * G::kRowBytes;
  auto kv_head = [&](int h) { return static_cast<int>(static_cast<uint32_t>(h) * p.head_magic >> 22); };

  // ---- copy this warp's tokens of one tile into a stage. The block table's entries for the
  // tile after it are fetched on the way, so that no copy waits for them. The lines are marked to
  // leave L2 first: a stream larger than L2 would push out the scores that the second launch
  // reads, and what a smaller one leaves there stays all the same (16 sequences of 1000 .. 8192
  // tokens with weights: 57.0 us without the mark, 53.5 us with it; 32 of 4096: 86.6 us, 85.4 us).
  constexpr int kRowsPer = 32 / G::kChunks;     // rows per instruction
  const int r0 = lane / G::kChunks, ch = lane % G::kChunks;
  const int64_t lane_off = r0 * row_pitch + ch * 16;
  const uint64_t policy = l2_policy_evict_first();
  [[maybe_unused]] uint64_t keep;      // for the scores
  if constexpr (MASS) keep = p.drop_scores ? l2_policy_evict_last() : l2_policy_evict_normal();
  int32_t page[G::kGroups];
  // Records: lane g fetches and copies group g's keys, lane kGroups + g its values.
  const int my_group = lane % G::kGroups, my_half = lane / G::kGroups;
  [[maybe_unused]] const int32_t page_records = p.kv_heads * (c.page_tokens >> 4);
  [[maybe_unused]] uint32_t phases = 0;           // bit of a stage: the parity its copies complete next
  auto fetch_pages = [&] {
    if constexpr (G::kRecords) {
      const int32_t tok = load.tile * G::CT + warp * G::KT + my_group * 16;
      page[0] = my_half < 2 && tok < load.len
                    ? c.table[static_cast<int64_t>(p.b.id[load.i]) * c.max_pages + page_of_group(tok >> 4, c.magic)] : -1;
      return;
    }
    const int32_t* table = c.table + static_cast<int64_t>(p.b.id[load.i]) * c.max_pages;
#pragma unroll
    for (int g = 0; g < G::kGroups; ++g) {
      const int32_t tok = load.tile * G::CT + warp * G::KT + g * 16;
      if (tok < load.len) page[g] = table[page_of_group(tok >> 4, c.magic)];
    }
  };
  fetch_pages();
  auto issue_records = [&](int stage) {
    if (left_load <= 0) return;
    const int32_t tok = load.tile * G::CT + warp * G::KT + my_group * 16;
    const bool held = my_half < 2 && tok < load.len, good = held && page[0] >= 0 && page[0] < c.n_pages;
    const uint32_t ready = __ballot_sync(0xffffffffu, good), all = __ballot_sync(0xffffffffu, held);
    constexpr uint32_t kMask = (1u << G::kGroups) - 1u;
    bad = (bad & ~(kMask << (stage * G::kGroups))) | ((all & ~ready & kMask) << (stage * G::kGroups));
    uint64_t* bar = &sh.full[warp][stage];
    if (lane == 0) {
      if (all & ~ready) atomicCAS(c.err_word, 0, SR_DEVERR_BAD_PAGE);
      mbar_arrive_expect_tx(bar, __popc(ready) * record_bytes(D));
    }
    __syncwarp();
    if (good) {
      // records before this one: of the pages before, of the heads before, of the page
      const int32_t in_page = (tok >> 4) - page_of_group(tok >> 4, c.magic) * (c.page_tokens >> 4);
      const int64_t at = (static_cast<int64_t>(page[0]) * page_records + kv_head(load.h * S + sub) * (c.page_tokens >> 4) + in_page) *
                         record_bytes(D);
      copy_bulk(stage0 + stage * G::kStageBytes + my_half * G::kHalfBytes + my_group * record_bytes(D),
                static_cast<const char*>(my_half == 0 ? c.k_pages : c.v_pages) + at, record_bytes(D), bar, policy);
    }
    cursor_next<G::CT>(load, sh, n_kv, left_load);
    if (left_load > 0) fetch_pages();
  };
  auto issue = [&](int stage) {
    if constexpr (G::kRecords) {
      issue_records(stage);
      return;
    }
    if (left_load > 0) {
      const uint32_t ks = stage0 + stage * G::kStageBytes, vs = ks + G::kHalfBytes;
#pragma unroll
      for (int g = 0; g < G::kGroups; ++g) {
        const int32_t tok = load.tile * G::CT + warp * G::KT + g * 16;
        int32_t live = load.len - tok;
        int64_t row = 0;
        if (live > 0) {
          const uint32_t bit = 1u << (stage * G::kGroups + g);
          bad &= ~bit;
          if (page[g] >= 0 && page[g] < c.n_pages) {
            row = static_cast<int64_t>(page[g]) * c.page_tokens + (tok - page_of_group(tok >> 4, c.magic) * c.page_tokens);
          } else {
            if (lane == 0) atomicCAS(c.err_word, 0, SR_DEVERR_BAD_PAGE);
            bad |= bit;
            live = 0;
          }
        }
        int64_t at = row * row_pitch + lane_off + kv_head(load.h * S + sub) * G::kRowBytes;
        if (live >= 16) {
#pragma unroll
          for (int x = 0; x < 16 / kRowsPer; ++x, at += kRowsPer * row_pitch) {
            const uint32_t to = chunk_at<G::kChunks>(g * 16 + x * kRowsPer + r0, ch);
            copy16(ks + to, static_cast<const char*>(c.k_pages) + at, policy);
            copy16(vs + to, static_cast<const char*>(c.v_pages) + at, policy);
          }
        } else {
#pragma unroll
          for (int x = 0; x < 16 / kRowsPer; ++x, at += kRowsPer * row_pitch) {
            const int r = x * kRowsPer + r0;
            const uint32_t to = chunk_at<G::kChunks>(g * 16 + r, ch);
            const int64_t from = r < live ? at : 0;       // past the length: zeros, nothing read
            copy16_or_zero(ks + to, static_cast<const char*>(c.k_pages) + from, r < live);
            copy16_or_zero(vs + to, static_cast<const char*>(c.v_pages) + from, r < live);
          }
        }
      }
      cursor_next<G::CT>(load, sh, n_kv, left_load);
      if (left_load > 0) fetch_pages();
    }
    copy_commit();
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) issue(s);

  // 4 bits: products with 128 instead of shifts, since the pipe that shifts also masks and permutes, and is the one that
  // bounds this kernel
  [[maybe_unused]] uint32_t shift7;
  asm volatile("mov.u32 %0, 128;" : "=r"(shift7));
  [[maybe_unused]] const DecodeMasks masks = decode_masks();
  // ---- the items of this stretch, one after the other
  int stage = 0;
  const int j4 = lane % 4, r8 = lane / 4;
  // The group's queries as right operands, [head tile][16 dims]. Those of the next item are
  // fetched before the current one's results are merged, so that their latency hides behind that.
  uint32_t qb[NT][D / 16][2];
  auto fetch_q = [&](int i, int h) {
    const int columns = columns_of<MODE>(p, i);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = 8 * t + r8;
      const __nv_bfloat16* qp = p.q + row_of<MODE>(p, i, h * S + sub, min(r, columns - 1)) * D;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        if constexpr (TYPE == SR_PAGE_BF16) {
#pragma unroll
          for (int x = 0; x < 2; ++x)
            qb[t][kk][x] = r < columns ? *reinterpret_cast<const uint32_t*>(qp + kk * 16 + 8 * x + 2 * j4) : 0u;
        } else if constexpr (TYPE == SR_PAGE_INT4) {
          // pairs as the decoding of a word of keys leaves them: values i and i + 4 of its eight
          if (kk % 2 == 0) {
            const uint4 raw = r < columns ? *reinterpret_cast<const uint4*>(qp + kk * 16 + 8 * j4) : make_uint4(0u, 0u, 0u, 0u);
            qb[t][kk][0] = __byte_perm(raw.x, raw.z, 0x5410);
            qb[t][kk][1] = __byte_perm(raw.x, raw.z, 0x7632);
            qb[t][kk + 1][0] = __byte_perm(raw.y, raw.w, 0x5410);
            qb[t][kk + 1][1] = __byte_perm(raw.y, raw.w, 0x7632);
          }
        } else {
          // the order of the dims in which a 16-byte row of keys arrives: four neighbours per lane
          const uint2 raw = r < columns ? *reinterpret_cast<const uint2*>(qp + kk * 16 + 4 * j4) : make_uint2(0u, 0u);
          qb[t][kk][0] = raw.x;
          qb[t][kk][1] = raw.y;
        }
      }
    }
  };
  fetch_q(comp.i, comp.h);
  while (left > 0) {
    const int item_i = comp.i, comp_h = comp.h, item_h = comp_h * S + sub;
    const int32_t first_tile = comp.tile, tiles = comp.tiles;
    const int32_t end_tile = min(tiles, first_tile + left);
    const int32_t len = comp.len;
    [[maybe_unused]] int32_t seen_by_all = 0;      // tokens that the first new one sees
    if constexpr (MODE == kRows) seen_by_all = len - (p.row0[item_i + 1] - p.row0[item_i]) + 1;
    const int columns = columns_of<MODE>(p, item_i);
    const int64_t item_u = sh.cum[item_i] + static_cast<int64_t>(comp.h) * (tiles + kItemCost) + kItemCost;   // its first tile
    // log2-scaled scores = product * xs, of this lane's heads 8 t + 2 j4 and the next
    float xs[NT][2];
    {
      const float scale = c.scale_log2 * (G::kRecords ? kDecoded : 1.f) *
                          (c.kv_exp ? exp2f(static_cast<float>(c.kv_exp[kv_head(item_h)])) : 1.f);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float x = scale;
        if constexpr (TYPE != SR_PAGE_BF16) {
          // queries to fp16, scaled by a power of two to a largest element in [1, 2)
          auto pair = [](uint32_t y) { return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&y)); };
          float top = 0.f;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const float2 a = pair(qb[t][kk][0]), b = pair(qb[t][kk][1]);
            top = fmaxf(fmaxf(top, fmaxf(fabsf(a.x), fabsf(a.y))), fmaxf(fabsf(b.x), fabsf(b.y)));
          }
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const int e = top > 0.f && top < INFINITY ? max(ilogbf(top), -120) : 0;
          const float down = ldexpf(1.f, -e);
          x *= ldexpf(1.f, e);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const float2 a = pair(qb[t][kk][0]), b = pair(qb[t][kk][1]);
            qb[t][kk][0] = pack_half2(a.x * down, a.y * down);
            qb[t][kk][1] = pack_half2(b.x * down, b.y * down);
          }
        }
        // a scale so small that it underflows: the scores are zero as well as with this one, and masked ones stay -inf
        x = fmaxf(x, 0x1p-126f);
        xs[t][0] = __shfl_sync(0xffffffffu, x, 8 * j4);       // lanes of head 2 j4, then of the next
        xs[t][1] = __shfl_sync(0xffffffffu, x, 8 * j4 + 4);
      }
    }
    // o: [head tile][16 dims]: rows are dims, columns heads. m: the reference of the exponentials, an
    // earlier maximum less kLift, raised only when a score passes it by 2^kSlack, so that most
    // tiles need no maximum across lanes; l: this lane's share of the weights' sum. Weights reach
    // 2^8 (bf16), 2^14 (fp16), and what rounds to fp16's smallest is 2^-30 of the largest or less.
    constexpr float kLess = 1.f - 0x1p-8f;
    constexpr float kLift = TYPE == SR_PAGE_BF16 ? 0.f : 6.f, kSlack = 8.f;
    float o[NT][D / 16][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[t][k][x] = 0.f;
      m[t][0] = m[t][1] = -INFINITY;
      l[t][0] = l[t][1] = 0.f;
    }

    for (int32_t tile = first_tile; tile < end_tile; ++tile) {
      issue((stage + kStages - 1) % kStages);
      if constexpr (G::kRecords) {
        if (!__all_sync(0xffffffffu, wait_bounded(&sh.full[warp][stage], phases >> stage & 1u, wc, 0x21))) {
          // A copy did not come in time: the outputs are void (err_word tells), and this warp leaves. Its shared memory is
          // not given back before the copies of this tile and those ahead have come, or have had their time once more.
          for (int x = 0; x < kStages && left > 0; ++x) {
            const int s = (stage + x) % kStages;
            wait_drain(&sh.full[warp][s], phases >> s & 1u, kCopyTimeoutNs);
            cursor_next<G::CT>(comp, sh, n_kv, left);
          }
          return;
        }
        phases ^= 1u << stage;
      } else {
        copy_wait<kStages - 1>();
      }
      if constexpr (G::kInStep)
        __syncthreads();
      else
        __syncwarp();
      const uint32_t ks = stage0 + stage * G::kStageBytes, vs = ks + G::kHalfBytes;
      const int32_t tok = tile * G::CT + warp * G::KT;
      int32_t live[G::kGroups], any = 0;
#pragma unroll
      for (int g = 0; g < G::kGroups; ++g) {
        live[g] = (bad >> (stage * G::kGroups + g)) & 1u ? 0 : min(max(len - tok - g * 16, 0), 16);
        any += live[g];
      }
      // where this lane's scores go for the second launch: [head][tokens of the tile]
      [[maybe_unused]] float* score = nullptr;
      if constexpr (MASS)
        if ((item_u + tile) * S + sub < p.score_tiles)
          score = p.scores + (((item_u + tile) * S + sub) * group + 2 * j4) * G::CT + warp * G::KT + r8;
      if (any) {
        // scores: rows are keys, columns heads. Two accumulators each, so that no product waits for the
        // one before it; groups inside steps for the same reason.
        float s[G::kGroups][NT][4], s2[G::kGroups][NT][4];
#pragma unroll
        for (int g = 0; g < G::kGroups; ++g)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int x = 0; x < 4; ++x) s[g][t][x] = s2[g][t][x] = 0.f;
        // lane -> (key, chunk) of the four matrices of 8 keys x 16 bytes that one load brings
        const int kr = (lane % 8) + 8 * ((lane / 8) % 2), kc = lane / 16;
        if constexpr (TYPE == SR_PAGE_BF16) {
#pragma unroll
          for (int kk = 0; kk < D / 16; kk += 2)
#pragma unroll
            for (int g = 0; g < G::kGroups; ++g) {
              uint32_t a[4], b[4];
              ldsm4(a, ks + chunk_at<G::kChunks>(g * 16 + kr, 2 * kk + kc));
              ldsm4(b, ks + chunk_at<G::kChunks>(g * 16 + kr, 2 * kk + 2 + kc));
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                mma16816<TYPE>(s[g][t], a[0], a[1], a[2], a[3], qb[t][kk][0], qb[t][kk][1]);
                mma16816<TYPE>(s2[g][t], b[0], b[1], b[2], b[3], qb[t][kk + 1][0], qb[t][kk + 1][1]);
              }
            }
        } else if constexpr (TYPE == SR_PAGE_INT4) {
          // a word is eight neighbouring dims of one key: two steps of four. Its scale: of keys r8 and r8 + 8, the
          // first or the second block of the chunk's two.
          const uint32_t pick = 0x4040u | (j4 >> 1) * 0x0101u;
#pragma unroll
          for (int g = 0; g < G::kGroups; ++g) {
            const uint32_t rec = ks + g * record_bytes(D);
            uint32_t sc[2][D / 64];
#pragma unroll
            for (int x = 0; x < 2; ++x) load_words(sc[x], rec + 8 * D + (r8 + 8 * x) * (D / 16));
#pragma unroll
            for (int ch = 0; ch < D / 32; ch += 2) {
              uint32_t a[4];
              ldsm4(a, rec + ch * 256 + lane * 16);
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                uint32_t lo[4], hi[4];
                decode_word(lo, a[2 * y], scale_pair(__byte_perm(sc[0][ch / 2], 0, pick + y * 0x0202u) * shift7), masks);
                decode_word(hi, a[2 * y + 1], scale_pair(__byte_perm(sc[1][ch / 2], 0, pick + y * 0x0202u) * shift7), masks);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                  mma16816<TYPE>(s[g][t], lo[0], hi[0], lo[1], hi[1], qb[t][2 * (ch + y)][0], qb[t][2 * (ch + y)][1]);
                  mma16816<TYPE>(s2[g][t], lo[2], hi[2], lo[3], hi[3], qb[t][2 * (ch + y) + 1][0], qb[t][2 * (ch + y) + 1][1]);
                }
              }
            }
          }
        } else {
#pragma unroll
          for (int kk = 0; kk < D / 16; kk += 2)
#pragma unroll
            for (int g = 0; g < G::kGroups; ++g) {
              uint32_t a[4];
              ldsm4(a, ks + chunk_at<G::kChunks>(g * 16 + kr, kk + kc));
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const uint32_t lo0 = half2_of_e4m3(a[2 * x]), lo1 = half2_of_e4m3(a[2 * x + 1]);
                const uint32_t hi0 = half2_of_e4m3(a[2 * x] >> 16), hi1 = half2_of_e4m3(a[2 * x + 1] >> 16);
#pragma unroll
                for (int t = 0; t < NT; ++t)
                  mma16816<TYPE>(x ? s2[g][t] : s[g][t], lo0, lo1, hi0, hi1, qb[t][kk + x][0], qb[t][kk + x][1]);
              }
            }
        }
#pragma unroll
        for (int g = 0; g < G::kGroups; ++g)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int x = 0; x < 4; ++x) s[g][t][x] += s2[g][t][x];
        // a few new tokens: those of them that a column does not see
        if constexpr (MODE == kRows) {
          if (p.causal && tok + G::KT > seen_by_all) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const int col = 8 * t + 2 * j4 + x, j = static_cast<int>(static_cast<uint32_t>(col) * p.group_magic >> 16);
                const int left_here = seen_by_all + j - tok;       // tokens of the warp's that the column sees
#pragma unroll
                for (int g = 0; g < G::kGroups; ++g)
#pragma unroll
                  for (int y = 0; y < 2; ++y)
                    if (g * 16 + r8 + 8 * y >= left_here) s[g][t][x + 2 * y] = -INFINITY;
              }
          }
        }
        if (any != 16 * G::kGroups) {                 // keys past the length, or without a page
#pragma unroll
          for (int g = 0; g < G::kGroups; ++g)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int x = 0; x < 4; ++x)
                if (r8 + 8 * (x / 2) >= live[g]) s[g][t][x] = -INFINITY;
        }
        bool raise = false;
        float top[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float y = fmaxf(s[0][t][x], s[0][t][x + 2]);
#pragma unroll
            for (int g = 1; g < G::kGroups; ++g) y = fmax3(y, s[g][t][x], s[g][t][x + 2]);
            top[t][x] = y * xs[t][x] - kLift;      // of this lane's keys; xs > 0
            raise |= top[t][x] > m[t][x] + kSlack;
          }
        if constexpr (MASS) {
          if (score) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int x = 0; x < 4; ++x)
                if (8 * t + 2 * j4 + x % 2 < group)
#pragma unroll
                  for (int g = 0; g < G::kGroups; ++g)
                    store_hinted(score + (8 * t + x % 2) * G::CT + g * 16 + 8 * (x / 2), s[g][t][x] * xs[t][x % 2], keep);
          }
        }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            float f[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
              for (int k = 4; k < 32; k *= 2) top[t][x] = fmaxf(top[t][x], __shfl_xor_sync(0xffffffffu, top[t][x], k));
              const float m1 = fmaxf(m[t][x], top[t][x]);
              f[x] = m[t][x] == -INFINITY ? 0.f : ex2_approx(m[t][x] - m1);
              m[t][x] = m1;
              l[t][x] *= f[x];
            }
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
#pragma unroll
              for (int x = 0; x < 4; ++x) o[t][k][x] *= f[x % 2];
          }
        }
        // the weights as right operands; bf16: as two numbers, the first rounded from a little less
        // than the weight, so that the second is positive as well and an infinite value stays infinite
        uint32_t w[G::kGroups][NT][2];
        [[maybe_unused]] uint32_t w_low[G::kGroups][NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float n0 = m[t][0] == -INFINITY ? 0.f : -m[t][0], n1 = m[t][1] == -INFINITY ? 0.f : -m[t][1];
#pragma unroll
          for (int g = 0; g < G::kGroups; ++g) {
            float e[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              e[x] = ex2_approx(fmaf(s[g][t][x], xs[t][x % 2], x % 2 ? n1 : n0));
              l[t][x % 2] += e[x];
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              if constexpr (TYPE == SR_PAGE_BF16) {
                const uint32_t hi = pack_bf16x2(e[2 * x] * kLess, e[2 * x + 1] * kLess);
                w[g][t][x] = transpose8x8(hi);
                w_low[g][t][x] = transpose8x8(pack_bf16x2(e[2 * x] - __uint_as_float(hi << 16),
                                                          e[2 * x + 1] - __uint_as_float(hi & 0xFFFF0000u)));
              } else {
                w[g][t][x] = transpose8x8(pack_half2(e[2 * x], e[2 * x + 1]));
              }
            }
          }
        }
        [[maybe_unused]] uint32_t odd = 0;
        [[maybe_unused]] const int odd0 = max(seen_by_all - tok, 0);        // the warp's first token that some columns do not see
        if constexpr (MODE == kRows)
          if (p.causal && tok + G::KT > seen_by_all) odd = take_odd<D, TYPE>(vs, odd0, min(len - tok, G::KT), lane);
        if constexpr (TYPE == SR_PAGE_BF16) {
          const int vr = (lane % 8) + 8 * (lane / 16), vc = (lane / 8) % 2;
#pragma unroll
          for (int g = 0; g < G::kGroups; ++g)
#pragma unroll
            for (int k = 0; k < D / 16; k += 2) {
              uint32_t a[4], b[4];
              ldsm4t(a, vs + chunk_at<G::kChunks>(g * 16 + vr, 2 * k + vc));
              ldsm4t(b, vs + chunk_at<G::kChunks>(g * 16 + vr, 2 * k + 2 + vc));
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                mma16816<TYPE>(o[t][k], a[0], a[1], a[2], a[3], w[g][t][0], w[g][t][1]);
                mma16816<TYPE>(o[t][k + 1], b[0], b[1], b[2], b[3], w[g][t][0], w[g][t][1]);
              }
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                mma16816<TYPE>(o[t][k], a[0], a[1], a[2], a[3], w_low[g][t][0], w_low[g][t][1]);
                mma16816<TYPE>(o[t][k + 1], b[0], b[1], b[2], b[3], w_low[g][t][0], w_low[g][t][1]);
              }
            }
        } else if constexpr (TYPE == SR_PAGE_INT4) {
          // a transposed 16-bit element is four neighbouring dims of one key, so that a decoded pair is one dim of two
          // keys: a product's rows 0-7 are the dims 4 r + 0 (or 2) of the chunk, rows 8-15 the next ones. Tokens that are
          // not there, or whose record is not, get a scale of zero.
          const uint32_t pick = 0x4240u + (r8 >> 2) * 0x0101u;     // of a word's four scales the two of this lane's blocks
#pragma unroll
          for (int g = 0; g < G::kGroups; ++g) {
            const uint32_t rec = vs + g * record_bytes(D);
            uint32_t sc[2][2 * (D / 64)];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              load_words(sc[x], rec + 8 * D + (2 * j4 + 8 * x) * (D / 16));
              if (live[g] != 16) {
#pragma unroll
                for (int y = 0; y < 2 * (D / 64); ++y)
                  if (live[g] <= 2 * j4 + 8 * x + y / (D / 64)) sc[x][y] = 0;
              }
#pragma unroll
              for (int y = 0; y < 2 * (D / 64); ++y) sc[x][y] = __byte_perm(sc[x][y], 0, pick) * shift7;
            }
#pragma unroll
            for (int ch = 0; ch < D / 32; ch += 2) {
              uint32_t a[4];
              ldsm4t(a, rec + ch * 256 + lane * 16);
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                uint32_t v0[4], v1[4];
                auto pair_of = [&](int x) {
                  return scale_pair(__byte_perm(sc[x][ch / 2], sc[x][D / 64 + ch / 2], y == 0 ? 0x5410 : 0x7632));
                };
                decode_word(v0, a[2 * y], pair_of(0), masks);
                decode_word(v1, a[2 * y + 1], pair_of(1), masks);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                  mma16816<TYPE>(o[t][2 * (ch + y)], v0[0], v0[1], v1[0], v1[1], w[g][t][0], w[g][t][1]);
                  mma16816<TYPE>(o[t][2 * (ch + y) + 1], v0[2], v0[3], v1[2], v1[3], w[g][t][0], w[g][t][1]);
                }
              }
            }
          }
        } else {
          // a transposed 16-bit element is two neighbouring dims of one key: rows 0-7 of the
          // product are the even dims, rows 8-15 the odd ones
          const int vr = (lane % 8) + 8 * ((lane / 8) % 2), vc = lane / 16;
#pragma unroll
          for (int g = 0; g < G::kGroups; ++g)
#pragma unroll
            for (int k = 0; k < D / 16; k += 2) {
              uint32_t a[4];
              ldsm4t(a, vs + chunk_at<G::kChunks>(g * 16 + vr, k + vc));
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const uint32_t y0 = __byte_perm(a[2 * x], 0, 0x3120), y1 = __byte_perm(a[2 * x + 1], 0, 0x3120);
                const uint32_t a0 = half2_of_e4m3(y0), a1 = half2_of_e4m3(y0 >> 16);
                const uint32_t a2 = half2_of_e4m3(y1), a3 = half2_of_e4m3(y1 >> 16);
#pragma unroll
                for (int t = 0; t < NT; ++t) mma16816<TYPE>(o[t][k + x], a0, a1, a2, a3, w[g][t][0], w[g][t][1]);
              }
            }
        }
        if constexpr (MODE == kRows) {
#pragma unroll 1
          for (; odd; odd &= odd - 1) {
            const int32_t token = tok + odd0 + __ffs(odd) - 1;
            const int32_t seq = p.b.id[item_i];
            const int kv = kv_head(item_h);
            const float scale = c.scale_log2 * (G::kRecords ? kDecoded : 1.f) * (c.kv_exp ? exp2f(static_cast<float>(c.kv_exp[kv])) : 1.f);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const int col = 8 * t + 2 * j4 + x, j = static_cast<int>(static_cast<uint32_t>(col) * p.group_magic >> 16);
                if (col >= columns || token >= seen_by_all + j) continue;
                const float wt = weight_again<D, TYPE>(p, seq, token, kv, row_of<MODE>(p, item_i, item_h, col), scale, m[t][x]);
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
#pragma unroll
                  for (int y = 0; y < 2; ++y) {
                    const int dim = TYPE == SR_PAGE_BF16 ? 16 * k + r8 + 8 * y
                                    : TYPE == SR_PAGE_E4M3 ? 16 * k + 2 * r8 + y : 32 * (k / 2) + 4 * r8 + 2 * (k % 2) + y;
                    const float v = page_value<D, TYPE>(c, p.kv_heads, c.v_pages, seq, token, kv, dim);
                    if (!(fabsf(v) < INFINITY)) o[t][k][x + 2 * y] = fmaf(wt, v, o[t][k][x + 2 * y]);
                  }
              }
          }
        }
      } else if constexpr (MASS) {
        // no token here, or none with a page: weights of zero
        if (score) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (8 * t + 2 * j4 + x % 2 < group)
#pragma unroll
                for (int g = 0; g < G::kGroups; ++g) score[(8 * t + x % 2) * G::CT + g * 16 + 8 * (x / 2)] = -INFINITY;
        }
      }
      __syncwarp();
      stage = (stage + 1) % kStages;
      cursor_next<G::CT>(comp, sh, n_kv, left);
    }
    if (left > 0) fetch_q(comp.i, comp.h);

    // ---- merge the four warps' results: each puts its sums into the stage that it has just
    // read, which the next copy fills, then all threads add them up and write
    const bool whole = first_tile == 0 && end_tile == tiles;
    float* part = part_at<D>(p, blockIdx.x, first_tile == 0 ? 1 : 0);
    const int free_stage = (stage + kStages - 1) % kStages;
    const float vscale =
        (G::kRecords ? kDecoded : 1.f) * (c.kv_exp ? exp2f(static_cast<float>(c.kv_exp[p.kv_heads + kv_head(item_h)])) : 1.f);
    constexpr int kQuads = D / 4;                 // of a row
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (8 * t >= columns) break;
      float* mine = reinterpret_cast<float*>(smem + (warp * kStages + free_stage) * G::kStageBytes);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float y = l[t][x];
#pragma unroll
        for (int k = 4; k < 32; k *= 2) y += __shfl_xor_sync(0xffffffffu, y, k);
        if (r8 == 0) {
          sh.ml[warp][2 * j4 + x][0] = m[t][x];
          sh.ml[warp][2 * j4 + x][1] = y;
        }
      }
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float* row = mine + (2 * j4 + x) * G::kMergeRow + 16 * k;
          if constexpr (TYPE == SR_PAGE_BF16) {
            row[r8] = o[t][k][x];
            row[r8 + 8] = o[t][k][x + 2];
          } else if constexpr (TYPE == SR_PAGE_INT4) {
            if (k % 2 == 0)
              *reinterpret_cast<float4*>(row + 4 * r8) = make_float4(o[t][k][x], o[t][k][x + 2], o[t][k + 1][x], o[t][k + 1][x + 2]);
          } else {
            *reinterpret_cast<float2*>(row + 2 * r8) = make_float2(o[t][k][x], o[t][k][x + 2]);
          }
        }
      __syncthreads();
#pragma unroll 1
      for (int y = threadIdx.x; y < 8 * kQuads; y += kThreads) {
        const int r = y / kQuads, quad = y - r * kQuads, row = 8 * t + r;
        if (row >= columns) break;
        float top = sh.ml[0][r][0];
#pragma unroll
        for (int v = 1; v < kWarps; ++v) top = fmaxf(top, sh.ml[v][r][0]);
        float sum = 0.f;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int v = 0; v < kWarps; ++v) {
          const float mv = sh.ml[v][r][0];
          const float f = mv == -INFINITY ? 0.f : ex2_approx(mv - top);
          sum = fmaf(f, sh.ml[v][r][1], sum);
          const float4 z = *reinterpret_cast<const float4*>(smem + (v * kStages + free_stage) * G::kStageBytes +
                                                            (r * G::kMergeRow + 4 * quad) * 4);
          a.x = fmaf(f, z.x, a.x);
          a.y = fmaf(f, z.y, a.y);
          a.z = fmaf(f, z.z, a.z);
          a.w = fmaf(f, z.w, a.w);
        }
        const float scale = whole ? (sum == 0.f ? 0.f : vscale / sum) : vscale;
        a.x *= scale;
        a.y *= scale;
        a.z *= scale;
        a.w *= scale;
        if (whole) {
          if (sum == 0.f) a = make_float4(0.f, 0.f, 0.f, 0.f);       // no weight: 0, whatever the values are
          const int64_t out = row_of<MODE>(p, item_i, item_h, row);
          *reinterpret_cast<uint2*>(p.o + out * D + 4 * quad) = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
          if (quad == 0) {
            const float lse2 = sum == 0.f ? -INFINITY : top + log2f(sum);
            if (p.lse) p.lse[out] = lse2 * kLn2;
            if (MASS) p.lse2[out] = weight_reference(lse2);
          }
        } else {
          *reinterpret_cast<float4*>(part + row * D + 4 * quad) = a;
          if (quad == 0) {
            part[p.part_rows * D + 2 * row] = top;
            part[p.part_rows * D + 2 * row + 1] = sum;
          }
        }
      }
      if constexpr (G::kRecords) fence_proxy_async_smem();
      __syncthreads();   // the stages may be filled again
    }
    if (whole) {
      if (p.items && threadIdx.x == 0) p.items[item_i * c.n_kv + item_h] = make_int2(0, 1);
    } else {
      // The parts of this item lie with CTAs c0 .. c1. The last of a group of kJoin to
      // arrive joins the group, the last group to be joined the item.
      auto owner = [&](int64_t u) {   // of unit u of the line
        const int64_t longer = rest * (share + 1);
        return static_cast<int>(u < longer ? div_pos(u, share + 1) : rest + div_pos(u - longer, share));
      };
      const int c0 = cut ? (item_i * n_kv + comp_h) * p.pieces : owner(item_u);
      const int n_parts = cut ? cut : owner(item_u + tiles - 1) - c0 + 1;
      auto arrive = [&](int32_t* ctr, int need) -> bool {   // behind a barrier; true for the whole CTA in the last one
        if (threadIdx.x == 0) {
          const bool all = add_acq_rel(ctr, 1) == need - 1;
          if (all) *ctr = 0;
          sh.last = all;
        }
        __syncthreads();
        const bool all = sh.last;
        __syncthreads();
        return all;
      };
      if (p.items) {
        if (first_tile == 0 && threadIdx.x == 0) p.items[item_i * c.n_kv + item_h] = make_int2(c0 * S + sub, n_parts);
      } else if (n_parts <= kJoin) {
        if (arrive(p.arrivals + c0 * S + sub, n_parts)) join_parts<D, MODE>(p, c0 * S + sub, 1, S, n_parts, nullptr, item_i, item_h, warp, lane);
      } else {
        const int g = (me - c0) / kJoin, lead = (c0 + g * kJoin) * S + sub, s0 = g == 0 ? 1 : 0;
        const int size = min(kJoin, n_parts - g * kJoin);
        if (arrive(p.group_arrivals + 2 * lead + s0, size)) {
          join_parts<D, MODE>(p, lead, s0, S, size, part_at<D>(p, lead, s0), item_i, item_h, warp, lane);
          __syncthreads();
          if (arrive(p.arrivals + c0 * S + sub, (n_parts + kJoin - 1) / kJoin))
            join_parts<D, MODE>(p, c0 * S + sub, 1, kJoin * S, (n_parts + kJoin - 1) / kJoin, nullptr, item_i, item_h, warp, lane);
        }
      }
    }
  }
}

// The join as a launch of its own, for many rows of many parts: a CTA per query row, its
// warps share the parts and add up in a fixed order.
constexpr int kJoinWarps = 8;
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) paged_join_kernel(const __grid_constant__ PagedAttnParams p) {
  constexpr int kCols = D / 32, kBatch = 8;
  __shared__ float ml[kJoinWarps][2];
  __shared__ float sums[kJoinWarps][D];
  grid_dep_launch_dependents();
  grid_dep_wait();
  const int group = p.c.group, item = blockIdx.x / group, r = blockIdx.x - item * group;
  const int2 it = p.items[item];
  const int n = it.y;
  if (n == 1) return;                     // written by the CTA that had it whole
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  float top = -INFINITY, sum = 0.f, a[kCols];
#pragma unroll
  for (int x = 0; x < kCols; ++x) a[x] = 0.f;
#pragma unroll 1
  for (int k0 = warp; k0 < n; k0 += kBatch * kJoinWarps) {
    float v[kBatch][kCols];
    float2 m[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int kk = min(k0 + k * kJoinWarps, n - 1);
      const float* src = part_at<D>(p, it.x + kk * p.spread, kk == 0 ? 1 : 0);
      m[k] = *(reinterpret_cast<const float2*>(src + group * D) + r);
      src += r * D + lane * kCols;
      if constexpr (kCols == 4) {
        const float4 x = *reinterpret_cast<const float4*>(src);
        v[k][0] = x.x; v[k][1] = x.y; v[k][2] = x.z; v[k][3] = x.w;
      } else {
        const float2 x = *reinterpret_cast<const float2*>(src);
        v[k][0] = x.x; v[k][1] = x.y;
      }
      if (k0 + k * kJoinWarps >= n) m[k] = make_float2(-INFINITY, 0.f);   // past the end: no weight
    }
    float t = top;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) t = fmaxf(t, m[k].x);
    const float f = top == -INFINITY ? 1.f : ex2_approx(top - t);
    top = t;
    sum *= f;
#pragma unroll
    for (int x = 0; x < kCols; ++x) a[x] *= f;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const float w = m[k].x == -INFINITY ? 0.f : ex2_approx(m[k].x - top);
      sum = fmaf(w, m[k].y, sum);
      if (k0 + k * kJoinWarps < n)
#pragma unroll
        for (int x = 0; x < kCols; ++x) a[x] = fmaf(w, v[k][x], a[x]);
    }
  }
  if (lane == 0) {
    ml[warp][0] = top;
    ml[warp][1] = sum;
  }
#pragma unroll
  for (int x = 0; x < kCols; ++x) sums[warp][lane * kCols + x] = a[x];
  __syncthreads();
  const int64_t out = static_cast<int64_t>(item) * group + r;   // [n][n_kv][group] is [n][n_heads]
  if (threadIdx.x >= D / 2) return;
  float all = ml[0][0];
#pragma unroll
  for (int w = 1; w < kJoinWarps; ++w) all = fmaxf(all, ml[w][0]);
  float l = 0.f, y0 = 0.f, y1 = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    const float f = ml[w][0] == -INFINITY ? (ml[w][1] == 0.f ? 0.f : 1.f) : ex2_approx(ml[w][0] - all);
    l = fmaf(f, ml[w][1], l);
    y0 = fmaf(f, sums[w][2 * threadIdx.x], y0);
    y1 = fmaf(f, sums[w][2 * threadIdx.x + 1], y1);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if (l == 0.f) y0 = y1 = 0.f;          // no weight: 0, whatever the values are
  reinterpret_cast<uint32_t*>(p.o + out * D)[threadIdx.x] = pack_bf16x2(y0 * inv, y1 * inv);
  if (threadIdx.x == 0) {
    const float lse2 = l == 0.f ? -INFINITY : all + log2f(l);
    if (p.lse) p.lse[out] = lse2 * kLn2;
    p.lse2[out] = weight_reference(lse2);
  }
}

// The weights: mass(t) <- decay * mass(t) + sum over heads of 2^(x_h(t) - lse2_h).
// Latency bound (the scores mostly still lie in L2), so few dependent loads: a CTA takes
// 128 tokens, four per thread in one 16-byte load per head; eight threads share a token's
// heads, with their loads in flight together, and add up in a fixed order. It adds 6 us to a
// call with 73,000 tokens and 40 heads and 6.5 us with 131,000 and 32 (64 tokens per CTA, and
// half as many CTAs, measured the same). The first launch pays for what L2 writes back of the
// scores meanwhile (8 us for the 17 MB of 32 sequences of 4096 tokens; 1 us if all go to one small
// place). So in large batches they are stored to leave L2 last and dropped from it once read (DROP):
// 94.5 us in all without that, 91.2 us with it; 8 of 16384 101.3 us, 98.1 us; 32 of 2048, at
// kDropScores, 50.5 us, 49.7 us; below, 32 of 512, 19.6 us, 20.4 us. The rule goes by the capacity, since only the device
// knows the lengths: short sequences in a large capacity pay that last difference.
constexpr int64_t kDropScores = 1ll << 21;
constexpr int kMassTokens = 128;
constexpr int kMassShare = 8;
constexpr int kMassQuads = kMassTokens / 4;
constexpr int kMassThreads = kMassQuads * kMassShare;
template <int CT, bool DROP>
__global__ void __launch_bounds__(kMassThreads) paged_mass_kernel(const __grid_constant__ PagedAttnParams p, int per) {
  __shared__ float4 sums[kMassShare][kMassQuads];
  grid_dep_launch_dependents();
  grid_dep_wait();
  const PagedView& c = p.c;
  const int i = blockIdx.x / per, S = p.spread;
  const int32_t seq = p.b.id[i];
  const int64_t unit0 = p.unit0[i];
  const int32_t len = min(max(c.seq_len[seq], 0), c.cap);
  const int32_t tiles = (len + CT - 1) / CT;
  if (p.unit0[p.b.n] * S > p.score_tiles) {    // not all are stored: no sequence's weights change
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicCAS(c.err_word, 0, SR_DEVERR_WORKSPACE);
    return;
  }
  const int32_t* table = c.table + static_cast<int64_t>(seq) * c.max_pages;
  const float* lse2 = p.lse2 + static_cast<int64_t>(i) * c.n_heads;
  const int quad = threadIdx.x % kMassQuads, share = threadIdx.x / kMassQuads;
  // from a key head's scores to the next one's on the line; neighbours of one CTA group lie side by side
  const int64_t pitch = static_cast<int64_t>(tiles + kItemCost) * S * c.group * CT;
  for (int32_t t0 = (blockIdx.x % per) * kMassTokens; t0 < len; t0 += per * kMassTokens) {
    const int32_t t = t0 + 4 * quad;
    float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
    float old[4];
    bool seen = false;
    float* mass = c.token_mass + static_cast<int64_t>(seq) * c.cap + t;
    if (t < len) {
      const float* x = p.scores + (unit0 + kItemCost + t / CT) * S * c.group * CT + t % CT;
      if (share == 0) {
        seen = paged_row(table, t, c.page_tokens, c.n_pages) >= 0;   // else left as they are
#pragma unroll
        for (int k = 0; k < 4; ++k) old[k] = t + k < len ? mass[k] : 0.f;
      }
      int kv = share / c.group, g = share - kv * c.group;
#pragma unroll 8
      for (int h = share; h < c.n_heads; h += kMassShare) {
        const int side = kv / S;
        const float4 v = __ldcg(reinterpret_cast<const float4*>(x + side * pitch + ((kv - side * S) * c.group + g) * CT));
        const float l = __ldcg(lse2 + h);
        w.x += ex2_approx(v.x - l);
        w.y += ex2_approx(v.y - l);
        w.z += ex2_approx(v.z - l);
        w.w += ex2_approx(v.w - l);
        g += kMassShare;
        while (g >= c.group) {
          g -= c.group;
          ++kv;
        }
      }
    }
    sums[share][quad] = w;
    __syncthreads();
    if (DROP && t0 + kMassTokens <= len) {         // read by this CTA alone, and read now
      constexpr int kLines = kMassTokens / 32;     // of a head's scores
      for (int y = threadIdx.x; y < c.n_heads * kLines; y += kMassThreads) {
        const int h = y / kLines, kv = h / c.group, g = h - kv * c.group, side = kv >> p.spread_log2;
        const int32_t first = t0 + (y - h * kLines) * 32;
        discard_line(p.scores + (unit0 + kItemCost + first / CT) * S * c.group * CT + first % CT + side * pitch +
                     ((kv - side * S) * c.group + g) * CT);
      }
    }
    if (seen) {
      float4 all = sums[0][quad];
#pragma unroll
      for (int k = 1; k < kMassShare; ++k) {
        const float4 y = sums[k][quad];
        all.x += y.x;
        all.y += y.y;
        all.z += y.z;
        all.w += y.w;
      }
      const float sum[4] = {all.x, all.y, all.z, all.w};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (t + k < len) mass[k] = fmaf(p.mass_decay, old[k], sum[k]);
    }
    __syncthreads();
  }
}

template <int D, int TYPE>
constexpr int kSmem = Geo<D, TYPE>::kStageArea + static_cast<int>(sizeof(SharedHead));

template <int D, int TYPE, int NT>
cudaError_t prepare() {
  static_assert(Geo<D, TYPE>::kCtasPerSm * (kSmem<D, TYPE> + 1024) <= 228 * 1024, "the CTAs of an SM do not fit");
  cudaError_t e = cudaFuncSetAttribute(paged_attn_kernel<D, TYPE, NT, kPlain>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem<D, TYPE>);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(paged_attn_kernel<D, TYPE, NT, kMass>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem<D, TYPE>);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(paged_attn_kernel<D, TYPE, NT, kRows>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem<D, TYPE>);
  return e;
}

template <int D, int TYPE, int NT, int MODE>
cudaError_t launch(const Params<MODE>& p0, cudaStream_t st) {
  using G = Geo<D, TYPE>;
  Params<MODE> p = p0;
  p.spread = kSpread;
  p.spread_log2 = kSpreadLog2;
  while (p.c.n_kv % p.spread) p.spread /= 2, --p.spread_log2;
  const int ctas = std::min(G::kCtasPerSm * sm_count(), kMaxPagedCtas) / p.spread * p.spread;
  const int slots = ctas >> p.spread_log2, items = p.b.n * (p.c.n_kv >> p.spread_log2);
  p.each = (items + slots - 1) / slots;
  p.whole_cost = 16ll * p.each * slots;
  p.pieces = slots / items;
  p.cut_cost = p.pieces > 1 ? 16ll * slots / p.pieces : 0;
  const int extra = p.pieces > 1 ? G::kWholeExtra : G::kAloneExtra;
  p.whole_extra = 16ll * slots * extra;
  p.drop_scores = static_cast<int64_t>(p.b.n) * p.c.cap * p.c.n_heads >= kDropScores;
  // Who joins: the last CTA to arrive (its four warps take rows in turn, sixteen parts at a time, about 1.6 us
  // a turn), or a launch of its own (about 2 us of the GPU and as much of the host, more CTAs than it can use
  // in large batches). One sequence of 4096 tokens, 4 query heads per key head (39 parts): 12.6 us and 9.0 us;
  // 4 of 5000, 16 heads: 28.8 us and 10.5 us; 1 of 16 tokens: 4.1 us and 5.1 us; 256 of 16: 19 us and 29 us.
  const int parts = std::min(ctas / (p.b.n * p.c.n_kv) + 1, p.c.cap / G::CT + 1);
  const int turns = (p.c.group + 3) / 4 * ((parts + kJoinBatch - 1) / kJoinBatch);
  if (turns <= 2 + p.b.n * p.c.n_heads / 2048) p.items = nullptr;
  // no item is cut (see kWhole): nothing to join (1 sequence of 300 tokens, 16 heads: 9.8 us with the launch, 8.5 us)
  if (p.each == 1 && (p.c.cap + G::CT - 1) / G::CT + kItemCost <= extra) p.items = nullptr;
  if (MODE == kRows) p.items = nullptr;
  cudaError_t e = launch_dependent(paged_attn_kernel<D, TYPE, NT, MODE>, static_cast<unsigned>(ctas), kThreads,
                                   kSmem<D, TYPE>, st, p);
  if (e != cudaSuccess) return e;
  if (p.items) {
    e = launch_dependent(paged_join_kernel<D>, static_cast<unsigned>(p.b.n) * p.c.n_heads, kJoinWarps * 32, 0, st, p);
    if (e != cudaSuccess) return e;
  }
  if constexpr (MODE != kMass) return e; else {
  const int per = std::max(1, std::min((p.c.cap + kMassTokens - 1) / kMassTokens, 16 * sm_count() / p.b.n));
  return launch_dependent(p.drop_scores ? paged_mass_kernel<G::CT, true> : paged_mass_kernel<G::CT, false>,
                          static_cast<unsigned>(p.b.n) * per, kMassThreads, 0, st, p, per);
  }
}

}  // namespace

// The launchers of one page type, which has a translation unit to itself.
template <int TYPE>
cudaError_t attn_prepare(int head_dim) {
  if (head_dim == 128) {
    // a few new tokens may take both tiles of columns whatever the group
    const cudaError_t e = prepare<128, TYPE, 1>();
    return e == cudaSuccess ? prepare<128, TYPE, 2>() : e;
  }
  const cudaError_t e = prepare<64, TYPE, 1>();
  return e == cudaSuccess ? prepare<64, TYPE, 2>() : e;
}
template <int D, int TYPE>
cudaError_t attn_launch_d(const PagedAttnParams& p, cudaStream_t st) {
  const bool mass = p.mass_decay >= 0.f;
  if (p.c.group <= 8) return mass ? launch<D, TYPE, 1, kMass>(p, st) : launch<D, TYPE, 1, kPlain>(p, st);
  return mass ? launch<D, TYPE, 2, kMass>(p, st) : launch<D, TYPE, 2, kPlain>(p, st);
}
template <int TYPE>
cudaError_t attn_launch(const PagedAttnParams& p, cudaStream_t st) {
  return p.c.head_dim == 128 ? attn_launch_d<128, TYPE>(p, st) : attn_launch_d<64, TYPE>(p, st);
}
template <int TYPE>
cudaError_t rows_launch(const PagedRowsParams& p, cudaStream_t st) {
  if (p.c.head_dim == 128) return p.part_rows <= 8 ? launch<128, TYPE, 1, kRows>(p, st) : launch<128, TYPE, 2, kRows>(p, st);
  return p.part_rows <= 8 ? launch<64, TYPE, 1, kRows>(p, st) : launch<64, TYPE, 2, kRows>(p, st);
}
template <int TYPE>
int attn_tile_tokens(int head_dim) {
  return head_dim == 128 ? Geo<128, TYPE>::CT : Geo<64, TYPE>::CT;
}

}  // namespace sr
