// paged_prompt.cu -- attention of several new tokens per sequence over the paged token cache, on the tcgen05
// tensor cores:  o[r][h] = softmax(scale * q[r][h] . K) V  over the tokens that row r sees.
//
// A block is up to 256 query rows of one sequence and one key/value head: the rows of tile t are t * tpt .. of the
// block's new tokens, each with the heads that share the key head (tpt = 128 / group tokens fill a tile). Two tiles
// share every tile of 128 keys. A block whose rows fill one tile only gives the keys' even tiles to softmax group 0 and
// the odd ones to group 1, which merge at the end. A step is two score tiles in both forms, and all blocks' steps
// form one line that the CTAs, one per SM, share in equal stretches; whoever has a block whole writes its
// output, of a block cut between CTAs each writes a partial result, and the last of them joins them in the order of the
// line: on the way out of tensor memory where the others had written theirs before it began (mostly so: a CTA begins with
// the end of one block and ends with the beginning of another), in a pass of its own otherwise, with the same
// arithmetic. The lengths never reach the host and results do not depend on timing.
//
// Warp roles: 0-3 and 4-7 softmax groups (thread i owns row i of its tile), 8 issues the MMAs, 9 walks the tiles and looks
// up the block table, 10-11 copy queries, 12-15 bring keys and values. bf16 tiles come by tensor copies; e4m3 and 4 bits
// through registers, decoded to fp16, exactly, into the same 128-byte swizzle (two warps a tile, each register loaded
// again as soon as it is stored). Queries are bf16, or for fp16 products each row times a power of two (as in
// paged_attention.cuh), which the softmax group that owns the row writes in its place. TMEM: S0 [0,128) S1 [128,256)
// scores, O0 [256,256+d) O1 [384,384+d) sums; the weights go over the first half of their scores and from there to the
// second product.
//
// A weight of zero times a value that is no finite number is none either, so among new tokens that some rows do not see such
// values leave the tile (a flag for each 32 tokens tells), and are added to the rows that do see them at the block's end.
//
// What bounds it. Two score tiles and their products are 2048 clocks of the tensor pipe at 128 dims; a step takes about 3100: a
// group's chain (scores out, maximum, exponentials, weights in, second product, next scores) is longer than the other group's
// products that run meanwhile, and the issuing warp waits in order. That is not a limit: attention.cu, of the same groups and
// hand-overs, takes 2680 .. 2740, and where this kernel's other 400 go has not been measured. At 64 dims the products are
// half and the chain is the same. Instructions matter as much: one cache serves all roles' loops, and unrolling the
// loading warps' took up to a quarter longer. 8192 tokens from nothing, 32 heads, 8 key heads of 128, bf16: 455 us, 1208
// TFLOP/s (63 % of the burst rate); 4096 after 4096: 300 us, 1375 TFLOP/s (72 %), e4m3 350 us, 4 bits 366 us (of 64 dims: 252,
// 291, 292 us, 43, 37, 37 %); four sequences, 131 .. 1021 tokens after 2003 .. 16384, 40 heads, 4 bits: 545 us, 1010 TFLOP/s; two
// frames of 1560 that see 10920 tokens, 40 key heads, e4m3: 653 us, 1069 TFLOP/s. The first form of this kernel took 1323
// us for the first of these, with partial results joined row by row (55 us of it), queries copied 8 rows at a time.
//
// Precision. Scores, statistics and sums are fp32. For the second product weights are rounded once: to fp16 (2^-11), or, where
// the values are bf16, to bf16 (2^-8), since both operands have one type. That is a choice for speed: with what the rounding
// leaves as a second bf16 number (as in paged_attention.cuh, whose time is the stream) outputs are off by 0.0017 of
// themselves in the mean square, their own rounding, instead of 0.0023, and 8192 tokens take 762 us instead of 457.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "sr_device.cuh"
#include "sr_kernels.h"
#include "sr_paged.h"
#include "sr_paged_device.cuh"

namespace sr {

namespace {

constexpr int kThreads = 512;
constexpr int BM = 128, BN = 128;
constexpr int kMmaWarp = 8, kPlanWarp = 9, kQWarp0 = 10, kLoadWarp0 = 12;
constexpr int kQWarps = 2, kLoadWarps = 4;
constexpr int kLaunchRegs = 128;
constexpr uint32_t kRegsSoftmax = 176;
constexpr float kLn2 = 0.69314718055994531f;
constexpr uint64_t kTimeoutNs = 2000000000ull;
// Steps that changing blocks costs (queries, a chain that starts anew, results): a long prompt's first CTAs have many short
// blocks. With 1, 2, 3, 4, 6, in a captured graph: 8192 tokens from nothing, 128 dims, bf16 495, 467, 441, 440, 436 us, e4m3 573,
// 534, 509, 494, 500, 4 bits 595, 554, 526, 526, 527; 64 dims 382, 369, 374, 376, 376, and 438, 409, 399, 405, 408 (e4m3), 443, 413,
// 410, 414, 418. 4096 after 4096 and frames that see everything differ by 3 % at most (bf16 303, 303, 298, 300, 300; e4m3, 1560
// of 10920 364, 364, 360, 359, 356).
constexpr int kItemCost = 4;
// A block's flags are kept for kFlagSlots blocks: who writes those of the eighth block behind one has had a stage back (of
// 8 at most, two tiles a block) that the second block behind it used, whose weights softmax group 0 made after both
// groups had read the first one's flags.
constexpr int kFlagSlots = 8, kFlagTiles = 3;
constexpr int kBarBytes = 3 * 1024;
template <int D, int TYPE>
struct Cfg {
  static constexpr bool kHalf = TYPE != SR_PAGE_BF16;       // products of fp16, else of bf16
  static constexpr uint32_t kRegsOther = 72, kRegsLoad = 160 - kRegsOther;
  static_assert(2 * 128 * kRegsSoftmax + 128 * (kRegsOther + kRegsLoad) <= kThreads * kLaunchRegs,
                "register split exceeds what the block is launched with");
  static constexpr int kUnrollT = kHalf ? 1 : 2;            // (where the loading warps' loops are longer, this one is shorter)
  static constexpr int kAtoms = D / 64;
  static constexpr int kAtomBytes = BM * 128;
  static constexpr int kTileBytes = kAtoms * kAtomBytes;
  static constexpr int kStages = D == 128 ? 5 : 8;
  // loading warps that share a tile; the others are at the next tiles meanwhile
  static constexpr int kPerTile = TYPE == SR_PAGE_BF16 ? 1 : 2;
  static constexpr int kTeams = kLoadWarps / kPerTile, kSubs = 4 / kPerTile;     // a warp's shares of a tile, 32 tokens each
  static constexpr int kSmemQ = 2 * kTileBytes;
  static constexpr int kSmemKV = kStages * kTileBytes;
  static constexpr int kSmemBytes = kSmemQ + kSmemKV + kBarBytes;
  static_assert(kSmemBytes <= 232448, "more than 227 KB of shared memory per block");
  static constexpr uint32_t kIdescS = kHalf ? idesc_f16_f32(BM, BN, 0) : idesc_bf16_f32(BM, BN, 0);
  static constexpr uint32_t kIdescPV = kHalf ? idesc_f16_f32(BM, D, 1) : idesc_bf16_f32(BM, D, 1);
  // the reference of the exponentials lies kLift below an earlier maximum and is raised when a score passes it by kSlack
  static constexpr float kLift = kHalf ? 6.f : 0.f, kSlack = 8.f;
  static constexpr float kDecodedBy = TYPE == SR_PAGE_INT4 ? kDecoded : 1.f;
};

// One block of query rows, and the part of its steps that this CTA takes.
struct Block {
  int i, h, b;           // sequence of the call, item head, block of the sequence
  int32_t base;          // tokens before the new ones; negative where the sequence is shorter than its rows
  int32_t tok0, ntok;    // its new tokens
  int32_t lim_min, lim;  // tokens that its first and last row see
  int32_t tiles, steps;  // key tiles, steps in all
  bool split;            // one query tile: the groups share the key tiles
  int32_t s0, s1;        // steps of this CTA
  __device__ __forceinline__ int count(int t) const {
    return !split ? s1 - s0 : t == 0 ? s1 - s0 : max(min(s1, tiles / 2) - s0, 0);
  }
  __device__ __forceinline__ int tile(int t, int j) const { return split ? 2 * (s0 + j) + t : s0 + j; }
};

struct Start {
  int64_t left;          // units of this CTA's stretch from its first step on
  int64_t share, rest;   // units of every CTA, and how many have one more
  int32_t i, h, b, s0;
  int64_t u;             // unit of the first block's first step (not this CTA's)
};

// A tile of 128 tokens' keys or values, for the loading warps.
struct Tile {
  int64_t off[8];      // where each group of 16 tokens begins for this head (bf16: its pool row); -1: zeros
  int32_t lim;         // tokens from here on (within the tile) are zeros
  int32_t watch;       // tokens from here on are seen by some rows only: values that are no finite numbers leave the tile
  int32_t head;        // key/value head
  int32_t meta;        // bit 0: values; bits 1-3: slot of the block's flags; bits 8..: flag word. -1: no more tiles
};
constexpr int kTileSlots = 8;

struct Record {        // a block, as the softmax groups read it
  Block k;
  int32_t c0, parts;   // the first of the CTAs that share it, and how many do
  bool last;           // the others had written their parts before this CTA began
};

struct Bars {
  uint64_t q_raw, q_full, q_empty, q_seen;   // q_raw: fp16 products, the rows as they came
  uint64_t kv_full[8], kv_empty[8];
  uint64_t s_full[2], p_half[2], p_full[2], o_done[2];
  uint64_t x_full, x_empty, part_done, part_last, drain;
  uint64_t fixed[kLoadWarps];          // bf16: values that a loading warp finishes have landed
  uint64_t tile_full[kTileSlots], tile_empty[kTileSlots];
  Tile tile[kTileSlots];
  Record rec[2];
  uint32_t tmem_base;
  int bad;               // an entry that is no page of the pool has been met
  int abort;
  int last;
  int joined;            // split blocks: group 0 has joined the parts
  Start start;
  // of a block: new tokens with values that are no finite numbers, by 32 tokens of a key tile, the tiles counted from the
  // first that some row does not see whole
  uint32_t flags[kFlagSlots][4][kFlagTiles];
  int8_t qexp[BM];               // split blocks, fp16 products: the rows' exponents for group 1
  float xm[BM], xl[BM];
};
static_assert(sizeof(Bars) <= kBarBytes, "barrier area too small");

struct Setup {                   // overlays the stages before they are used
  int64_t cum[kMaxPagedSeqs + 1];
  unsigned long long per_head[kMaxPagedSeqs];
  int32_t len[kMaxPagedSeqs];
  int none;                      // some block's rows see nothing
};

__device__ __forceinline__ void set_block(const PromptParams& p, Block& k, int32_t len) {
  const int32_t count = p.row0[k.i + 1] - p.row0[k.i];
  k.base = len - count;
  k.tok0 = k.b * 2 * p.tpt;
  k.ntok = min(2 * p.tpt, count - k.tok0);
  k.lim = max(p.causal ? k.base + k.tok0 + k.ntok : len, 0);
  k.lim_min = max(p.causal ? k.base + k.tok0 + 1 : len, 0);
  k.split = k.ntok <= p.tpt;
  k.tiles = (k.lim + BN - 1) / BN;
  k.steps = k.split ? (k.tiles + 1) / 2 : k.tiles;
}
__device__ __forceinline__ int32_t seq_length(const PromptParams& p, int i) {
  return min(max(__ldg(p.c.seq_len + p.id[i]), 0), p.c.cap);
}
__device__ __forceinline__ int blocks_of(const PromptParams& p, int i) {
  return (p.row0[i + 1] - p.row0[i] + 2 * p.tpt - 1) / (2 * p.tpt);
}
__device__ __forceinline__ int seq_of_block(const PromptParams& p, int x) {   // x among the blocks of all sequences
  int lo = 0, hi = p.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (p.blk0[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}
__device__ __forceinline__ int64_t units_of(const Block& k) { return k.steps > 0 ? k.steps + kItemCost : 0; }

// This CTA's blocks, one after the other; every role walks them by itself.
struct Walker {
  const PromptParams& p;
  Block k;
  int32_t left;                  // units left (launch_paged_prompt takes no call whose stretches hold 2^31)
  int64_t u;                     // unit of the block's first step
  int32_t len;
  int nb;
  bool first;
  __device__ __forceinline__ Walker(const PromptParams& p_, const Start& s) : p(p_) {
    k.i = s.i;
    k.h = s.h;
    k.b = s.b;
    left = static_cast<int32_t>(s.left);
    u = s.u;
    first = true;
    if (left > 0) {
      len = seq_length(p, k.i);
      nb = blocks_of(p, k.i);
      set_block(p, k, len);
      k.s0 = s.s0;
    }
  }
  __device__ __forceinline__ bool next() {
    if (!first) {
      if (left <= 0) return false;
      u += k.steps;
      do {                       // the line holds a unit here, so that some block has steps
        if (++k.b == nb) {
          k.b = 0;
          if (++k.h == p.c.n_kv) {
            k.h = 0;
            do {
              ++k.i;
              nb = blocks_of(p, k.i);
            } while (nb == 0);
            len = seq_length(p, k.i);
          }
        }
        set_block(p, k, len);
      } while (k.steps == 0);
      k.s0 = 0;
      u += kItemCost;
      left -= kItemCost;
    }
    if (left <= 0) return false;
    first = false;
    k.s1 = min(k.steps, k.s0 + left);
    left -= k.s1 - k.s0;
    return true;
  }
};

__device__ __forceinline__ int64_t div_pos(int64_t a, int64_t b) {   // a >= 0, b > 0; mostly short numbers
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}
__device__ __forceinline__ int owner_of(int64_t u, int64_t share, int64_t rest) {
  const int64_t longer = rest * (share + 1);
  return static_cast<int>(u < longer ? div_pos(u, share + 1) : rest + div_pos(u - longer, share));
}

// -------------------------------------------------------------- loading keys and values
struct TileRef {
  int32_t tok0, lim, watch;      // first token; as in Tile, of the sequence
  int32_t seq, head, meta;       // row of the block table
};

// The tiles of this CTA in the order in which the MMAs take them: before every step's keys the values of the step before.
struct TileWalk {
  Walker w;
  int j, t, part;      // step of the block (0 .. n), softmax group, 0 values 1 keys
  int n;
  bool open;
  int block;           // blocks so far
  __device__ __forceinline__ TileWalk(const PromptParams& p, const Start& s) : w(p, s) {
    block = -1;
    open = w.next();
    begin();
  }
  __device__ __forceinline__ void begin() {
    j = t = part = 0;
    n = open ? w.k.s1 - w.k.s0 : 0;
    ++block;
  }
  __device__ __forceinline__ bool next(TileRef& r, const PromptParams& p) {
    while (open) {
      while (j <= n) {
        const int jj = part == 0 ? j - 1 : j, tt = t, pp = part;
        const bool there = jj >= 0 && jj < w.k.count(tt);
        // on to the next place
        if (++part == 2) {
          part = 0;
          if (w.k.split && t == 0) {
            t = 1;
          } else {
            t = 0;
            ++j;
          }
        }
        if (!there) continue;
        const int tile = w.k.tile(tt, jj);
        const int flag = max(tile - w.k.lim_min / BN, 0);
        r.tok0 = tile * BN;
        r.lim = w.k.lim;
        r.watch = p.causal ? w.k.lim_min : INT32_MAX;
        r.seq = p.id[w.k.i];
        r.head = static_cast<int>(static_cast<uint32_t>(w.k.h) * p.head_magic >> 22);
        r.meta = (pp == 0 ? 1 : 0) | (block % kFlagSlots) << 1 | flag << 8;
        return true;
      }
      open = w.next();
      begin();
    }
    return false;
  }
};

__device__ __forceinline__ void store16(uint32_t dst, const uint4& x) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(dst), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w) : "memory");
}
__device__ __forceinline__ uint4 load16(uint32_t src) {
  uint4 x;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(src) : "memory");
  return x;
}
// 16-byte piece `piece` (of 8 elements) of row r of a tile
template <int D>
__device__ __forceinline__ uint32_t piece_at(int r, int piece) {
  return static_cast<uint32_t>((piece >> 3) * (BM * 128) + r * 128 + (((piece & 7) ^ (r & 7)) << 4));
}
// zero the elements that are no finite numbers; true if there were any
template <bool HALF>
__device__ __forceinline__ bool finite_only(uint32_t& x) {
  constexpr uint32_t kExp = HALF ? 0x7C00u : 0x7F80u;
  const bool lo = (x & kExp) == kExp, hi = (x & kExp << 16) == kExp << 16;
  if (lo) x &= 0xFFFF0000u;
  if (hi) x &= 0x0000FFFFu;
  return lo || hi;
}
template <bool HALF>
__device__ __forceinline__ bool finite_only(uint4& x) {
  bool any = finite_only<HALF>(x.x);
  any |= finite_only<HALF>(x.y);
  any |= finite_only<HALF>(x.z);
  any |= finite_only<HALF>(x.w);
  return any;
}

// A share of a tile: 32 tokens, two groups of 16.
struct Share {
  int64_t off[2];
  int32_t lim, watch, head, meta;         // lim, watch: of these 32
  __device__ __forceinline__ bool values() const { return meta & 1; }
  __device__ __forceinline__ bool watched() const { return values() && watch < 32; }
};

// 16-byte pieces of a share that a lane holds. e4m3: four lanes take 64 bytes of a token's row, eight tokens at once;
// 4 bits: lanes 0-15 a chunk of a group's 16 tokens, lanes 16-31 the next one.
template <int D, int TYPE>
struct Raw {
  static constexpr int kVec = TYPE == SR_PAGE_E4M3 ? D / 16 : TYPE == SR_PAGE_INT4 ? D / 32 : 1;
  uint4 x[kVec];
  uint32_t s[TYPE == SR_PAGE_INT4 ? kVec : 1];
};
// Where a lane's pieces lie. Tokens that are not there are zeros (their scales are, for 4 bits).
template <int D, int TYPE>
struct Source {
  const uint8_t* at[2];        // this lane's place in each group
  int32_t live[2];             // tokens of the group that are there
  __device__ __forceinline__ void set(const Share& r, const PagedView& c, int kv_heads, int lane) {
    const uint8_t* pages = static_cast<const uint8_t*>(r.values() ? c.v_pages : c.k_pages);
    const int64_t mine = TYPE == SR_PAGE_INT4 ? lane * 16 : static_cast<int64_t>(lane / 4) * kv_heads * D + lane % 4 * 16;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      at[x] = pages + r.off[x] + mine;
      live[x] = r.off[x] < 0 ? 0 : r.lim - x * 16;
    }
  }
  __device__ __forceinline__ void load(Raw<D, TYPE>& v, int i, int kv_heads, int lane) const {
    constexpr int kPer = Raw<D, TYPE>::kVec / 2;
    const int x = i / kPer, y = i % kPer;
    if constexpr (TYPE == SR_PAGE_INT4) {
      const bool there = (lane & 15) < live[x];
      v.x[i] = there ? __ldg(reinterpret_cast<const uint4*>(at[x] + y * 512)) : make_uint4(0, 0, 0, 0);
      v.s[i] = there ? __ldg(reinterpret_cast<const uint16_t*>(at[x] + 8 * D - lane * 16 + (lane & 15) * (D / 16) + 2 * (lane / 16) + 4 * y)) : 0;
    } else if constexpr (TYPE == SR_PAGE_E4M3) {
      constexpr int kAcross = D / 64;         // pieces of a token
      const bool there = y / kAcross * 8 + lane / 4 < live[x];
      v.x[i] = there ? __ldg(reinterpret_cast<const uint4*>(at[x] + y / kAcross * 8 * static_cast<int64_t>(kv_heads) * D + y % kAcross * 64))
                     : make_uint4(0, 0, 0, 0);
    }
  }
};
// Decodes piece i into rows chunk * 32 .. of a tile.
template <int D, int TYPE>
__device__ __forceinline__ void store_raw(const Raw<D, TYPE>& v, int i, uint32_t tile, int chunk, int lane, const DecodeMasks& masks) {
  constexpr int kPer = Raw<D, TYPE>::kVec / 2;
  const int x = i / kPer, y = i % kPer;
  const uint4 z = v.x[i];
  if constexpr (TYPE == SR_PAGE_INT4) {
    const uint32_t b = v.s[i], word[4] = {z.x, z.y, z.z, z.w};
    const ScalePair s0 = scale_pair(__byte_perm(b, 0, 0x4040) << 7), s1 = scale_pair(__byte_perm(b, 0, 0x4141) << 7);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t e[4];
      decode_word(e, word[q], q < 2 ? s0 : s1, masks);
      store16(tile + piece_at<D>(chunk * 32 + x * 16 + (lane & 15), (2 * y + lane / 16) * 4 + q), make_uint4(e[0], e[1], e[2], e[3]));
    }
  } else if constexpr (TYPE == SR_PAGE_E4M3) {
    constexpr int kAcross = D / 64;
    const int row = chunk * 32 + x * 16 + y / kAcross * 8 + lane / 4, piece = y % kAcross * 8 + lane % 4 * 2;
    store16(tile + piece_at<D>(row, piece),
            make_uint4(half2_of_e4m3(z.x), half2_of_e4m3(z.x >> 16), half2_of_e4m3(z.y), half2_of_e4m3(z.y >> 16)));
    store16(tile + piece_at<D>(row, piece + 1),
            make_uint4(half2_of_e4m3(z.z), half2_of_e4m3(z.z >> 16), half2_of_e4m3(z.w), half2_of_e4m3(z.w >> 16)));
  }
}

__device__ __forceinline__ void copy16_or_zero(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
// Values as the products need them, row by row of a share: zeros where there is no token (ZERO), finite where some rows do
// not see them; returns a bit per token of the 32 whose values were not (and are zeros now).
template <int D, bool HALF, bool ZERO>
__device__ __forceinline__ uint32_t clean_share(const Share& r, uint32_t tile, int chunk, int lane) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;
  uint32_t odd = 0;
  __syncwarp();
#pragma unroll 4
  for (int x = 0; x < 32 / kRows; ++x) {
    const int row = x * kRows + lane / kLanes;
    const uint32_t at = tile + piece_at<D>(chunk * 32 + row, lane % kLanes);
    if (ZERO && (row >= r.lim || (row & 16 ? r.off[1] : r.off[0]) < 0)) {
      store16(at, make_uint4(0, 0, 0, 0));
    } else if (row >= r.watch) {
      uint4 y = load16(at);
      if (finite_only<HALF>(y)) {
        odd |= 1u << row;
        store16(at, y);
      }
    }
  }
  return odd;
}

// -------------------------------------------------------------- values that are no finite numbers, seen by some rows only
// Adds to a row of sums (in memory, each times `to`) the weight of token t times its values that are no finite numbers.
// Runs only where such values lie among a block's new tokens; the weight is computed again, from the query row and the key.
template <int D, int TYPE>
__device__ __noinline__ void add_odd(const PromptParams& p, float* o, int32_t seq, int32_t t, int head, const __nv_bfloat16* q,
                                     float scale, float m, float to) {
  float x = 0.f;
  for (int d = 0; d < D; ++d) x = fmaf(__bfloat162float(q[d]), page_value<D, TYPE>(p.c, p.kv_heads, p.c.k_pages, seq, t, head, d), x);
  const float w = ex2_approx(x * scale - (m == -INFINITY ? 0.f : m)) * to;
  for (int d = 0; d < D; ++d) {
    const float v = page_value<D, TYPE>(p.c, p.kv_heads, p.c.v_pages, seq, t, head, d);
    if (!(fabsf(v) < INFINITY)) o[d] = fmaf(w, v, o[d]);
  }
}

// -------------------------------------------------------------- partial results
// 32 bytes, aligned to as many: whole sectors, where a lane has a row to itself
__device__ __forceinline__ void store32(void* dst, const uint32_t* x) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]),
               "r"(x[5]), "r"(x[6]), "r"(x[7])
               : "memory");
}
__device__ __forceinline__ void load32(float* x, const float* src) {
  asm volatile("ld.global.L1::no_allocate.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7])
               : "l"(src)
               : "memory");
}
template <int D>
__host__ __device__ constexpr int64_t slot_floats() { return 2 * BM * (D + 2); }
template <int D>
__device__ __forceinline__ float* slot_at(const PromptParams& p, int cta, int slot) {
  return p.parts + (static_cast<int64_t>(cta) * 2 + slot) * slot_floats<D>();
}

// A block's parts are joined in the order of the line: a = sum of w_x v_x, l = sum of w_x l_x with w_x = 2^(m_x - top) and
// top the largest m_x. A maximum of -inf stands for no score, or for NaN alone.
__device__ __forceinline__ float part_weight(float2 ml, float top) {
  return ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : ex2_approx(ml.x - top);
}
template <int D>
__device__ __forceinline__ const float* part_at(const PromptParams& p, int c0, int x) {
  return slot_at<D>(p, c0 + x, x == 0 ? 1 : 0);
}
template <int D>
__device__ __forceinline__ float2 part_ml(const PromptParams& p, int c0, int x, int row) {
  return __ldcg(reinterpret_cast<const float2*>(part_at<D>(p, c0, x) + 2 * BM * D) + row);
}

// Joins the n parts of a block, that of CTA c0 (slot 1) and of those behind it (slot 0): a warp per row, its lanes the dims.
// What it costs is the latency of the loads, so kJoinBatch of them are on their way: of as many rows, part by
// part, or, where a warp has few rows, of one row's parts.
constexpr int kJoinBatch = 8;
template <int D, bool ROWS>
__device__ __noinline__ void join_block(const PromptParams& p, const Block& k, int c0, int n, int warp, int lane) {
  constexpr int N = D / 32, B = kJoinBatch, R = ROWS ? B : 1;
  __threadfence();
  const int group = p.c.group, rows = k.ntok * group;
  for (int r0 = warp * R; r0 < rows; r0 += 8 * R) {
    int at[R];                                  // rows of the two tiles
    float top[R], sum[R], a[R][N];
#pragma unroll
    for (int y = 0; y < R; ++y) {
      const int r = min(r0 + y, rows - 1), tok = static_cast<int>(static_cast<uint32_t>(r) * p.group_magic >> 16);
      at[y] = tok >= p.tpt ? BM + r - p.tpt * group : r;
      top[y] = -INFINITY;
      sum[y] = 0.f;
#pragma unroll
      for (int z = 0; z < N; ++z) a[y][z] = 0.f;
    }
    if constexpr (ROWS) {
#pragma unroll 1
      for (int x = 0; x < n; ++x) {
        float m[R];
#pragma unroll
        for (int y = 0; y < R; ++y) m[y] = part_ml<D>(p, c0, x, at[y]).x;
#pragma unroll
        for (int y = 0; y < R; ++y) top[y] = fmaxf(top[y], m[y]);
      }
    } else {
      for (int x = lane; x < n; x += 32) top[0] = fmaxf(top[0], part_ml<D>(p, c0, x, at[0]).x);
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) top[0] = fmaxf(top[0], __shfl_xor_sync(0xffffffffu, top[0], s));
    }
#pragma unroll 1
    for (int x0 = 0; x0 < n; x0 += ROWS ? 1 : B) {
      float2 ml[B];
      float v[B][N];
#pragma unroll
      for (int y = 0; y < B; ++y) {
        const int x = ROWS ? x0 : min(x0 + y, n - 1), row = at[ROWS ? y : 0];
        ml[y] = part_ml<D>(p, c0, x, row);
        const float* src = part_at<D>(p, c0, x) + row * D;
        if constexpr (N == 4) {
          const float4 z = __ldcg(reinterpret_cast<const float4*>(src) + lane);
          v[y][0] = z.x; v[y][1] = z.y; v[y][2] = z.z; v[y][3] = z.w;
        } else {
          const float2 z = __ldcg(reinterpret_cast<const float2*>(src) + lane);
          v[y][0] = z.x; v[y][1] = z.y;
        }
      }
#pragma unroll
      for (int y = 0; y < B; ++y) {
        const int q = ROWS ? y : 0;
        if (!ROWS && x0 + y >= n) break;
        const float w = part_weight(ml[y], top[q]);
        sum[q] = fmaf(w, ml[y].y, sum[q]);
#pragma unroll
        for (int z = 0; z < N; ++z) a[q][z] = fmaf(w, v[y][z], a[q][z]);
      }
    }
#pragma unroll
    for (int y = 0; y < R; ++y) {
      const int r = r0 + y;
      if (r >= rows) break;
      const int tok = static_cast<int>(static_cast<uint32_t>(r) * p.group_magic >> 16), hh = r - tok * group;
      const float inv = sum[y] == 0.f ? 0.f : 1.f / sum[y];
      const int64_t out = (static_cast<int64_t>(p.row0[k.i]) + k.tok0 + tok) * p.c.n_heads + k.h * group + hh;
      uint32_t* o = reinterpret_cast<uint32_t*>(p.o + out * D + lane * N);
      auto of = [&](int z) { return sum[y] == 0.f ? 0.f : a[y][z] * inv; };     // no weight: 0, whatever the values are
      o[0] = pack_bf16x2(of(0), of(1));
      if constexpr (N == 4) o[1] = pack_bf16x2(of(2), of(3));
      if (lane == 0 && p.lse) p.lse[out] = sum[y] == 0.f ? -INFINITY : (top[y] + log2f(sum[y])) * kLn2;
    }
  }
}

// place of dim i (of 8) among the columns of a tile: 4-bit words decode to the pairs (0,4) (1,5) (2,6) (3,7)
template <int TYPE>
__device__ __forceinline__ constexpr int column_of(int i) {
  return TYPE == SR_PAGE_INT4 ? (i & ~7) + ((i & 3) * 2 + ((i >> 2) & 1)) : i;
}

template <int D, int TYPE>
__global__ void __launch_bounds__(kThreads, 1) paged_prompt_kernel(const __grid_constant__ PromptParams p) {
  using C = Cfg<D, TYPE>;
  grid_dep_launch_dependents();
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw;                  // the kernel has no other shared memory: it begins on a multiple of 1024
  uint8_t* sQ = smem;
  uint8_t* sKV = smem + C::kSmemQ;
  Bars* bars = reinterpret_cast<Bars*>(smem + C::kSmemQ + C::kSmemKV);
  Setup* setup = reinterpret_cast<Setup*>(sKV);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const PagedView& c = p.c;
  WaitCtx wc{&bars->abort, c.err_word, kTimeoutNs};

  if (threadIdx.x == 0) {
    mbar_init(&bars->q_raw, kQWarps);
    mbar_init(&bars->q_full, C::kHalf ? 8 : kQWarps);
    mbar_init(&bars->q_empty, 1);
    mbar_init(&bars->q_seen, 8);
    for (int s = 0; s < 8; ++s) {
      mbar_init(&bars->kv_full[s], C::kPerTile);
      mbar_init(&bars->kv_empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars->s_full[t], 1);
      mbar_init(&bars->p_half[t], 4);
      mbar_init(&bars->p_full[t], 4);
      mbar_init(&bars->o_done[t], 1);
    }
    mbar_init(&bars->x_full, BM);
    mbar_init(&bars->x_empty, BM);
    mbar_init(&bars->part_done, 2 * BM);
    mbar_init(&bars->part_last, 1);
    mbar_init(&bars->drain, 1);
    for (int s = 0; s < kLoadWarps; ++s) mbar_init(&bars->fixed[s], 1);
    for (int s = 0; s < kTileSlots; ++s) {
      mbar_init(&bars->tile_full[s], 1);
      mbar_init(&bars->tile_empty[s], C::kPerTile);
    }
    bars->abort = 0;
    bars->bad = 0;
    mbar_fence_init();
  }
  if (warp == 0) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  if (threadIdx.x < p.n) setup->per_head[threadIdx.x] = 0;
  if (threadIdx.x == 0) setup->none = 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dep_wait();
  const uint32_t tmem = bars->tmem_base;

  // ---- the line of steps: units of each sequence's blocks for one head, then of the sequences one after the other
  {
    if (threadIdx.x < p.n) setup->len[threadIdx.x] = seq_length(p, threadIdx.x);
    __syncthreads();
    for (int x0 = warp * 32; x0 < p.blocks; x0 += kThreads) {
      const int x = min(x0 + lane, p.blocks - 1), lo = p.n == 1 ? 0 : seq_of_block(p, x);
      Block k;
      k.i = lo;
      k.b = x - p.blk0[lo];
      set_block(p, k, setup->len[lo]);
      // one addition for a warp's blocks of a sequence: on shared memory 64 bits are added one after the other
      const uint32_t same = __match_any_sync(0xffffffffu, lo);
      const uint32_t units = __reduce_add_sync(same, x0 + lane < p.blocks ? static_cast<uint32_t>(units_of(k)) : 0u);
      if (lane == __ffs(same) - 1) atomicAdd(&setup->per_head[lo], static_cast<unsigned long long>(units));
      if (k.steps == 0) setup->none = 1;
    }
    __syncthreads();
    for (int x = setup->none ? blockIdx.x : p.blocks; x < p.blocks; x += gridDim.x) {
      Block k;
      k.i = seq_of_block(p, x);
      k.b = x - p.blk0[k.i];
      set_block(p, k, setup->len[k.i]);
      if (k.steps > 0) continue;
      const int64_t row = static_cast<int64_t>(p.row0[k.i]) + k.tok0;
      uint4* o = reinterpret_cast<uint4*>(p.o + row * c.n_heads * D);
      for (int y = threadIdx.x; y < k.ntok * c.n_heads * (D / 8); y += kThreads) o[y] = make_uint4(0, 0, 0, 0);
      for (int y = threadIdx.x; y < k.ntok * c.n_heads; y += kThreads)
        if (p.lse) p.lse[row * c.n_heads + y] = -INFINITY;
    }
    if (warp == 0) {
      constexpr int kPer = kMaxPagedSeqs / 32;
      int64_t mine = 0;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int i = lane * kPer + k;
        mine += i < p.n ? static_cast<int64_t>(setup->per_head[i]) * c.n_kv : 0;
      }
      int64_t incl = mine;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, s);
        if (lane >= s) incl += y;
      }
      int64_t at = incl - mine;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int i = lane * kPer + k;
        if (i <= p.n) setup->cum[i] = at;
        at += i < p.n ? static_cast<int64_t>(setup->per_head[i]) * c.n_kv : 0;
      }
      if (lane == 31 && p.n == kMaxPagedSeqs) setup->cum[p.n] = at;
      __syncwarp();
      const int64_t T = setup->cum[p.n];
      Start s;
      s.left = 0;
      s.share = s.rest = s.u = 0;
      s.i = s.h = s.b = s.s0 = 0;
      const int64_t ctas = min(static_cast<int64_t>(gridDim.x), T);
      if (static_cast<int64_t>(blockIdx.x) < ctas) {
        s.share = div_pos(T, ctas);
        s.rest = T - s.share * ctas;
        const int64_t u0 = blockIdx.x * s.share + min(static_cast<int64_t>(blockIdx.x), s.rest);
        s.left = s.share + (static_cast<int64_t>(blockIdx.x) < s.rest ? 1 : 0);
        int lo = 0, hi = p.n - 1;
        while (lo < hi) {
          const int mid = (lo + hi + 1) / 2;
          if (setup->cum[mid] <= u0) lo = mid; else hi = mid - 1;
        }
        const int64_t per_head = static_cast<int64_t>(setup->per_head[lo]);
        int64_t within = u0 - setup->cum[lo];
        s.i = lo;
        s.h = static_cast<int>(div_pos(within, per_head));
        within -= s.h * per_head;
        const int32_t len = setup->len[lo];
        const int nb = blocks_of(p, lo);
        for (int b0 = 0; b0 < nb; b0 += 32) {          // the block that holds unit `within` of this head's
          Block k;
          k.i = lo;
          k.b = b0 + lane;
          int64_t units = 0;
          if (k.b < nb) {
            set_block(p, k, len);
            units = units_of(k);
          }
          int64_t run = units;
#pragma unroll
          for (int x = 1; x < 32; x <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, run, x);
            if (lane >= x) run += y;
          }
          const uint32_t past = __ballot_sync(0xffffffffu, run > within);
          if (past) {
            const int l = __ffs(past) - 1;
            s.b = b0 + l;
            within -= __shfl_sync(0xffffffffu, run - units, l);
            break;
          }
          within -= __shfl_sync(0xffffffffu, run, 31);
        }
        // `within` the block: its cost comes before its steps
        const int64_t before = max(kItemCost - within, static_cast<int64_t>(0));
        s.left -= before;
        s.s0 = static_cast<int32_t>(max(within - kItemCost, static_cast<int64_t>(0)));
        s.u = u0 + before - s.s0;
      }
      if (lane == 0) bars->start = s;
    }
    fence_proxy_async_smem();        // the stages, which held the set-up, may be filled by tensor copies
    __syncthreads();
  }

  if (warp >= kLoadWarp0) {
    regs_dec<C::kRegsLoad>();
    // ------------------------------------------------------------ keys and values
    const int team = (warp - kLoadWarp0) / C::kPerTile, member = (warp - kLoadWarp0) % C::kPerTile;
    const uint32_t skv = smem_u32(sKV);
    bool ok = true;
    int n = team;                        // the tile that this team loads next
    auto acquire = [&](int tile) {       // its stage
      if (ok && tile >= C::kStages)
        ok = __all_sync(0xffffffffu, wait_bounded(&bars->kv_empty[tile % C::kStages], (tile / C::kStages - 1) & 1u, wc, 1));
    };
    auto ready = [&](int tile) -> const Tile& {
      if (ok) ok = __all_sync(0xffffffffu, wait_bounded(&bars->tile_full[tile % kTileSlots], (tile / kTileSlots) & 1u, wc, 11));
      return bars->tile[tile % kTileSlots];
    };
    auto release = [&](int tile) {       // its description has been read
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->tile_empty[tile % kTileSlots]);
    };
    auto share = [&](Share& r, const Tile& d, int chunk) {
      r.off[0] = d.off[2 * chunk];
      r.off[1] = d.off[2 * chunk + 1];
      r.lim = d.lim - chunk * 32;
      r.watch = d.watch - chunk * 32;
      r.head = d.head;
      r.meta = d.meta;
    };
    auto note = [&](const Share& r, int chunk, uint32_t odd) {
      if (!r.values() || r.watch >= 32 + (3 - chunk) * 32) return;        // of tiles that some rows do not see whole
      odd = __reduce_or_sync(0xffffffffu, odd);
      if (lane == 0) bars->flags[r.meta >> 1 & 7][chunk][min(r.meta >> 8, kFlagTiles - 1)] = odd;
    };
    auto publish = [&](int tile) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->kv_full[tile % C::kStages]);
    };
    // (few instructions in each role's loop: they share the instruction cache with the softmax groups, and a kernel whose
    // loops were unrolled further took up to a quarter longer)
    if constexpr (TYPE == SR_PAGE_BF16) {
      const uint64_t policy = l2_policy_evict_last();
      const bool wide = c.page_tokens % 32 == 0;       // boxes of 32 rows, else of 16
      uint32_t fixes = 0;
      for (;; n += C::kTeams) {
        const Tile& d = ready(n);
        if (!ok || d.meta < 0) break;
        acquire(n);
        if (!ok) break;
        uint64_t* full = &bars->kv_full[n % C::kStages];
        uint8_t* tile = sKV + n % C::kStages * C::kTileBytes;
        // Keys that no row sees may be anything: their scores are replaced. Values are finished here where some are no tokens,
        // or not seen by all rows, once the copies have landed on a barrier of this warp's own.
        const bool values = d.meta & 1;
        bool fix = values && (d.lim < BN || d.watch < BN);
        uint32_t held = 0;               // copies, by 32 tokens or by 16
#pragma unroll
        for (int x = 0; x < 8; ++x)
          if (d.off[x] >= 0) held |= 1u << x;
        fix |= values && held != 0xFFu;
        if (wide) held &= 0x55u;         // a copy of 32 tokens begins with its first 16
        uint64_t* landed = fix ? &bars->fixed[team] : full;
        if (lane == 0) {
          mbar_arrive_expect_tx(landed, __popc(held) * (wide ? 32 : 16) * D * 2);
          const CUtensorMap* map = values ? &p.vmap : &p.kmap;
          const int head = d.head * D;
#pragma unroll 1
          for (uint32_t left = held; left; left &= left - 1) {
            const int x = __ffs(left) - 1;
#pragma unroll
            for (int a = 0; a < C::kAtoms; ++a)
              tma_load_2d(tile + a * C::kAtomBytes + x * 16 * 128, map, landed, head + a * 64, static_cast<int>(d.off[x]), policy);
          }
        }
        __syncwarp();
        if (fix) {
          ok = __all_sync(0xffffffffu, wait_bounded(landed, fixes & 1u, wc, 13));
          ++fixes;
          if (!ok) break;
#pragma unroll 1
          for (int x = 0; x < 4; ++x) {
            Share r;
            share(r, d, x);
            note(r, x, clean_share<D, false, true>(r, smem_u32(tile), x, lane));
          }
          publish(n);
        }
        release(n);
      }
      // copies that nobody waited for (after an error) land before shared memory is given back
      if (!ok || bars->abort)
        for (int k = 1; k <= C::kStages; ++k)
          if (n - k >= 0 && (n - k) % C::kTeams == team)
            wait_drain(&bars->kv_full[(n - k) % C::kStages], ((n - k) / C::kStages) & 1u, kTimeoutNs);
      if ((!ok || bars->abort) && fixes > 0) wait_drain(&bars->fixed[team], (fixes - 1) & 1u, kTimeoutNs);
    } else {
      // a share's bytes are on their way in registers: as soon as one of them is stored the next share's follows it
      const DecodeMasks masks = decode_masks();
      Raw<D, TYPE> raw;
      Source<D, TYPE> from;
      Share r;
      int sub = 0, at = n;                 // of tile n, the next to be taken; the tile of the share in hand
      bool more = true;
      auto next = [&]() {
        r.off[0] = r.off[1] = -1;
        r.lim = 0;
        r.meta = 0;
        if (more) {
          const Tile& d = ready(n);
          more = ok && d.meta >= 0;
          if (more) share(r, d, member * C::kSubs + sub);
        }
        if (more && ++sub == C::kSubs) {
          release(n);
          sub = 0;
          n += C::kTeams;
        }
        from.set(r, c, p.kv_heads, lane);
      };
      int done = 0;                        // shares of the tile in hand that are stored
      next();
#pragma unroll
      for (int i = 0; i < Raw<D, TYPE>::kVec; ++i) from.load(raw, i, p.kv_heads, lane);
      bool have = more;
      while (have) {
        const Share mine = r;
        const int chunk = member * C::kSubs + done;
        next();
        have = more;
        if (done == 0) acquire(at);
        if (!ok) break;
        const uint32_t tile = skv + at % C::kStages * C::kTileBytes;
#pragma unroll
        for (int i = 0; i < Raw<D, TYPE>::kVec; ++i) {
          store_raw<D, TYPE>(raw, i, tile, chunk, lane, masks);
          from.load(raw, i, p.kv_heads, lane);
        }
        note(mine, chunk, mine.watched() ? clean_share<D, true, false>(mine, tile, chunk, lane) : 0);
        if (++done == C::kSubs) {
          publish(at);
          done = 0;
          at += C::kTeams;
        }
      }
    }
  } else if (warp >= kMmaWarp) {
    regs_dec<C::kRegsOther>();
    bool ok = true;
    uint32_t items = 0;
    if (warp == kPlanWarp) {
      // ---------------------------------------------------------- the order of the tiles, and where their tokens lie
      // four tiles at a time, lane 8 q + g with group g of tile q; the entries of the next four are on their way
      TileWalk walk(p, bars->start);
      TileRef r, nr;
      int32_t page = 0, npage = 0;
      const int g = lane & 7, mine = lane / 8;
      int count = 0, ncount = 0;                   // tiles of the four that there are
      auto next = [&]() {
        ncount = 0;
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          TileRef t;
          if (!walk.next(t, p)) break;
          if (mine == q) nr = t;
          ++ncount;
        }
        const int32_t tok = nr.tok0 + g * 16;
        if (mine < ncount)
          npage = tok < nr.lim ? __ldg(c.table + static_cast<int64_t>(nr.seq) * c.max_pages + page_of_group(tok >> 4, c.magic)) : 0;
      };
      for (int n = -4; ok; n += 4) {
        r = nr;
        page = npage;
        count = ncount;
        if (count == 4 || n < 0) next(); else ncount = 0;
        if (n < 0) continue;
        // behind the last tile an end for each team
#pragma unroll 1
        for (int q = 0; ok && q < 4; ++q)
          if (n + q >= kTileSlots)
            ok = __all_sync(0xffffffffu, wait_bounded(&bars->tile_empty[(n + q) % kTileSlots], ((n + q) / kTileSlots - 1) & 1u, wc, 12));
        if (!ok) break;
        Tile& d = bars->tile[(n + mine) % kTileSlots];
        if (mine < count) {
          const int32_t tok = r.tok0 + g * 16;
          int64_t off = -1;
          if (tok < r.lim) {
            if (page >= 0 && page < c.n_pages) {
              const int32_t slot_in = tok - page_of_group(tok >> 4, c.magic) * c.page_tokens;
              if constexpr (TYPE == SR_PAGE_INT4) {
                off = record_at(page, slot_in, r.head, p.kv_heads, c.page_tokens, D);
              } else {
                off = static_cast<int64_t>(page) * c.page_tokens + slot_in;
                if constexpr (TYPE == SR_PAGE_E4M3) off = (off * p.kv_heads + r.head) * D;
              }
            } else {
              atomicCAS(c.err_word, 0, SR_DEVERR_BAD_PAGE);
              bars->bad = 1;
            }
          }
          d.off[g] = off;
          if (g == 0) {
            d.lim = min(r.lim - r.tok0, BN);
            d.watch = r.watch == INT32_MAX ? BN : min(max(r.watch - r.tok0, 0), BN);
            d.head = r.head;
            d.meta = r.meta;
          }
        } else if (g == 0) {
          d.meta = -1;
        }
        __syncwarp();
        if (g == 0) mbar_arrive(&bars->tile_full[(n + mine) % kTileSlots]);
        if (count < 4) {
          // as many ends again, for the teams whose turn came before the last tile
          if (count == 0) break;
          r.lim = 0;
          nr = r;
          ncount = 0;
        }
      }
    } else if (warp >= kQWarp0) {
      Walker walk(p, bars->start);
      // ---------------------------------------------------------- queries
      constexpr int kLanes = D / 8, kRows = 32 / kLanes;      // lanes of a row, rows per load
      const int w = warp - kQWarp0;
      const uint32_t sq = smem_u32(sQ);
      const int group = c.group;
      while (walk.next()) {
        const Block& k = walk.k;
        if (items > 0) {
          // the MMAs are done with the last block's, and its scales are read
          ok = __all_sync(0xffffffffu, wait_bounded(&bars->q_empty, (items - 1) & 1u, wc, 2) &&
                                           wait_bounded(&bars->q_seen, (items - 1) & 1u, wc, 2));
          if (!ok) break;
        }
        if (w == 0 && lane == 0) {
          const Start& s = bars->start;
          Record r{k, 0, 1, false};
          if (k.s0 > 0 || k.s1 < k.steps) {
            r.c0 = owner_of(walk.u, s.share, s.rest);
            r.parts = owner_of(walk.u + k.steps - 1, s.share, s.rest) - r.c0 + 1;
            int32_t done;
            asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(done) : "l"(p.arrivals + r.c0) : "memory");
            r.last = done == r.parts - 1;
          }
          bars->rec[items & 1] = r;
        }
        const int tiles = k.split ? 1 : 2;
        const int64_t row00 = static_cast<int64_t>(p.row0[k.i]) + k.tok0;
        // this warp's half of each tile's rows, all copies in flight together
        for (int t = 0; t < tiles; ++t) {
          const uint32_t tile = sq + t * C::kTileBytes;
          const __nv_bfloat16* src = p.q + (row00 * c.n_heads + k.h * group) * D + lane % kLanes * 8;
#pragma unroll 4
          for (int x = w * (BM / kQWarps) + lane / kLanes; x < (w + 1) * (BM / kQWarps); x += kRows) {
            const int tok = static_cast<int>(static_cast<uint32_t>(x) * p.group_magic >> 16);
            const int token = t * p.tpt + tok, hh = x - tok * group;
            const bool there = tok < p.tpt && token < k.ntok;
            copy16_or_zero(tile + piece_at<D>(x, lane % kLanes), src + (there ? (static_cast<int64_t>(token) * c.n_heads + hh) * D : 0), there);
          }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        if constexpr (!C::kHalf) fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(C::kHalf ? &bars->q_raw : &bars->q_full);
        ++items;
      }
      // the end: a record of no block, once the last one but one has been read
      if (ok && items > 0) ok = __all_sync(0xffffffffu, wait_bounded(&bars->q_seen, (items - 1) & 1u, wc, 2));
      if (ok && w == 0 && lane == 0) bars->rec[items & 1].k.i = -1;
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(C::kHalf ? &bars->q_raw : &bars->q_full);
    } else {
      // ---------------------------------------------------------- MMA issuer (the warp in step, one lane issues)
      Walker walk(p, bars->start);
      const uint32_t leader = elect_one();
      const uint32_t sq = smem_u32(sQ), skv = smem_u32(sKV), tm = __shfl_sync(0xffffffffu, tmem, 0);
      bool issued = false;
      int stage = 0;
      uint32_t phase = 0, pb = 0;               // ring position; bit t: parity of group t's next P
      auto take = [&]() -> int {                // the next tile of the ring
        const int s = stage;
        if (ok) ok = __all_sync(0xffffffffu, wait_bounded(&bars->kv_full[s], phase, wc, 3));
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1u;
        }
        return s;
      };
      auto qk = [&](int t, bool split, int s) {
        const uint32_t qt = sq + (split ? 0 : t) * C::kTileBytes, kt = skv + s * C::kTileBytes;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk / 4) * C::kAtomBytes + (kk % 4) * 32;
          mma_ss_w(tm + t * BN, sdesc_sw128(qt + off, 16, 1024), sdesc_sw128(kt + off, 16, 1024), C::kIdescS, kk > 0 ? 1u : 0u, leader);
        }
        tc_commit_w(&bars->s_full[t], leader);
        issued = true;
      };
      auto pv = [&](int t, int s, bool acc) {
        const uint32_t vt = skv + s * C::kTileBytes;
        const uint32_t par = pb >> t & 1u;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (ok) ok = __all_sync(0xffffffffu, wait_bounded(half == 0 ? &bars->p_half[t] : &bars->p_full[t], par, wc, 4));
          if (!ok) return;
          tc_fence_after();
#pragma unroll
          for (int kk = half * 4; kk < half * 4 + 4; ++kk)
            mma_ts_w(tm + 256 + t * 128, tm + t * BN + kk * 8, sdesc_sw128(vt + kk * 16 * 128, C::kAtomBytes, 1024), C::kIdescPV,
                     (acc || kk > 0) ? 1u : 0u, leader);
        }
        pb ^= 1u << t;
      };
      while (walk.next()) {
        const Block& k = walk.k;
        ok = __all_sync(0xffffffffu, wait_bounded(&bars->q_full, items & 1u, wc, 3));
        if (!ok) break;
        // the same in all lanes, and known to be
        const int n = __shfl_sync(0xffffffffu, k.s1 - k.s0, 0), n1 = __shfl_sync(0xffffffffu, k.count(1), 0);
        const bool split = __shfl_sync(0xffffffffu, k.split ? 1 : 0, 0) != 0;
        int v = 0, kt = 0;
#pragma unroll 1
        for (int j = 0; j <= n && ok; ++j) {
#pragma unroll C::kUnrollT
          for (int t = 0; t < 2; ++t) {
            const int cnt = t == 0 ? n : n1;
            if (j > 0 && j <= cnt) {
              if (split || t == 0) v = take();
              if (!ok) break;
              tc_fence_after();
              pv(t, v, j > 1);
              if (!ok) break;
              if (j == cnt) tc_commit_w(&bars->o_done[t], leader);
              if (split || t == 1) tc_commit_w(&bars->kv_empty[v], leader);
            }
            if (j < cnt) {
              if (split || t == 0) kt = take();
              if (!ok) break;
              tc_fence_after();
              qk(t, split, kt);
              if (split || t == 1) tc_commit_w(&bars->kv_empty[kt], leader);
            }
          }
          if (ok && j == n - 1) tc_commit_w(&bars->q_empty, leader);
        }
        ++items;
        if (!ok) break;
      }
      if ((!ok || bars->abort) && issued) {
        // no tensor-core work may still be running when TMEM is released
        tc_commit_w(&bars->drain, leader);
        wait_drain(&bars->drain, 0, kTimeoutNs);
      }
    }
  } else {
    regs_inc<kRegsSoftmax>();
    // ------------------------------------------------------------ softmax groups
    const int t = warp / 4, row = threadIdx.x % BM;
    const uint32_t lane_base = static_cast<uint32_t>((warp % 4) * 32) << 16;
    const uint32_t t_s = tmem + lane_base + t * BN, t_o = tmem + lane_base + 256 + t * 128;
    const int group = c.group;
    const int tr = static_cast<int>(static_cast<uint32_t>(row) * p.group_magic >> 16), hh = row - tr * group;
    bool ok = true;
    uint32_t items = 0, sb = 0, od[2] = {0, 0}, nx = 0, cuts = 0;
    while (ok) {
      ok = __all_sync(0xffffffffu, wait_bounded(C::kHalf ? &bars->q_raw : &bars->q_full, items & 1u, wc, 5));
      if (!ok) break;
      const Record& rec = bars->rec[items & 1];      // there until every warp has begun the next block
      const Block& k = rec.k;
      if (k.i < 0) break;
      const int kv = static_cast<int>(static_cast<uint32_t>(k.h) * p.head_magic >> 22);
      float sl2 = c.scale_log2 * C::kDecodedBy * (c.kv_exp ? exp2f(static_cast<float>(c.kv_exp[kv])) : 1.f);
      if constexpr (C::kHalf) {
        // the query row becomes fp16 in place, scaled by a power of two to a largest element in [1, 2)
        int e = 0;
        if (t == 0 || !k.split) {
          const uint32_t tile = smem_u32(sQ) + t * C::kTileBytes;
          uint32_t top = 0;                         // of |x|, as bf16 bits: their order, NaN last
#pragma unroll 4
          for (int y = 0; y < D / 8; ++y) {
            const uint4 v = load16(tile + piece_at<D>(row, y));
            top = __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
          }
          const float most = __uint_as_float(max(top & 0xFFFFu, top >> 16) << 16);
          e = most > 0.f && most < INFINITY ? max(ilogbf(most), -120) : 0;
          const float down = ldexpf(1.f, -e);
#pragma unroll 4
          for (int y = 0; y < D / 8; ++y) {
            const uint32_t at = tile + piece_at<D>(row, y);
            const uint4 v = load16(at);
            auto half = [&](uint32_t z) {
              const __half2 h = __floats2half2_rn(__uint_as_float(z << 16) * down, __uint_as_float(z & 0xFFFF0000u) * down);
              return *reinterpret_cast<const uint32_t*>(&h);
            };
            const uint32_t h[4] = {half(v.x), half(v.y), half(v.z), half(v.w)};
            if constexpr (TYPE == SR_PAGE_INT4)
              store16(at, make_uint4(__byte_perm(h[0], h[2], 0x5410), __byte_perm(h[0], h[2], 0x7632),
                                     __byte_perm(h[1], h[3], 0x5410), __byte_perm(h[1], h[3], 0x7632)));
            else
              store16(at, make_uint4(h[0], h[1], h[2], h[3]));
          }
          if (k.split) bars->qexp[row] = static_cast<int8_t>(e);
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->q_full);
        if (k.split && t == 1) {
          ok = __all_sync(0xffffffffu, wait_bounded(&bars->q_full, items & 1u, wc, 5));
          if (!ok) break;
          e = bars->qexp[row];
        }
        sl2 *= ldexpf(1.f, e);
      }
      sl2 = fmaxf(sl2, 0x1p-126f);
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->q_seen);
      const int token = (k.split ? 0 : t * p.tpt) + tr;          // of the block's
      const bool live = tr < p.tpt && token < k.ntok;
      const int32_t lim = !live ? k.lim : p.causal ? max(k.base + k.tok0 + token + 1, 0) : k.lim;
      const int32_t* table = c.table + static_cast<int64_t>(p.id[k.i]) * c.max_pages;
      const int cnt = k.count(t), step = k.split ? 2 * BN : BN;
      int32_t ks = k.tile(t, 0) * BN;                 // first token of the key tile
      const int32_t seen = k.lim;
      float m = -INFINITY, l = 0.f;
      const float2 sl2x2 = make_float2(sl2, sl2);
      for (int j = 0; j < cnt; ++j) {
        const int valid = lim - ks;
        ks += step;
        ok = __all_sync(0xffffffffu, wait_bounded(&bars->s_full[t], (sb + static_cast<uint32_t>(j)) & 1u, wc, 5));
        if (!ok) break;
        tc_fence_after();
        const bool bad = *reinterpret_cast<volatile int*>(&bars->bad);
        if (bad || __any_sync(0xffffffffu, valid < BN)) {
          // keys that the row does not see, or that have no page (once the planning warp has met an entry that is none of
          // the pool, in whatever tile): in tensor memory, 32 at a time, which keeps the common path short
          uint32_t there = 0xFFu;
          if (bad) {
            const int32_t tok = ks - step + (lane & 7) * 16;
            const int32_t page = tok < seen ? __ldg(table + page_of_group(tok >> 4, c.magic)) : 0;
            there = __ballot_sync(0xffffffffu, page >= 0 && page < c.n_pages);
          }
#pragma unroll 1
          for (int x = 0; x < 4; ++x) {
            uint32_t z[32];
            tmem_ld32(t_s + x * 32, z);
            tmem_wait_ld();
            tmem_fix(z);
            const int left = valid - x * 32;
            uint32_t keep = left >= 32 ? 0xffffffffu : left <= 0 ? 0u : (1u << left) - 1u;
            keep &= (there >> (2 * x) & 1u ? 0x0000FFFFu : 0u) | (there >> (2 * x) & 2u ? 0xFFFF0000u : 0u);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!(keep >> i & 1u)) z[i] = 0xFF800000u;
            tmem_st32(t_s + x * 32, z);
          }
          tmem_wait_st();
        }
        uint32_t rr[4][32];
#pragma unroll
        for (int x = 0; x < 4; ++x) tmem_ld32(t_s + x * 32, rr[x]);
        tmem_wait_ld();
#pragma unroll
        for (int x = 0; x < 4; ++x) tmem_fix(rr[x]);
        float* s = reinterpret_cast<float*>(&rr[0][0]);
        float a0 = fmaxf(s[0], s[1]), a1 = fmaxf(s[2], s[3]), a2 = fmaxf(s[4], s[5]), a3 = fmaxf(s[6], s[7]);
#pragma unroll
        for (int i = 8; i < BN; i += 8) {
          a0 = fmax3(a0, s[i], s[i + 1]);
          a1 = fmax3(a1, s[i + 2], s[i + 3]);
          a2 = fmax3(a2, s[i + 4], s[i + 5]);
          a3 = fmax3(a3, s[i + 6], s[i + 7]);
        }
        const float top = fmax3(a0, a1, fmaxf(a2, a3)) * sl2 - C::kLift;
        float f = 1.f;                    // factor that takes O and l to the new reference
        const bool rescale = __any_sync(0xffffffffu, top > m + C::kSlack);
        if (rescale) {
          const float m1 = fmaxf(m, top);
          f = m == -INFINITY ? 0.f : ex2_approx(m - m1);
          m = m1;
        }
        const float neg = m == -INFINITY ? 0.f : -m;
        const float2 negm = make_float2(neg, neg);
        float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          uint32_t pk[16];
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            const int i = x * 32 + 2 * q;
            const float2 y = __ffma2_rn(make_float2(s[i], s[i + 1]), sl2x2, negm);
            const float2 e = make_float2(ex2_approx(y.x), ex2_approx(y.y));
            acc[q % 4] = __fadd2_rn(acc[q % 4], e);
            if constexpr (C::kHalf) {
              const __half2 h = __floats2half2_rn(e.x, e.y);
              pk[q] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
              pk[q] = pack_bf16x2(e.x, e.y);
            }
          }
          tmem_st16(t_s + x * 16, pk);
          if (x == 1) {
            if (rescale && j > 0) {
              // O was last written by the last step's product, which the commit behind S covers
#pragma unroll 1
              for (int q = 0; q < D / 32; ++q) {
                uint32_t o[32];
                tmem_ld32(t_o + q * 32, o);
                tmem_wait_ld();
                tmem_fix(o);
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                tmem_st32(t_o + q * 32, o);
              }
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->p_half[t]);
          }
        }
        const float2 s01 = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
        l = l * f + (s01.x + s01.y);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->p_full[t]);
      }
      if (!ok) break;
      sb += static_cast<uint32_t>(cnt);

      // ---- the block's end
      const bool whole = k.s0 == 0 && k.s1 == k.steps;
      bool joined = false;
      const uint32_t w0 = od[0], w1 = od[1];
      const bool merge = k.split && k.count(1) > 0;
      od[0] += 1;
      od[1] += !k.split || merge ? 1u : 0u;
      const int slot = items % kFlagSlots;
      if (k.split && t == 1) {
        // hand (m, l) to group 0 and wait until it has read them and O_1
        bars->xm[row] = cnt > 0 ? m : -INFINITY;
        bars->xl[row] = cnt > 0 ? l : 0.f;
        mbar_arrive(&bars->x_full);
        ok = __all_sync(0xffffffffu, wait_bounded(&bars->x_empty, nx & 1u, wc, 9));
        ++nx;
        if (!ok) break;
        joined = bars->joined;
      } else {
        if (k.split) ok = wait_bounded(&bars->x_full, nx & 1u, wc, 9);
        ok = ok && wait_bounded(&bars->o_done[t], (t == 0 ? w0 : w1) & 1u, wc, 6);
        if (merge) ok = ok && wait_bounded(&bars->o_done[1], w1 & 1u, wc, 6);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        float f0 = 1.f, f1 = 0.f;
        if (merge) {
          const float m1 = bars->xm[row], l1 = bars->xl[row];
          const float mm = fmaxf(m, m1);
          f0 = m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : ex2_approx(m - mm);
          f1 = m1 == -INFINITY ? (l1 == 0.f ? 0.f : 1.f) : ex2_approx(m1 - mm);
          l = l * f0 + l1 * f1;
          m = mm;
        }
        // (the values' loading came before the products that o_done stands for)
        const int f_lo = k.split ? 2 * k.s0 : k.s0, f_hi = k.split ? min(2 * k.s1, k.tiles) : k.s1, f_0 = k.lim_min / BN;
        uint32_t odd = 0;
        if (p.causal)
#pragma unroll 1
          for (int x = max(f_lo, f_0); x < f_hi; ++x)
            for (int y = 0; y < 4; ++y) odd |= bars->flags[slot][y][min(x - f_0, kFlagTiles - 1)];
        const float vscale = C::kDecodedBy * (c.kv_exp ? exp2f(static_cast<float>(c.kv_exp[p.kv_heads + kv])) : 1.f);
        // a block whose other parts are there is joined on the way, as join_block would
        const int c0 = rec.c0, parts = rec.parts, me = static_cast<int>(blockIdx.x) - c0;
        const bool join = !whole && rec.last && !odd;
        joined = join;
        const float to = whole ? (l == 0.f ? 0.f : vscale / l) : vscale;
        const int prow = (k.split ? 0 : t) * BM + row;
        float top = m, sum = 0.f, inv = 0.f;
        if (join) {
          for (int x = 0; x < parts; ++x)
            if (x != me) top = fmaxf(top, part_ml<D>(p, c0, x, prow).x);
          for (int x = 0; x < parts; ++x) {
            const float2 ml = x == me ? make_float2(m, l) : part_ml<D>(p, c0, x, prow);
            sum = fmaf(part_weight(ml, top), ml.y, sum);
          }
          inv = sum == 0.f ? 0.f : 1.f / sum;
        }
        const int64_t out = (static_cast<int64_t>(p.row0[k.i]) + k.tok0 + token) * c.n_heads + k.h * group + hh;
        // a whole block with odd values goes through the slot too (free: only the last block can be cut behind it), since
        // add_odd reads the query row, whose place the output may take
        float* part = slot_at<D>(p, blockIdx.x, k.s0 == 0 ? 1 : 0) + prow * D;
#pragma unroll 1
        for (int x = 0; x < D / 32; ++x) {
          uint32_t o[32];
          tmem_ld32(t_o + x * 32, o);
          tmem_wait_ld();
          tmem_fix(o);
          float* of = reinterpret_cast<float*>(o);
          if (merge) {
            uint32_t o1[32];
            tmem_ld32(tmem + lane_base + 256 + 128 + x * 32, o1);
            tmem_wait_ld();
            tmem_fix(o1);
            // (a factor of zero, too: both groups' sums have been written, and a NaN among them is one that the row sees)
#pragma unroll
            for (int i = 0; i < 32; ++i) of[i] = fmaf(__uint_as_float(o1[i]), f1, of[i] * f0);
          }
          float y[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) y[i] = of[column_of<TYPE>(i)] * to;
          if (join && live) {
            float a[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) a[i] = 0.f;
#pragma unroll 1
            for (int z = 0; z < parts; ++z) {
              const float2 ml = z == me ? make_float2(m, l) : part_ml<D>(p, c0, z, prow);
              const float w = part_weight(ml, top);
              if (z == me) {
#pragma unroll
                for (int i = 0; i < 32; ++i) a[i] = fmaf(w, y[i], a[i]);
              } else {
                const float* src = part_at<D>(p, c0, z) + prow * D + x * 32;
                float v[32];
#pragma unroll
                for (int i = 0; i < 4; ++i) load32(v + 8 * i, src + 8 * i);
#pragma unroll
                for (int i = 0; i < 32; ++i) a[i] = fmaf(w, v[i], a[i]);
              }
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i] = a[i] * inv;
          }
          if (live) {
            if ((whole && !odd) || join) {
              uint32_t z[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) z[i] = pack_bf16x2(y[2 * i], y[2 * i + 1]);
              __nv_bfloat16* dst = p.o + out * D + x * 32;
              if (p.o_aligned) {
                store32(dst, z);
                store32(dst + 16, z + 8);
              } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) reinterpret_cast<uint4*>(dst)[i] = make_uint4(z[4 * i], z[4 * i + 1], z[4 * i + 2], z[4 * i + 3]);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i) store32(part + x * 32 + 8 * i, reinterpret_cast<const uint32_t*>(y) + 8 * i);
            }
          }
        }
        if (odd && live) {
          const float raw_scale = c.scale_log2 * C::kDecodedBy * (c.kv_exp ? exp2f(static_cast<float>(c.kv_exp[kv])) : 1.f);
#pragma unroll 1
          for (int z = 4 * max(f_lo, f_0); z < 4 * f_hi; ++z) {
            uint32_t bits = bars->flags[slot][z % 4][min(z / 4 - f_0, kFlagTiles - 1)];
#pragma unroll 1
            for (; bits; bits &= bits - 1) {
              const int32_t at = z * 32 + __ffs(bits) - 1;
              if (at < lim) add_odd<D, TYPE>(p, part, p.id[k.i], at, kv, p.q + out * D, raw_scale, m, to);
            }
          }
          if (whole)
#pragma unroll 1
            for (int i = 0; i < D; i += 2)
              *reinterpret_cast<uint32_t*>(p.o + out * D + i) = pack_bf16x2(part[i], part[i + 1]);
        }
        // no weight: the output is 0, whatever the values are (over what was written above, which keeps that short)
        if (live && (join ? sum == 0.f : whole && l == 0.f))
#pragma unroll 1
          for (int i = 0; i < D; i += 8) *reinterpret_cast<uint4*>(p.o + out * D + i) = make_uint4(0, 0, 0, 0);
        if (live) {
          if (join) {
            if (p.lse) p.lse[out] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
          } else if (!whole)
            *reinterpret_cast<float2*>(slot_at<D>(p, blockIdx.x, k.s0 == 0 ? 1 : 0) + 2 * BM * D + 2 * prow) = make_float2(m, l);
          else if (p.lse)
            p.lse[out] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
        }
        if (join && threadIdx.x == 0) p.arrivals[c0] = 0;
        if (k.split) {
          if (threadIdx.x == 0) bars->joined = join;
          tc_fence_before();
          mbar_arrive(&bars->x_empty);
          ++nx;
        }
      }
      if (!whole && !joined) {
        // the last of the block's CTAs to arrive joins their parts, if it has not done so above
        __threadfence();
        mbar_arrive(&bars->part_done);
        if (threadIdx.x == 0) {
          int last = 0;
          if (wait_bounded(&bars->part_done, cuts & 1u, wc, 10)) {
            __threadfence();
            last = atomicAdd(p.arrivals + rec.c0, 1) == rec.parts - 1;
            if (last) p.arrivals[rec.c0] = 0;
          }
          bars->last = last;
          mbar_arrive(&bars->part_last);
        }
        ok = __all_sync(0xffffffffu, wait_bounded(&bars->part_last, cuts & 1u, wc, 10));
        ++cuts;
        if (ok && bars->last) {
          if (k.ntok * group > 32)
            join_block<D, true>(p, k, rec.c0, rec.parts, warp, lane);
          else
            join_block<D, false>(p, k, rec.c0, rec.parts, warp, lane);
        }
      }
      ++items;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, int TYPE>
cudaError_t prepare() {
  cudaFuncAttributes a;
  cudaError_t e = cudaFuncGetAttributes(&a, paged_prompt_kernel<D, TYPE>);
  if (e != cudaSuccess) return e;
  // the softmax groups' registers are granted only if the launch has as many as the split assumes
  if (a.numRegs != kLaunchRegs || a.maxThreadsPerBlock < kThreads) return cudaErrorInvalidConfiguration;
  return cudaFuncSetAttribute(paged_prompt_kernel<D, TYPE>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D, TYPE>::kSmemBytes);
}

template <int D, int TYPE>
cudaError_t launch(const PromptParams& p, cudaStream_t st) {
  return launch_dependent(paged_prompt_kernel<D, TYPE>, static_cast<unsigned>(std::min(sm_count(), kMaxPromptCtas)), kThreads,
                          Cfg<D, TYPE>::kSmemBytes, st, p);
}

template <int D>
cudaError_t launch(const PromptParams& p, cudaStream_t st) {
  if (p.c.page_type == SR_PAGE_BF16) return launch<D, SR_PAGE_BF16>(p, st);
  if (p.c.page_type == SR_PAGE_INT4) return launch<D, SR_PAGE_INT4>(p, st);
  return launch<D, SR_PAGE_E4M3>(p, st);
}

}  // namespace

size_t paged_prompt_floats(int head_dim) {
  return static_cast<size_t>(2 * kMaxPromptCtas) * (head_dim == 128 ? slot_floats<128>() : slot_floats<64>());
}

cudaError_t paged_prompt_prepare(int head_dim, int page_type) {
  if (page_type == SR_PAGE_BF16) return head_dim == 128 ? prepare<128, SR_PAGE_BF16>() : prepare<64, SR_PAGE_BF16>();
  if (page_type == SR_PAGE_INT4) return head_dim == 128 ? prepare<128, SR_PAGE_INT4>() : prepare<64, SR_PAGE_INT4>();
  return head_dim == 128 ? prepare<128, SR_PAGE_E4M3>() : prepare<64, SR_PAGE_E4M3>();
}

bool paged_prompt_plan(PromptParams& p) {
  p.tpt = BM / p.c.group;
  p.group_magic = (65536u + static_cast<uint32_t>(p.c.group) - 1u) / static_cast<uint32_t>(p.c.group);   // exact below 256
  int64_t blocks = 0;
  for (int i = 0; i < p.n; ++i) {
    p.blk0[i] = static_cast<int32_t>(blocks);
    blocks += (p.row0[i + 1] - p.row0[i] + 2 * p.tpt - 1) / (2 * p.tpt);
  }
  p.blocks = static_cast<int32_t>(blocks);
  p.o_aligned = (reinterpret_cast<uintptr_t>(p.o) & 31) == 0;
  // a CTA's stretch of steps is counted in 32 bits (half an hour of work and more)
  return blocks * p.c.n_kv <= (int64_t(1) << 31) / (p.c.cap / BN + 1 + kItemCost) * std::min(sm_count(), kMaxPromptCtas);
}

cudaError_t launch_paged_prompt(const PromptParams& p, cudaStream_t st) {
  return p.c.head_dim == 128 ? launch<128>(p, st) : launch<64>(p, st);
}

}  // namespace sr
