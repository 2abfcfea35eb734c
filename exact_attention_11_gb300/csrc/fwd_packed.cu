// fwd_packed.cu -- exact attention of several queries per sequence for
// sequences of different lengths in one call, with grouped key/value heads,
// on the sm_103a tensor cores:
//   packed   prompts packed one after another, q [T, H, d], k and v [T, Hk, d],
//            sequence s in rows cu_seqlens[s] .. cu_seqlens[s+1] - 1, every
//            query against its own sequence's keys (causal or not);
//   paged    a chunk of new queries per sequence, q [T, H, d], against the
//            paged cache that holds the sequence's whole context (the chunk's
//            own keys included): query i of n sees keys 0 .. ctx - n + i.
// Each has a form with a sliding window and first tokens that stay visible (kWindow:
// position p sees keys j <= p with j > p - window or j < sinks), and the paged one a form
// for groups of sequences that share a prefix's cache blocks (kShared, kSharedFew).
//
// What is computed per row: O = softmax(scale q K^T) V over the visible keys,
// key tile by key tile with the running maximum and sum of eqs. (2)-(4) of
// "Flash Attention" (suniverse77.github.io, section "Online Softmax"), as in
// fwd_bf16.cu, whose warp roles, TMEM plan and MMA order this kernel shares:
// two 128-row query tiles A and B take turns on the tensor core, O and S stay
// in TMEM, P is written over S, one softmax warpgroup per tile.
//
// What differs, and why:
//  * A query tile's 128 rows are (token, head of the group) pairs, tokens
//    outermost: 128 / G tokens of the G query heads that share a key/value
//    head.  K and V are read once for the whole group, short chunks still fill
//    MMA rows, and the causal diagonal touches 128 / G keys of a row instead
//    of 128.  A tile is one TMA box (64 of d) x G heads x (128 / G) tokens; when
//    G does not divide 128 the last rows of the tile hold no query.
//  * Sequence bounds are device data.  An item is (block of two tiles, context
//    partition, key/value head).  Up to kCachedSeqs sequences, each CTA reads the
//    bounds once, sorts the sequences by their heaviest item and numbers all items
//    with a prefix sum in shared memory, heaviest sequence first and within a
//    sequence from its last block (the heaviest under the causal mask) down, so
//    that the call ends with its lightest items; beyond, sequence s starts at block
//    cu_seqlens[s] / (2 * 128/G) + s, which needs no prefix sum and leaves some
//    numbers unused.  The producer warp finds an item's sequence by a 32-way
//    search and hands the decoded item to the other roles.
//  * The key tile that a sequence ends in also holds the next sequence's rows
//    (packed) or whatever the cache slots past the context hold (paged).  Their
//    scores are set to -inf, and since a zero weight does not cancel a NaN, the
//    softmax warps that use that tile first clear their V rows in shared memory
//    before they hand over P.  (A spare warp that did it, and had to follow every
//    tile for its barriers' sake, cost 2% on long prompts.)
//  * Paged K and V are read as in the grouped decode (decode_gqa_tc.cu): K in
//    no-swizzle core matrices, V^T in 32-byte-swizzle blocks of 16 tokens, both
//    K-major B operands here, one copy a block (K in two halves a block: 355 us for
//    4 x 1024 tokens over 8192, not 345).  Block ids outside the cache read as zeros.
//  * Few rows over long contexts do not fill the GPU, and a long context beside
//    short ones would finish alone: a block's context is then cut into equal
//    partitions (parts_of); each writes its unnormalised fp32 rows and (max, sum),
//    and paged_merge_kernel joins them (eq. (4)).
//  * kWindow: a block of queries visits the keys from the first that its first query sees
//    on, and before them the cells of 16 keys that hold first tokens, which share the
//    first key tile with the window's start (8 prompts up to 8192, window 1024, 4 first
//    tokens: 260 us; with a key tile of their own 272).  Inside an item positions count
//    along that list, so only the copies' addresses and the mask's lower bound differ.
//  * kShared, kSharedFew: a group's prefix is walked by the rows of all its sequences as if
//    they were one sequence's, and what each has behind it on its own; both write partial
//    rows, which the merge joins.  The items of up to 112 sequences and groups are numbered
//    by every CTA for itself, of more by a kernel of one block ahead.
//
// What bounds it: for long prompts the tensor pipe and the softmax chain (S out of
// TMEM, exponentials, P back) of a two-tile step, 1.4 us where the MMAs alone take
// 1.37; for chunks of one query tile that chain alone, 1.3 us a key tile; for a few
// tokens over long contexts the 16 copies of a paged key tile and HBM; for short
// prompts the start (5 us) and the chain of an SM's few items.  Measured: 8 prompts up
// to 4096 tokens, 32 / 8 heads, d = 128, causal, 182 us (1497 TFLOP/s); one of 16384,
// 8 / 1 heads, fp16, 311 - 328 us (1768 - 1676); 32 prompts up to 200, 16 heads, d = 64, 16 us;
// chunks of 4 x 1024 tokens over 8192, 345 us (1494 TFLOP/s), up to 1024 over up to
// 16384, 91 us; 64 single tokens over 4096, 180 us (6.0 TB/s).  Windows: 8 prompts up to
// 8192, 32 / 8 heads, d = 128, window 1024: 260 us (1230 TFLOP/s; a block's nine key tiles
// take 1.5 us each, its start and end 3); one of 16384, 8 / 1 heads, fp16, window 4000,
// 150 - 154 us (1605 - 1575); 64 single tokens, window 4096, 182 us (5.9 TB/s); chunks up to
// 2048 over up to 32768, window 4096, 171 us (1430 TFLOP/s).  These are times of a replayed
// call on the same tensors; with other tensors from call to call, whose lines are not in L2,
// the prompts take 274 - 277, the one of 16384 165 - 166 and the chunks 181 us.  Shared prefixes, single tokens, 32 / 8
// heads: 64 sequences behind 8192 tokens, up to 512 of their own, 38 us (2.6 TB/s: start,
// the chains of an SM's four or five short items, merge; 314 without sharing); 256 behind
// 32768, up to 2048 of their own, 280 us (4.3 TB/s; first the prefix, bound by the tensor
// cores, 65 us, then the rest at 5.8 TB/s; 4579 without).
// Rounding: P to the element type before P V, O once at the end; scores, maxima, sums,
// partial rows and their merge are fp32.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstddef>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "kernels.h"
#include "packed.cuh"
#include "ptx.cuh"

namespace fattn {
namespace {

constexpr int BM = 128;             // rows of a query tile (MMA M)
constexpr int BN = 128;             // keys per tile
constexpr int kThreads = 384;
// The register split of fwd_bf16.cu: 168 at launch, 88 / 208 / 208 after.
constexpr uint32_t kRegsProducer = 88, kRegsSoftmax = 208;
static_assert(kRegsProducer + 2 * kRegsSoftmax == 3 * 168, "launch register budget");
constexpr uint32_t kTmemCols = 512;
constexpr float kRescaleThreshold = 8.0f;   // log2 units (see fwd_bf16.cu)
constexpr int kBlk = kDecodeBlockSize;      // 16 tokens per cache block
constexpr int kTileBlocks = BN / kBlk;      // 8 cache blocks per key tile
constexpr int kBarArea = 3 * 1024;          // bytes of barriers, items and sequence bounds

// Shared memory: two Q tile buffers, a ring of `kSlots` key or value tiles (K of
// tile 0, V of tile 0, K of tile 1, ...), output staging (packed), barriers and
// the item ring, then the cached sequence bounds.  Both Q buffers and the tile
// ring are first in, first out across items: a one-tile item's Q may arrive while
// the one before is still in use.  The paged kernel, which often waits on HBM with
// one short query tile, has a fifth slot in place of the staging.
template <int D, bool PAGED>
struct Cfg {
  static constexpr int kSlots = D == 64 ? 8 : (PAGED ? 5 : 4);
  static constexpr int kBoxes = D / 64;
  static constexpr int kTileBytes = BM * D * 2;
  static constexpr int kBoxBytes = BM * 128;
  static constexpr int kQ = 0;
  static constexpr int kRing = kQ + 2 * kTileBytes;
  static constexpr int kStage = kRing + kSlots * kTileBytes;   // 8 x 4 KB
  static constexpr int kBar = kStage + (PAGED ? 0 : 8 * 4096);
  static constexpr int kAlloc = kBar + kBarArea;
  static_assert(kAlloc <= 227 * 1024, "shared memory budget");
  static constexpr uint32_t kColS0 = 0, kColS1 = 128, kColO0 = 256, kColO1 = 384;   // O: S + 256
};

constexpr int kMaxSlots = 8;
enum : int {
  kBarQFull = 0,       // + Q buffer (2)
  kBarQEmpty = 2,      // + Q buffer (2)
  kBarSFull = 4,       // + tile
  kBarPReady = 6,      // + 2 * tile + half, 4 warps
  kBarODone = 10,      // + tile
  kBarDrain = 12,
  kBarItemFull = 13,   // + ring slot (2)
  kBarItemEmpty = 15,  // + ring slot (2)
  kBarFull = 17,       // + slot: the key or value tile has landed
  kBarEmpty = kBarFull + kMaxSlots,   // + slot: its MMAs are done
  kNumBars = kBarEmpty + kMaxSlots + 1   // (even: Misc, which follows, holds 8-byte values)
};
// Arrivals that free an item slot: the MMA thread and the eight softmax warps.
constexpr int kItemConsumers = 1 + 8;

// A decoded work item.
struct Item {
  int live;          // 0: no more items
  int row0;          // packed row (token) of tile A's first token
  int n_tok[2];      // tokens of tiles A and B
  int kvh;           // key/value head
  int pos0;          // key index that tile A's first token sees last (its position)
  int kv_len;        // keys of the sequence
  int kv0;           // packed: first row of the sequence's keys; paged: sequence
  int kt0;           // first key tile of this partition
  int n[2];          // key tiles of tiles A and B in this partition
  int part;          // partition
  int split;         // the rows go to the partition workspace
  int clear[2];      // the step in which tile A's (B's) softmax clears V's last rows, or < 0
};

// kWindow: a block visits a list of cells of 16 keys: those of the sequence's first
// tokens, then those from the first key that its first token sees on; eight cells are a
// key tile.  Cell x of the list is the sequence's cell x, or x + skip from `at` on.
// Positions and lengths in an item count along the list: skip cells less than in the
// sequence (every real row lies behind the gap).
// With shared prefixes, skip is the first table column of the item's keys.
constexpr int kCell = 16;
static_assert(kCell == kBlk, "a cell of the paged list is a cache block");
struct Gap {
  int at, skip;
  __device__ int cell(int x) const { return x >= at ? x + skip : x; }
};

constexpr int kCachedSeqs = 112;
struct Misc {
  uint32_t tmem_base;
  int abort;
  Item item[2];
  int2 seq[kCachedSeqs + 1];    // (first row, context length)
  // By weight of their items, lightest first: the sequences, their partitions, and
  // the items of those before ([S]: of all).
  int first[kCachedSeqs + 1];
  int16_t parts[kCachedSeqs];
  uint8_t order[kCachedSeqs];
  int key[kCachedSeqs];         // scratch of the sort
  int16_t n_parts[kCachedSeqs];
};
static_assert(8 * kNumBars + sizeof(Misc) <= kBarArea, "barrier area");
// Status latched when the dynamic shared memory does not start on a 1024-byte
// boundary (the kernel then does nothing).
constexpr int kDevBadSmemBase = -2;

// What a query sees: all keys of its sequence up to its own (or, packed, all of
// them); or of those a window and the sequence's first tokens; or all of them where
// groups of sequences share the blocks of a prefix (paged), numbered ahead or, of few
// sequences, by every CTA.  (Both in one kernel cost 1.5% of 256 sequences behind 32768 tokens.)
enum : int { kAll = 0, kWindow = 1, kShared = 2, kSharedFew = 3 };
__host__ __device__ constexpr bool is_shared(int form) {
  return form == kShared || form == kSharedFew;
}

struct Args {
  uint16_t *o;
  float *lse;                   // [H][T] or null
  const int *cu_seqlens, *context_lens, *block_tables;
  float *ws_o;                  // [part][T * H][D]
  float2 *ws_ml;                // [part][T * H] (max in log2 units, sum)
  int *sched, *dev_status;
  int S, T, H, Hk, G, tpb;      // tpb: tokens per query tile, 128 / G
  int max_blocks, num_blocks;
  int fault_cta;                // a CTA that loses its copies (failure-path test), or -1
  int n_vblocks, n_split, causal;   // n_split: most partitions of a context
  float scale_log2;
};
// What a form's kernels need besides.  (Not in Args: the kernels of all keys spill two
// registers more when the parameters grow past 512 bytes.)
struct WindowArgs : Args {
  int window, sinks;            // up to 2^30 each
};
// The map of k or v (packed, kWindow: and one with boxes of 64 x 16 x 1).
struct CellMaps {
  CUtensorMap tiles, cells;
};
template <bool PAGED, int FORM>
using KvMap = std::conditional_t<!PAGED && FORM == kWindow, CellMaps, CUtensorMap>;
__device__ __forceinline__ const CUtensorMap &tile_map(const CUtensorMap &m) { return m; }
__device__ __forceinline__ const CUtensorMap &cell_map(const CUtensorMap &m) { return m; }
__device__ __forceinline__ const CUtensorMap &tile_map(const CellMaps &m) { return m.tiles; }
__device__ __forceinline__ const CUtensorMap &cell_map(const CellMaps &m) { return m.cells; }
// A prefix is walked once for all rows of its group: it and what each sequence has of
// its own are items of their own, numbered by shared_plan_kernel, and their partial rows
// lie in ws_o one behind the other, those of the prefix from partition n_split on.
struct SharedArgs : Args {
  const int *cu_groups, *prefix_lens;
  int P, pre_split;             // groups; most partitions of a prefix
  int ctas;                     // CTAs that have their first item in `start`
  int merge_heads;              // heads of a token that a warp of the merge joins; 0: by sequence
  int *head;                    // number of entries of `first` and `rec`
  int *first;                   // [entries + 1]: their first items, heaviest first
  int4 *rec;                    // [entries][2]: begin, n, kv_len, pos;
                                // table row, first table column, partitions, first ws_o partition
                                // (or -1: rows are written directly)
  int4 *seq;                    // [S][2]: begin, n, kv_len, pos (of the sequence's own keys);
                                // partitions, those of the prefix (0: none), -, -
  int4 *start;                  // [ctas][4]: Item and the first table column
};
template <int FORM>
using FormArgs = std::conditional_t<FORM == kWindow, WindowArgs,
                                    std::conditional_t<is_shared(FORM), SharedArgs, Args>>;

// Key tiles that `n` tokens, the last of which sees key `last` last, visit.
__device__ __forceinline__ int tiles_for(int n, int last, int kv_len) {
  return n > 0 ? (max(0, min(kv_len, last + 1)) + BN - 1) / BN : 0;
}

// All but the lowest n bits: all for n <= 0, none for n >= 32 (PTX clamps the shift).
__device__ __forceinline__ uint32_t high_bits(int n) {
  uint32_t r;
  asm("shl.b32 %0, %1, %2;" : "=r"(r) : "r"(~0u), "r"(max(n, 0)));
  return r;
}

// A query that sees every key of its sequence.
constexpr int kSeesAll = 0x3fffffff;

// Sequence s: its packed rows [begin, begin + n), keys and first position.
struct Seq {
  int begin, n, kv_len, pos;
};
__device__ __forceinline__ Seq make_seq(const Args &a, bool paged, int begin, int end, int ctx) {
  Seq q;
  q.begin = begin;
  q.n = max(end - begin, 0);
  if (paged) {
    q.kv_len = clampi(ctx, 0, a.max_blocks * kBlk);
    q.pos = q.kv_len - q.n;
  } else {
    q.kv_len = q.n;
    q.pos = a.causal ? 0 : kSeesAll;
  }
  return q;
}
__device__ __forceinline__ int seq_begin(const Args &a, int s) {
  return clampi(a.cu_seqlens[s], 0, a.T);
}
template <bool PAGED>
__device__ __forceinline__ Seq global_seq(const Args &a, int s) {
  return make_seq(a, PAGED, seq_begin(a, s), seq_begin(a, s + 1), PAGED ? a.context_lens[s] : 0);
}

// The gap in the list of a block whose first token is at position pos.
template <int FORM>
__device__ __forceinline__ Gap gap_of(const FormArgs<FORM> &a, int pos) {
  if constexpr (FORM == kWindow) {
    const int first = max(pos - a.window + 1, 0) / kCell;
    const int at = min((a.sinks + kCell - 1) / kCell, first);
    return {at, first - at};
  }
  return {0, 0};
}

// Work of a sequence: key tiles of its last block, and blocks.
struct Work {
  int tiles, blocks;
};
template <int FORM>
__device__ __forceinline__ Work work_of(const FormArgs<FORM> &a, const Seq &q) {
  const int blocks = (q.n + 2 * a.tpb - 1) / (2 * a.tpb);
  const int gap =
      FORM == kWindow ? gap_of<FORM>(a, q.pos + max(blocks - 1, 0) * 2 * a.tpb).skip * kCell : 0;
  return {tiles_for(q.n, q.pos + q.n - 1 - gap, q.kv_len - gap), blocks};
}

// Partitions.  With W key tiles of work per SM cut into partitions of p, a
// partition's cost c (in key tiles: its start, and its rows' trip through the
// workspace, 1 KB each at an SM's share of the HBM rate) adds W c / p, and the SMs
// end up to p apart, 0.7 p on average: p = sqrt(W c / 0.7) balances the two, at
// least four key tiles; what is shorter than 1.5 p stays whole.  (Constants fitted
// to a model of the schedule over nine mixes of chunks and contexts, then measured on
// an earlier form of the kernel, so only the ratios count: against kFixed 2.5, 2 and 3
// took 1.04 and 0.98 of the time for 16 drafts of up to 6 tokens over up to 4096, but
// 0.99 and 1.05 for 64 single tokens over 4096; kFixed 1, kRow 0.01 or 1 in place of 0.7
// took 1.3 for chunks of up to 1024 over up to 16384.)  `work`: key tiles of the call's
// blocks, of one key/value head.  Each block of the sequence cuts its own key tiles into
// that many.  (Roundings are spelled out: the merge kernel has to reach the same
// number.)  kWindow: the few rows of a sequence of one block cost little to cut, and its
// items come last, so where such sequences are less than an eighth of the work they take
// eight times theirs for the call's (chunks of 6, 1536, 3 and 2048 over up to 32768, window
// 4096: 171 us, 179 without; always their own work: 178 for 170 on 31 chunks up to 289; over
// three times 40 mixes of all kinds four or sixteen times theirs, or the call's, were within
// 0.3% of each other: it matters for such few rows only).
constexpr float kPartFixed = 2.5f, kPartRow = 0.02f;
__device__ __forceinline__ int parts_of(const Args &a, const Seq &q, int tiles, int64_t work,
                                        int most) {
  constexpr float kFixed = kPartFixed, kRow = kPartRow, kLeast = 4.f;
  if (most == 1) return 1;
  const float w = __fmul_rn(__ll2float_rn(work * a.Hk), 1.f / (152.f * 0.7f));
  const float c = __fmaf_rn(kRow, static_cast<float>(min(q.n, 2 * a.tpb) * a.G), kFixed);
  const float size = fmaxf(__fsqrt_rn(__fmul_rn(w, c)), kLeast);
  const float n = __fdiv_rn(static_cast<float>(tiles), size);
  return n < 1.5f ? 1 : min(__float2int_ru(n), most);
}
__device__ __forceinline__ int part_size(int total, int parts) {
  return max(1, (total + parts - 1) / parts);
}

__device__ __forceinline__ int64_t warp_sum(int64_t v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(~0u, v, off);
  return v;
}

// Sorts the sequences and numbers their items (one warp): Misc::seq -> order, parts,
// first.  Run once by a cold instruction cache: short code, not unrolled.
template <bool PAGED, int FORM>
__device__ __forceinline__ void number_items(const FormArgs<FORM> &a, Misc *m) {
  const int lane = threadIdx.x & 31;
  auto seq = [&](int i) {
    return make_seq(a, PAGED, m->seq[i].x, m->seq[i + 1].x, m->seq[i].y);
  };
  int64_t work = 0, work_short = 0;
  if (PAGED && a.n_split > 1) {
#pragma unroll 1
    for (int i = lane; i < a.S; i += 32) {
      const Work w = work_of<FORM>(a, seq(i));
      work += static_cast<int64_t>(w.tiles) * w.blocks;
      if (FORM == kWindow && w.blocks == 1) work_short += w.tiles;
    }
    work = warp_sum(work);
    if (FORM == kWindow) work_short = min(work, 8 * warp_sum(work_short));
  }
  // Key: key tiles of an item, then the index, so that no two are equal.
#pragma unroll 1
  for (int i = lane; i < a.S; i += 32) {
    const Seq q = seq(i);
    const Work x = work_of<FORM>(a, q);
    const int tiles = x.tiles;
    const int64_t of = FORM == kWindow && x.blocks == 1 ? work_short : work;
    const int parts = PAGED ? parts_of(a, q, tiles, of, a.n_split) : 1;
    const int size = PAGED ? part_size(tiles, parts) : tiles;
    m->key[i] = min(size, (1 << 23) - 1) * 128 + i;
    m->n_parts[i] = static_cast<int16_t>(parts);
  }
  __syncwarp();
#pragma unroll 1
  for (int i = lane; i < a.S; i += 32) {
    const int key = m->key[i];
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < a.S; ++j) rank += m->key[j] < key ? 1 : 0;
    m->order[rank] = static_cast<uint8_t>(i);
    m->parts[rank] = m->n_parts[i];
    m->first[rank] = work_of<FORM>(a, seq(i)).blocks * m->n_parts[i] * a.Hk;
  }
  __syncwarp();
  int carry = 0;
#pragma unroll 1
  for (int base = 0; base < a.S; base += 32) {
    const int n = base + lane < a.S ? m->first[base + lane] : 0;
    int sum = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int x = __shfl_up_sync(~0u, sum, off);
      if (lane >= off) sum += x;
    }
    if (base + lane < a.S) m->first[base + lane] = carry + sum - n;
    carry += __shfl_sync(~0u, sum, 31);
  }
  if (lane == 0) m->first[a.S] = carry;
  __syncwarp();
}

// kShared: item i of an entry, whose words are q and r.
__device__ __forceinline__ bool decode_entry(const SharedArgs &a, const int4 &q, const int4 &r,
                                             int i, Item &it, Gap &gap) {
  const int blk = i / a.Hk;
  it.kvh = i - blk * a.Hk;
  const int x = blk / r.z, part = blk - x * r.z, tok0 = x * 2 * a.tpb;
  it.live = 1;
  it.row0 = q.x + tok0;
  it.pos0 = q.w + tok0;
  it.kv_len = q.z;
  it.kv0 = r.x;
  gap = {0, r.y};
  int total[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    it.n_tok[t] = clampi(q.y - tok0 - t * a.tpb, 0, a.tpb);
    total[t] = tiles_for(it.n_tok[t], it.pos0 + t * a.tpb + it.n_tok[t] - 1, q.z);
  }
  const int size = part_size(max(total[0], total[1]), r.z);
  it.split = r.w >= 0;
  it.part = max(r.w, 0) + part;
  it.kt0 = part * size;
#pragma unroll
  for (int t = 0; t < 2; ++t) it.n[t] = clampi(total[t] - it.kt0, 0, size);
  it.clear[0] = q.z % BN != 0 ? q.z / BN - it.kt0 : -1;
  it.clear[1] = it.n[0] <= it.clear[0] ? it.clear[0] : -1;
  return part == 0 || it.n[0] > 0 || it.n[1] > 0;
}

// Item w of the numbered entries, in global memory.
__device__ __forceinline__ bool decode_shared(const SharedArgs &a, int w, Item &it, Gap &gap) {
  const int at = warp_search(*a.head, w, [&](int i) { return a.first[i]; });
  return decode_entry(a, a.rec[2 * at], a.rec[2 * at + 1], w - a.first[at], it, gap);
}

// Item w of n_items (whole warp); false if it has no work.  m: the numbered
// sequences, or null.
template <bool PAGED, int FORM>
__device__ __forceinline__ bool decode_item(const FormArgs<FORM> &a, const Misc *m, int n_items,
                                            int w, Item &it, Gap &gap) {
  const int tb = 2 * a.tpb, u = n_items - 1 - w;
  int s, blk, parts = 1;
  Seq q;
  it.part = 0;
  if (m != nullptr) {
    const int at = warp_search(a.S, u, [&](int i) { return m->first[i]; });
    s = m->order[at];
    q = make_seq(a, PAGED, m->seq[s].x, m->seq[s + 1].x, m->seq[s].y);
    const int r = u - m->first[at];
    blk = r / a.Hk;
    it.kvh = r - blk * a.Hk;
    if (PAGED && (parts = m->parts[at]) > 1) {
      const int x = blk / parts;
      it.part = blk - x * parts;
      blk = x;
    }
  } else {   // contexts are not cut here, and items come in the sequences' order
    const int vb = u / a.Hk;
    it.kvh = u - vb * a.Hk;
    s = warp_search(a.S, vb, [&](int i) { return seq_begin(a, i) / tb + i; });
    if (s < 0) return false;
    q = global_seq<PAGED>(a, s);
    blk = vb - q.begin / tb - s;
    if (blk < 0) return false;
  }
  const int tok0 = blk * tb;
  if (tok0 >= q.n) return false;
  it.live = 1;
  it.row0 = q.begin + tok0;
  it.pos0 = q.pos + tok0;
  it.kv0 = PAGED ? s : q.begin;
  gap = gap_of<FORM>(a, it.pos0);
  if (FORM == kWindow) it.pos0 -= gap.skip * kCell, q.kv_len -= gap.skip * kCell;
  it.kv_len = q.kv_len;
  int total[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    it.n_tok[t] = clampi(q.n - tok0 - t * a.tpb, 0, a.tpb);
    total[t] = tiles_for(it.n_tok[t], it.pos0 + t * a.tpb + it.n_tok[t] - 1, q.kv_len);
  }
  const int size = part_size(max(total[0], total[1]), parts);
  it.split = parts > 1;
  it.kt0 = it.part * size;
#pragma unroll
  for (int t = 0; t < 2; ++t) it.n[t] = clampi(total[t] - it.kt0, 0, size);
  // Where both tiles visit the sequence's ragged last key tile A clears its V, whose
  // P V goes first.
  it.clear[0] = q.kv_len % BN != 0 ? q.kv_len / BN - it.kt0 : -1;
  it.clear[1] = it.n[0] <= it.clear[0] ? it.clear[0] : -1;
  return it.part == 0 || it.n[0] > 0 || it.n[1] > 0;
}

// 16-bit element types: as in fwd_bf16.cu.
template <bool F16>
__device__ __forceinline__ constexpr uint32_t idesc16(uint32_t bf16_desc) {
  return F16 ? (bf16_desc & ~((1u << 7) | (1u << 10))) : bf16_desc;
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if (F16) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  return pack_bf16x2(lo, hi);
}

// High descriptor words: 128-byte swizzle with 1024-byte row groups
// (kSdescHi1024); no swizzle, 8-token groups 2 KB apart (paged K); 32-byte
// swizzle, 8-row groups 256 bytes apart (paged V^T).
constexpr uint32_t kHiPagedK = (2048u >> 4) | (1u << 14);
constexpr uint32_t kHiPagedV = (256u >> 4) | (1u << 14) | (6u << 29);

__device__ __forceinline__ void mma_ss_hi(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo,
                                          uint32_t b_hi, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .b64 da, db;\n .reg .pred p;\n mov.b64 da, {%1, %5};\n mov.b64 db, {%2, %6};\n"
      " setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(kSdescHi1024), "r"(b_hi)
      : "memory");
}
__device__ __forceinline__ void mma_ts_hi(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo,
                                          uint32_t b_hi, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .b64 db;\n .reg .pred p;\n mov.b64 db, {%2, %5};\n"
      " setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(b_hi)
      : "memory");
}

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap *m, int c0, int c1,
                                            int c2, int c3, int c4, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *m, int c0, int c1,
                                            int c2, int c3, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}

// 32 bytes to global memory, in one store where they are aligned to that (a caller's
// tensor need not be).
__device__ __forceinline__ void store32(void *p, const uint32_t *v) {
  if ((reinterpret_cast<uintptr_t>(p) & 31) != 0) {
    reinterpret_cast<uint4 *>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<uint4 *>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    return;
  }
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// A wait that all lanes of the warp leave with one answer.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t ph, volatile int *abort_flag) {
  return __all_sync(~0u, mbar_wait(bar, ph, abort_flag));
}

__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t ph) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, ph) && globaltimer_ns() - t0 < kWaitLimitNs) {
  }
}

// What a call with shared prefixes walks.  A sequence shares its group's prefix if all of
// that lies before its new tokens; sequences that do are walked behind it only, and the
// prefix, read through the table of the first of them, is walked by all rows of the group
// together.  Prefixes that save less than they cost (partial rows, the start of their
// items) are not shared.
struct PlanEntry {              // entry s: sequence s, or, from S on, group s - S
  Seq q;                        // its rows and keys
  Work w;
  int row, col;                 // table row, first table column
  int parts, slot;              // partitions, the first one's place in ws_o, or -1
  int group;                    // that whose prefix the sequence shares, or -1
};
// By all THREADS threads of a block.  The thread's first sequence stays in registers; with
// that, and the groups, global memory is read once, up to THREADS sequences.
template <int THREADS, int GROUPS>
struct Planner {
  struct Scratch {
    int g_first[GROUPS + 1], g_prefix[GROUPS], g_lead[GROUPS], g_blocks[GROUPS];
    int begins[THREADS + 1];    // of the first sequences
    unsigned long long work;
  };
  const SharedArgs &a;
  Scratch &m;
  const int tid;
  Seq mine;
  PlanEntry own;
  int64_t work;

  __device__ Planner(const SharedArgs &args, Scratch &scratch)
      : a(args), m(scratch), tid(threadIdx.x), mine{}, own{}, work(0) {
    if (tid < a.S) mine = global_seq<true>(a, tid);
    for (int s = tid; s <= min(a.S, THREADS); s += THREADS) m.begins[s] = seq_begin(a, s);
    for (int g = tid; g <= a.P; g += THREADS) {
      m.g_first[g] = a.P > 0 ? clampi(a.cu_groups[g], 0, a.S) : 0;
      if (g == a.P) break;
      m.g_prefix[g] = clampi(a.prefix_lens[g], 0, a.max_blocks * kBlk) / kBlk * kBlk;
      m.g_lead[g] = a.S;
      m.g_blocks[g] = 0;
    }
    if (tid == 0) m.work = 0;
    __syncthreads();
    for (int s = tid; s < a.S; s += THREADS) {
      const Seq q = whole(s);
      const int g = sharing(s, q);
      if (g < 0) continue;
      atomicMin(&m.g_lead[g], s);
      atomicAdd(&m.g_blocks[g], work_of<kShared>(a, q).blocks);
    }
    __syncthreads();
    int64_t sum = 0;
    for (int g = tid; g < a.P; g += THREADS) {
      const Seq q = group_seq(g);
      const Work w = work_of<kShared>(a, q);
      const float saved = static_cast<float>(m.g_blocks[g] - w.blocks) * w.tiles;
      const float cost = kPartFixed * w.blocks + 2.f * kPartRow * q.n * a.G;
      if (m.g_lead[g] == a.S || !(saved > cost))
        m.g_prefix[g] = 0;
      else
        sum += static_cast<int64_t>(w.tiles) * w.blocks;
    }
    __syncthreads();
    if (tid < a.S + a.P) own = entry(tid);
    for (int s = tid; s < a.S; s += THREADS) {
      const Work w = s == tid ? own.w : entry(s).w;
      sum += static_cast<int64_t>(w.tiles) * w.blocks;
    }
    sum = warp_sum(sum);
    if ((tid & 31) == 0) atomicAdd(&m.work, static_cast<unsigned long long>(sum));
    __syncthreads();
    work = static_cast<int64_t>(m.work);
    if (tid < a.S + a.P) cut(tid, own);
  }
  __device__ Seq whole(int s) const { return s == tid ? mine : global_seq<true>(a, s); }
  __device__ int begin_of(int s) const { return s <= THREADS ? m.begins[s] : seq_begin(a, s); }
  // The group of the whole sequence q if it shares the prefix, else -1.  (A sequence is in
  // the last group that begins at or before it, if in any.)
  __device__ int sharing(int s, const Seq &q) const {
    int lo = 0, n = a.P;
    while (n > 0) {
      const int half = n / 2;
      if (m.g_first[lo + half] <= s) lo += half + 1, n -= half + 1;
      else n = half;
    }
    if (lo == 0 || s >= m.g_first[lo]) return -1;
    const int prefix = m.g_prefix[lo - 1];
    return q.n > 0 && prefix > 0 && q.pos >= prefix ? lo - 1 : -1;
  }
  // The rows of a group's prefix; all see all of it.
  __device__ Seq group_seq(int g) const {
    Seq q;
    q.begin = begin_of(m.g_first[g]);
    q.n = max(begin_of(m.g_first[g + 1]) - q.begin, 0);
    q.kv_len = m.g_prefix[g];
    q.pos = kSeesAll;
    return q;
  }
  // (Without its partitions.)
  __device__ PlanEntry entry(int s) const {
    PlanEntry x;
    x.group = -1;
    if (s >= a.S) {
      const int g = s - a.S;
      x.row = min(m.g_lead[g], a.S - 1);
      x.col = 0;
      x.q = group_seq(g);
      if (m.g_prefix[g] == 0) x.q.n = 0;
    } else {
      x.q = whole(s);
      x.group = sharing(s, x.q);
      x.row = s;
      x.col = x.group >= 0 ? m.g_prefix[x.group] / kBlk : 0;
      x.q.kv_len -= x.col * kBlk;
      x.q.pos -= x.col * kBlk;
    }
    x.w = work_of<kShared>(a, x.q);
    return x;
  }
  __device__ void cut(int s, PlanEntry &x) const {
    const bool prefix = s >= a.S;
    x.parts = x.w.blocks == 0
                  ? 1
                  : parts_of(a, x.q, x.w.tiles, work, prefix ? a.pre_split : a.n_split);
    x.slot = prefix ? a.n_split : x.group >= 0 || x.parts > 1 ? 0 : -1;
  }
  __device__ PlanEntry entry_of(int s) const {
    if (s == tid) return own;
    PlanEntry x = entry(s);
    cut(s, x);
    return x;
  }
  // What the merge has to know of sequence s.
  __device__ void put_seq(int s, const PlanEntry &x) const {
    int pre = 0;
    if (x.group >= 0) {
      // Every block of the prefix cuts its tiles alike.
      const PlanEntry p = entry_of(a.S + x.group);
      const int size = part_size(p.w.tiles, p.parts);
      pre = (p.w.tiles + size - 1) / size;
    }
    a.seq[2 * s] = make_int4(x.q.begin, x.q.n, x.q.kv_len, x.q.pos);
    a.seq[2 * s + 1] = make_int4(x.parts, pre, 0, 0);
  }
};

// The numbered entries of a call with few sequences, in shared memory in place of
// Misc's: every CTA finds the same ones for itself (64 requests behind 8192 tokens:
// 39.9 us, 44.8 with a kernel ahead that numbers them; both before the merge loaded rows ahead).
struct PlanTable {
  int entries, items;
  int begins[kCachedSeqs + 1];  // first rows of the sequences
  int first[kCachedSeqs + 1];   // first items, heaviest entry first
  int kv_len[kCachedSeqs], col[kCachedSeqs];
  int16_t parts[kCachedSeqs];   // negative: rows are written directly
  uchar4 of[kCachedSeqs];       // first and last sequence of its rows (+ 1), table row, prefix?
};
constexpr int kPlanTableAt = 8 * kNumBars + offsetof(Misc, seq);
static_assert(kPlanTableAt + sizeof(PlanTable) <= kBarArea && kPlanTableAt % 8 == 0,
              "barrier area");

// By the whole block; scratch: the ring's memory, ahead of its first copies.
__device__ __forceinline__ void plan_items(const SharedArgs &a, PlanTable *m, uint8_t *scratch) {
  using Plan = Planner<kThreads, kCachedSeqs>;
  struct Work {
    Plan::Scratch plan;
    int key[kCachedSeqs], count[kCachedSeqs];
  };
  Work &x = *reinterpret_cast<Work *>(scratch);
  Plan plan(a, x.plan);
  const int tid = threadIdx.x, n = a.S + a.P;
  const PlanEntry &e = plan.own;
  // Key: key tiles of an item, then the index; entries without rows come last.
  int key = -1;
  if (tid < n) {
    if (e.w.blocks > 0)
      key = min(part_size(e.w.tiles, e.parts), (1 << 23) - 1) * 128 + tid;
    x.key[tid] = key;
    if (blockIdx.x == 0 && tid < a.S) plan.put_seq(tid, e);
  }
  if (tid <= a.S) m->begins[tid] = x.plan.begins[tid];
  __syncthreads();
  int rank = 0;
  if (tid < n) {
#pragma unroll 4
    for (int j = 0; j < n; ++j) rank += x.key[j] > key ? 1 : 0;
    if (key >= 0) {
      x.count[rank] = e.w.blocks * e.parts * a.Hk;
      const int g = tid - a.S;
      m->kv_len[rank] = e.q.kv_len;
      m->col[rank] = e.col;
      m->parts[rank] = static_cast<int16_t>(e.slot < 0 ? -e.parts : e.parts);
      m->of[rank] = g >= 0 ? make_uchar4(x.plan.g_first[g], x.plan.g_first[g + 1], e.row, 1)
                           : make_uchar4(tid, tid + 1, e.row, 0);
    }
  }
  const int entries = __syncthreads_count(key >= 0);
  if (tid < 32) {
    int carry = 0;
    for (int base = 0; base < entries; base += 32) {
      const int c = base + tid < entries ? x.count[base + tid] : 0;
      int sum = c;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int below = __shfl_up_sync(~0u, sum, off);
        if (tid >= off) sum += below;
      }
      if (base + tid < entries) m->first[base + tid] = carry + sum - c;
      carry += __shfl_sync(~0u, sum, 31);
    }
    if (tid == 0) m->entries = entries, m->items = carry;
  }
  fence_proxy_async_smem();     // the ring's copies come after what was written there
}

__device__ __forceinline__ bool decode_planned(const SharedArgs &a, const PlanTable *m, int w,
                                               Item &it, Gap &gap) {
  const int at = warp_search(m->entries, w, [&](int i) { return m->first[i]; });
  const uchar4 of = m->of[at];
  const int begin = m->begins[of.x], n = max(m->begins[of.y] - begin, 0), kv_len = m->kv_len[at];
  const int parts = m->parts[at];
  return decode_entry(a, make_int4(begin, n, kv_len, of.w ? kSeesAll : kv_len - n),
                      make_int4(of.z, m->col[at], abs(parts),
                                of.w ? a.n_split : parts < 0 ? -1 : 0),
                      w - m->first[at], it, gap);
}

template <int D, bool F16, bool PAGED, int FORM>
__global__ void __launch_bounds__(kThreads, 1)
    fwd_packed_kernel(const __grid_constant__ CUtensorMap tm_q,
                      const __grid_constant__ KvMap<PAGED, FORM> tm_k,
                      const __grid_constant__ KvMap<PAGED, FORM> tm_v, const FormArgs<FORM> a) {
  using C = Cfg<D, PAGED>;
  static_assert(!PAGED || (D == 128 && !F16), "the paged cache is bf16, d = 128");
  constexpr int R = C::kSlots;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t s_base = smem_u32(smem);
  if ((s_base & 1023u) != 0) {
    if (threadIdx.x == 0) atomicExch(a.dev_status, kDevBadSmemBase);
    return;
  }
  const uint32_t bars = s_base + C::kBar;
  auto bar = [&](int i) { return bars + 8u * i; };
  Misc *misc = reinterpret_cast<Misc *>(smem + C::kBar + 8 * kNumBars);
  volatile int *abort_flag = &misc->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // Consumer side of the item ring.  take_item waits for entry k (whole warp, or
  // the lone MMA thread); after reading what it needs of misc->item[k & 1], the
  // consumer frees the slot (one arrival per warp).
  auto take_item = [&](int k, bool whole_warp) -> bool {
    const bool full = mbar_wait(bar(kBarItemFull + (k & 1)), (k >> 1) & 1, abort_flag);
    return whole_warp ? __all_sync(~0u, full) : full;
  };
  auto free_item = [&](int k, bool whole_warp) {
    if (whole_warp) __syncwarp();
    if (!whole_warp || lane == 0) mbar_arrive(bar(kBarItemEmpty + (k & 1)));
  };
  auto item_of = [&](int k) -> const volatile Item & {
    return *reinterpret_cast<const volatile Item *>(&misc->item[k & 1]);
  };

  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(kBarQFull + t), 1);
      mbar_init(bar(kBarQEmpty + t), 1);
      mbar_init(bar(kBarSFull + t), 1);
      mbar_init(bar(kBarPReady + 2 * t), 4);
      mbar_init(bar(kBarPReady + 2 * t + 1), 4);
      mbar_init(bar(kBarODone + t), 1);
      mbar_init(bar(kBarItemFull + t), 1);
      mbar_init(bar(kBarItemEmpty + t), kItemConsumers);
    }
    mbar_init(bar(kBarDrain), 1);
    for (int s = 0; s < R; ++s) {
      mbar_init(bar(kBarFull + s), 1);
      mbar_init(bar(kBarEmpty + s), 1);
    }
    misc->abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&misc->tmem_base), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc->tmem_base;
  // A programmatic dependent of the kernel before it on the stream: nothing in
  // global memory is touched before that one has finished.  The merge kernel
  // may be scheduled from here on; it waits for this grid in turn.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (PAGED && threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  PlanTable *table = reinterpret_cast<PlanTable *>(smem + C::kBar + kPlanTableAt);
  if constexpr (FORM == kSharedFew) plan_items(a, table, smem + C::kRing);
  const bool cached = !is_shared(FORM) && a.S <= kCachedSeqs;
  if (cached)
    for (int i = threadIdx.x; i <= a.S; i += kThreads)
      misc->seq[i] = make_int2(seq_begin(a, i), PAGED && i < a.S ? a.context_lens[i] : 0);
  __syncthreads();

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsProducer));
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      // The whole warp decodes items and holds block ids; lane 0 waits, and
      // issues the packed copies; lanes 0 .. 7 issue a paged tile's copies.
      if (lane == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tile_map(tm_k));
        tma_prefetch_desc(&tile_map(tm_v));
      }
      if (cached) {
        number_items<PAGED, FORM>(a, misc);
      }
      const Misc *numbered = cached ? misc : nullptr;
      int n_items = cached ? misc->first[a.S] : a.n_vblocks * a.Hk;
      if constexpr (FORM == kShared) n_items = a.first[*a.head];
      if constexpr (FORM == kSharedFew) n_items = table->items;
      int e = 0, nq = 0;        // tiles and Q tiles copied so far
      bool ok = true;
      int w = blockIdx.x;       // the first item is the CTA's own; the rest are claimed
      int w_claim = 0;          // lane 0: the claim in flight
      auto claim = [&]() {
        if (lane == 0) w_claim = static_cast<int>(gridDim.x) + atomicAdd(a.sched, 1);
      };
      auto claimed = [&]() { return __shfl_sync(~0u, w_claim, 0); };
      // The next item with work at or after w, claiming on; live = 0 at the end.
      Item nxt;
      Gap nxt_gap;
      int nxt_id = 0;           // paged: block id of the item's block `lane`
      auto ids_of = [&](const Item &it, const Gap &gap, int tile) -> int {
        // Lane i: block i of the four key tiles from `tile` on; past the
        // context, a block that the cache does not have (reads as zeros).
        const int b = tile * kTileBlocks + lane;
        if (b >= (it.kv_len + kBlk - 1) / kBlk) return a.num_blocks;
        const int at = FORM == kWindow ? gap.cell(b) : is_shared(FORM) ? gap.skip + b : b;
        return a.block_tables[static_cast<int64_t>(it.kv0) * a.max_blocks + at];
      };
      // Packed: the copies of a key or value tile.  Where the list's gap lies inside it
      // (kWindow), cell by cell; else one box of 128 rows for every 64 values.
      auto load_rows = [&](const auto &map, const Item &it, const Gap &gap, int tile, uint32_t dst,
                           uint32_t full) {
        const int c0 = tile * (BN / kCell);
        if (FORM == kWindow && gap.skip > 0 && c0 < gap.at && c0 + BN / kCell > gap.at) {
          const int c = lane % (BN / kCell), b = lane / (BN / kCell);
          if (b < C::kBoxes)
            tma_load_3d(dst + b * C::kBoxBytes + c * kCell * 128, &cell_map(map), b * 64,
                        it.kv0 + gap.cell(c0 + c) * kCell, it.kvh, full);
        } else if (lane == 0) {
          const int row = it.kv0 + (FORM == kWindow ? gap.cell(c0) * kCell : tile * BN);
          for (int b = 0; b < C::kBoxes; ++b)
            tma_load_3d(dst + b * C::kBoxBytes, &tile_map(map), b * 64, row, it.kvh, full);
        }
      };
      auto find = [&]() {
        for (;;) {
          if (w >= n_items) {
            nxt.live = 0;
            return;
          }
          bool some;
          if constexpr (FORM == kShared)
            some = decode_shared(a, w, nxt, nxt_gap);
          else if constexpr (FORM == kSharedFew)
            some = decode_planned(a, table, w, nxt, nxt_gap);
          else
            some = decode_item<PAGED, FORM>(a, numbered, n_items, w, nxt, nxt_gap);
          if (some) break;
          claim();
          w = claimed();
        }
        if (PAGED) nxt_id = ids_of(nxt, nxt_gap, nxt.kt0);
      };
      // Waits (lane 0) for ring slot e % R to be free and announces its copy.
      auto open_slot = [&]() -> bool {
        bool good = true;
        if (lane == 0) {
          good = mbar_wait(bar(kBarEmpty + e % R), ((e / R) & 1) ^ 1, abort_flag);
          if (good) mbar_arrive_expect_tx(bar(kBarFull + e % R), C::kTileBytes);
        }
        return __shfl_sync(~0u, good, 0);
      };
      if constexpr (FORM == kShared) {
        // The CTA's own item comes decoded (found like the others, it takes 0.6 us longer).
        nxt.live = 0;
        if (w < n_items) {
          static_assert(sizeof(Item) == 60, "four words of 16 bytes with the table column");
          int4 x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = a.start[4 * w + i];
          memcpy(&nxt, x, sizeof nxt);
          nxt_gap = {0, x[3].w};
          nxt_id = ids_of(nxt, nxt_gap, nxt.kt0);
        }
      } else {
        find();
      }
      for (int k = 0; ok; ++k) {
        const Item it = nxt;
        const Gap gap = nxt_gap;
        int ids = nxt_id, ids_next = 0;
        const int slot = k & 1;
        if (lane == 0) {
          ok = mbar_wait(bar(kBarItemEmpty + slot), ((k >> 1) & 1) ^ 1, abort_flag);
          if (ok) {
            misc->item[slot] = it;
            mbar_arrive(bar(kBarItemFull + slot));
          }
        }
        if (!(ok = __shfl_sync(~0u, ok, 0)) || !it.live) break;
        if (static_cast<int>(blockIdx.x) == a.fault_cta) {
          // Failure-path test: as if the item's copies were lost; the MMA warp's
          // bounded wait for them runs out.
          ok = false;
          break;
        }
        // Query tile t into the next Q buffer, once the last Q K^T of the tile
        // that was there has read it.
        auto load_q = [&](int t) -> bool {
          if (it.n[t] == 0) return true;
          bool good = true;
          const int buf = nq & 1;
          if (lane == 0) {
            good = mbar_wait(bar(kBarQEmpty + buf), ((nq >> 1) & 1) ^ 1, abort_flag);
            if (good) {
              mbar_arrive_expect_tx(bar(kBarQFull + buf), a.G * a.tpb * D * 2);
              for (int b = 0; b < C::kBoxes; ++b)
                tma_load_3d(s_base + C::kQ + buf * C::kTileBytes + b * C::kBoxBytes, &tm_q, b * 64,
                            it.kvh * a.G, it.row0 + t * a.tpb, bar(kBarQFull + buf));
            }
          }
          good = __shfl_sync(~0u, good, 0);
          if (good) ++nq;
          return good;
        };
        const int n_max = max(it.n[0], it.n[1]);
        for (int j = 0; j < n_max; ++j) {
          const int tile = it.kt0 + j;
          // The next item is claimed as late as its loads allow (an item held by a
          // CTA that is busy is lost to the others: 2 sequences of 4096, 16 heads,
          // 113 us when it was claimed at the start, 94 so), decoded behind the last copy.
          if (j == max(n_max - 2, 0)) claim();
          int pb = 0;
          if (PAGED) {
            if ((j & 3) == 0) {
              if (j > 0) ids = ids_next;
              if (j + 4 < n_max) ids_next = ids_of(it, gap, tile + 4);
            }
            pb = __shfl_sync(~0u, ids, (j & 3) * kTileBlocks + (lane & 7));
          }
          if (!(ok = open_slot())) break;
          const uint32_t k_dst = s_base + C::kRing + (e % R) * C::kTileBytes;
          const uint32_t k_bar = bar(kBarFull + e % R);
          if (PAGED) {
            if (lane < kTileBlocks)
              tma_load_5d(k_dst + lane * 4096, &tile_map(tm_k), 0, 0, 0, it.kvh, pb, k_bar);
          } else {
            load_rows(tm_k, it, gap, tile, k_dst, k_bar);
          }
          ++e;
          if (j == 0 && !(ok = load_q(0) && load_q(1))) break;
          if (!(ok = open_slot())) break;
          const uint32_t v_dst = s_base + C::kRing + (e % R) * C::kTileBytes;
          const uint32_t v_bar = bar(kBarFull + e % R);
          if (PAGED) {
            if (lane < kTileBlocks)
              tma_load_4d(v_dst + lane * 4096, &tile_map(tm_v), 0, 0, it.kvh, pb, v_bar);
          } else {
            load_rows(tm_v, it, gap, tile, v_dst, v_bar);
          }
          ++e;
        }
        if (!ok) break;
        if (n_max == 0) claim();
        w = claimed();
        find();
      }
      // (A claim in flight after an abort: its value is read before the exit
      // is counted.)
      if (!ok && claimed() < 0) *abort_flag = 1;
      if (!ok && lane == 0) {
        // Let the copies in flight land before the CTA exits.
        for (int i = (nq > 2 ? nq - 2 : 0); i < nq; ++i)
          drain_wait(bar(kBarQFull + (i & 1)), (i >> 1) & 1);
        for (int i = (e > R ? e - R : 0); i < e; ++i)
          drain_wait(bar(kBarFull + i % R), (i / R) & 1);
      }
    } else if (warp == 1 && elect_one()) {
      // ---------------------------------------------------------- MMA issuer
      constexpr uint32_t idesc_qk = idesc16<F16>(idesc_bf16_f32(BM, BN, false));
      constexpr uint32_t idesc_pv = idesc16<F16>(idesc_bf16_f32(BM, D, !PAGED));
      constexpr uint32_t k_hi = PAGED ? kHiPagedK : kSdescHi1024;
      constexpr uint32_t v_hi = PAGED ? kHiPagedV : kSdescHi1024;
      const uint32_t dq = sdesc_lo(s_base + C::kQ, 16);
      const uint32_t dk = sdesc_lo(s_base + C::kRing, PAGED ? 128 : 16);
      const uint32_t dv = sdesc_lo(s_base + C::kRing, PAGED ? 16 : C::kBoxBytes);
      // Tile kvi's keys are entry 2 kvi of the ring, its values 2 kvi + 1.
      auto wait_full = [&](int e) {
        return mbar_wait(bar(kBarFull + e % R), (e / R) & 1, abort_flag);
      };
      // S_t = Q_t K^T with Q tile qi (buffer qi & 1); `last`: Q is not needed again.
      auto qk = [&](int t, int qi, int kvi, bool last) -> bool {
        if (!wait_full(2 * kvi)) return false;
        tc_fence_after();
        const uint32_t qa = dq + (((qi & 1) * C::kTileBytes) >> 4);
        const uint32_t kb = dk + ((((2 * kvi) % R) * C::kTileBytes) >> 4);
        const uint32_t s_col = tmem + (t ? C::kColS1 : C::kColS0);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * C::kBoxBytes + (kk & 3) * 32) >> 4;
          mma_ss_hi(s_col, qa + off, kb + (PAGED ? (kk * 256) >> 4 : off), k_hi, idesc_qk,
                    kk > 0 ? 1u : 0u);
        }
        mma_commit(bar(kBarSFull + t));
        if (last) mma_commit(bar(kBarQEmpty + (qi & 1)));
        return true;
      };
      // Half h of O_T += P_T V: keys 64h .. 64h + 63 of the tile.
      auto pv = [&](int t, int kvi, bool first, int h) {
        const uint32_t vb = dv + ((((2 * kvi + 1) % R) * C::kTileBytes) >> 4);
        const uint32_t s_col = tmem + (t ? C::kColS1 : C::kColS0);
        const uint32_t o_col = tmem + (t ? C::kColO1 : C::kColO0);
#pragma unroll
        for (int kk = 4 * h; kk < 4 * h + 4; ++kk)
          mma_ts_hi(o_col, s_col + kk * 8, vb + ((kk * (PAGED ? 4096 : 2048)) >> 4), v_hi,
                    idesc_pv, (!first || kk > 0) ? 1u : 0u);
      };
      int nq = 0, np[2] = {0, 0}, kv = 0;
      // First Q K^T of an item's tile t: takes the next Q tile.
      auto first_qk = [&](int t, int n, int kvi, int &qi) -> bool {
        qi = nq++;
        if (!mbar_wait(bar(kBarQFull + (qi & 1)), (qi >> 1) & 1, abort_flag)) return false;
        return qk(t, qi, kvi, n == 1);
      };
      // P V of step j.
      auto pv_step = [&](int t, int n, int j, int kvj) -> bool {
        for (int h = 0; h < 2; ++h) {
          if (!mbar_wait(bar(kBarPReady + 2 * t + h), np[t] & 1, abort_flag)) return false;
          tc_fence_after();
          pv(t, kvj, j == 0, h);
        }
        ++np[t];
        if (j == n - 1) mma_commit(bar(kBarODone + t));
        return true;
      };
      // An item as the issuer sees it: key tiles of A and B.
      struct Step {
        int live, n_a, n_b;
      };
      auto fetch = [&](int k, Step &x) -> bool {
        if (!take_item(k, false)) return false;
        const volatile Item &i = item_of(k);
        x.live = i.live, x.n_a = i.n[0], x.n_b = i.n[1];
        free_item(k, false);
        return true;
      };
      Step it, nx;
      int qa = 0, qb = 0;       // Q tiles of the item's A and B
      int qa_next = 0;
      bool a0_issued = false;   // the item's first Q K^T of tile A went out a step early
      bool ok = fetch(0, it);
      for (int k = 0; ok && it.live; ++k) {
        const int n_max = max(it.n_a, it.n_b);
        if (a0_issued)
          qa = qa_next;
        else if (it.n_a > 0 && !(ok = first_qk(0, it.n_a, kv, qa)))
          break;
        a0_issued = false;
        if (it.n_b > 0 && !(ok = first_qk(1, it.n_b, kv, qb))) break;
        if (n_max > 0) mma_commit(bar(kBarEmpty + (2 * kv) % R));
        bool fetched = false;
        for (int j = 0; j < n_max; ++j) {
          const int kvj = kv + j, ev = 2 * kvj + 1, sv = ev % R;
          if (!(ok = wait_full(ev))) break;
          if (j < it.n_a) {
            if (!(ok = pv_step(0, it.n_a, j, kvj))) break;
            if (j + 1 < it.n_a && !(ok = qk(0, qa, kvj + 1, j + 2 == it.n_a))) break;
          }
          if (j == n_max - 1) {
            // S_A is free: the next item's tile A starts now.
            if (!(ok = fetch(k + 1, nx))) break;
            fetched = true;
            if (nx.live && nx.n_a > 0) {
              if (!(ok = first_qk(0, nx.n_a, kv + n_max, qa_next))) break;
              a0_issued = true;
            }
          }
          if (j < it.n_b && !(ok = pv_step(1, it.n_b, j, kvj))) break;
          mma_commit(bar(kBarEmpty + sv));
          if (j + 1 < it.n_b && !(ok = qk(1, qb, kvj + 1, j + 2 == it.n_b))) break;
          if (j + 1 < n_max) mma_commit(bar(kBarEmpty + (2 * kvj + 2) % R));
        }
        if (!ok) break;
        kv += n_max;
        if (!fetched && !(ok = fetch(k + 1, nx))) break;
        it = nx;
      }
      // Drain: every MMA issued above has completed once this phase does.
      mma_commit(bar(kBarDrain));
      drain_wait(bar(kBarDrain), 0);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // ------------------------------------------------------------ softmax
    const int t = (warp - 4) >> 2;                 // query tile: 0 = A, 1 = B
    const int quarter = warp & 3;                  // TMEM lanes 32*quarter .. +31
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t s_tmem = tmem + lane_off + (t ? C::kColS1 : C::kColS0);
    const uint32_t o_tmem = s_tmem + 256;
    const uint64_t c2 = f2(a.scale_log2, a.scale_log2);
    // The loop over key tiles has no register to spare: what an item's start and end
    // need is computed there, or read from the item again (8 prompts up to 4096: 189 us
    // with eleven registers spilled, 183.5 with one).
    auto row_in_tile = [&]() { return quarter * 32 + static_cast<int>(threadIdx.x & 31); };
    int phases = 0;   // bit 0: S's phase, bit 1: O's; above: key tiles of the items before
    bool ok = true;
    for (int k = 0; ok; ++k) {
      if (!(ok = take_item(k, true))) break;
      const volatile Item &it = item_of(k);
      if (!it.live) break;
      const int n_mine = it.n[t];
      // Keys below lim are visible to this row (the first is key 0 of the partition).
      const int lim = min(it.kv_len, it.pos0 + t * a.tpb + row_in_tile() / a.G + 1) - it.kt0 * BN;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < n_mine; ++j, phases ^= 1) {
        if (j == it.clear[t]) {
          const int e = 2 * ((phases >> 2) + j) + 1, st = e % R, keep = it.kv_len % BN, r = row_in_tile();
          if (!(ok = wait_warp(bar(kBarFull + st), (e / R) & 1, abort_flag))) break;
          uint8_t *v = smem + C::kRing + st * C::kTileBytes;
          if (PAGED) {
            // Only the block that the context ends in: the later ones of the
            // tile were read as zeros.  V^T rows are 16 tokens (32 bytes), the
            // two 16-byte halves of row r exchanged where r & 4.
            uint16_t *vr = reinterpret_cast<uint16_t *>(v + keep / kBlk * 4096 + r * 32);
            for (int u = keep % kBlk; u % kBlk != 0; ++u)
              vr[((((u >> 3) ^ (r >> 2)) & 1) << 3) + (u & 7)] = 0;
          } else {
            for (int i = r; i < (BN - keep) * 8; i += BM)
#pragma unroll
              for (int b = 0; b < C::kBoxes; ++b)
                *reinterpret_cast<uint4 *>(v + b * C::kBoxBytes + (keep + (i >> 3)) * 128 +
                                           (i & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();   // ahead of this warp's arrivals on PReady
        }
        if (!(ok = wait_warp(bar(kBarSFull + t), phases & 1, abort_flag))) break;
        tc_fence_after();
        uint32_t sv[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(s_tmem + c * 32, sv[c]);
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_wait_ld(sv[c]);
#define S_(c) sv[(c) >> 5][(c) & 31]
        if constexpr (FORM == kWindow) {
          // Keys from lim - window on, or among the first `sinks`, are visible.  (A row
          // that holds a query sees its own position: lim is that + 1.)
          const int lim_j = lim - j * BN, low_j = lim_j - a.window;
          const int first_j = a.sinks - (it.kt0 + j) * BN;
          if (__any_sync(~0u, lim_j < BN || low_j > max(first_j, 0))) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const uint32_t bits = ~high_bits(lim_j - 32 * w) &
                                    (high_bits(low_j - 32 * w) | ~high_bits(first_j - 32 * w));
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (((bits >> c) & 1u) == 0u) sv[w][c] = __float_as_uint(-INFINITY);
            }
          }
        }
        const int lim_j = lim - j * BN;
        if (FORM != kWindow && __any_sync(~0u, lim_j < BN)) {
#pragma unroll
          for (int w = 0; w < 4; ++w) {   // by bit masks: half the instructions of compares
            const int n = lim_j - 32 * w;
            const uint32_t bits = n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u;
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (((bits >> c) & 1u) == 0u) sv[w][c] = __float_as_uint(-INFINITY);
          }
        }
        float mx[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          mx[i] = fmaxf(__uint_as_float(S_(2 * i)), __uint_as_float(S_(2 * i + 1)));
#pragma unroll
        for (int c = 4; c < BN; c += 4)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            mx[i] = fmax3(mx[i], __uint_as_float(S_(c + 2 * i)), __uint_as_float(S_(c + 2 * i + 1)));
        const float tmax = fmaxf(mx[0], mx[1]) * a.scale_log2;
        float alpha = 1.f;
        if (tmax > m + kRescaleThreshold) {  // also true while m = -inf
          alpha = ex2_approx(m - tmax);
          m = tmax;
        }
        // P V of tile j - 1 was issued before Q K^T of tile j: O_T is complete.
        if (j > 0 && __any_sync(~0u, alpha != 1.f)) {
          const uint64_t a2 = f2(alpha, alpha);
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t ov[32];
            tmem_ld32(o_tmem + c * 32, ov);
            tmem_wait_ld(ov);
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 x =
                  f2_split(fmul2(f2(__uint_as_float(ov[e]), __uint_as_float(ov[e + 1])), a2));
              ov[e] = __float_as_uint(x.x);
              ov[e + 1] = __float_as_uint(x.y);
            }
            tmem_st32(o_tmem + c * 32, ov);
          }
        }
        // A row that has seen no key yet has m = -inf: a finite number in its place
        // gives its (all masked) scores p = 0 rather than NaN.
        const float nmv = fminf(-m, FLT_MAX);
        const uint64_t nm2 = f2(nmv, nmv);
        uint64_t sum2[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 x = f2_split(
                ffma2(f2(__uint_as_float(sv[c][e]), __uint_as_float(sv[c][e + 1])), c2, nm2));
            const float2 p = make_float2(ex2_approx(x.x), ex2_approx(x.y));
            sum2[(e >> 1) & 1] = fadd2(sum2[(e >> 1) & 1], f2(p.x, p.y));
            // Rounded to the element type: the MMA takes no wider A operand.
            pk[e >> 1] = pack2<F16>(p.x, p.y);
          }
          tmem_st16(s_tmem + c * 16, pk);
          if (c & 1) {
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kBarPReady + 2 * t + (c >> 1)));
          }
        }
#undef S_
        const float2 sa = f2_split(fadd2(sum2[0], sum2[1]));
        l = l * alpha + (sa.x + sa.y);
      }
      if (!ok) break;
      // (Read here: the loop above has no registers to keep these.)
      phases += 4 * max(it.n[0], it.n[1]);
      const int part = PAGED && it.split ? it.part : -1;   // -1: the context is not cut
      // This row's place in the output, [token][head]; -1: it holds no query.
      const int my_tok = row_in_tile() / a.G;
      const int row = it.row0 + t * a.tpb + my_tok;
      const int head = it.kvh * a.G + row_in_tile() - my_tok * a.G;
      const int my_out = my_tok < min(it.n_tok[t], a.tpb) ? row * a.H + head : -1;
      const bool sees = min(it.kv_len, it.pos0 + t * a.tpb + my_tok + 1) > 0;
      free_item(k, true);
      // Epilogue, once the last P V is done.  A tile without key tiles writes
      // zeros if it has none at all, and nothing if other partitions have them.
      const bool some = n_mine > 0;
      if (!some && part > 0) continue;
      if (some) {
        if (!(ok = wait_warp(bar(kBarODone + t), (phases >> 1) & 1, abort_flag))) break;
        phases ^= 2;
        tc_fence_after();
      }
      if (PAGED && part >= 0) {
        // Unnormalised fp32 rows, a thread's own row from its registers (the few
        // rows of a split block do not repay staging them).
        const int64_t base = static_cast<int64_t>(part) * a.T * a.H;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t ov[32];
          tmem_ld32(o_tmem + c * 32, ov);
          tmem_wait_ld(ov);
          if (my_out >= 0) {
            float *dst = a.ws_o + (base + my_out) * D + c * 32;
#pragma unroll
            for (int q = 0; q < 4; ++q) store32(dst + 8 * q, &ov[8 * q]);
          }
        }
        if (my_out >= 0) a.ws_ml[base + my_out] = make_float2(m, l);
        continue;
      }
      const float inv_l = 1.f / l;
      // Packed, d = 128: through shared memory, eight lanes a row (8 prompts up to 4096:
      // 181 us; with a thread's own row from its registers, as the others, 186).  d = 64
      // and paged from the registers (32 prompts up to 200, d = 64: 15.9 us, 17.0 through
      // shared memory).
      constexpr bool kStaged = !PAGED && D == 128;
      // What an item's end keeps in registers moves the whole loop's: all keys, d = 128,
      // rows are normalised one value an instruction and lse's place is reckoned from the
      // output's (one prompt of 16384, fp16: 311 us, 318 otherwise; chunks over 16384 91.2, 92.0;
      // the other forms lose by it: 8 prompts with a window 262.5 for 261.6).
      constexpr bool kPlainEnd = D == 128 && FORM == kAll;
      uint8_t *stg = smem + C::kStage + (t * 4 + quarter) * 4096;
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
        uint32_t ov[2][32];
        // (Loaded for a tile without keys too, whose rows are set to zero below:
        // a branch around the loads makes the compiler keep copies of them.)
        tmem_ld32(o_tmem + 64 * h, ov[0]);
        tmem_ld32(o_tmem + 64 * h + 32, ov[1]);
        tmem_wait_ld(ov[0]);
        tmem_wait_ld(ov[1]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t *c16 = &ov[q >> 1][(q & 1) * 16];
          uint32_t v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (kPlainEnd) {
              v[e] = pack2<F16>(__uint_as_float(c16[2 * e]) * inv_l,
                                __uint_as_float(c16[2 * e + 1]) * inv_l);
            } else {
              const float2 x = f2_split(fmul2(f2(__uint_as_float(c16[2 * e]),
                                                 __uint_as_float(c16[2 * e + 1])),
                                              f2(inv_l, inv_l)));
              v[e] = pack2<F16>(x.x, x.y);
            }
          }
          // A row that sees no key is zero whatever its accumulator holds.  Packed, a
          // query sees itself at least: a sum of 0 means scores that are all -inf, NaN
          // (as inv_l makes it; without the select the compiler's registers cost 1%).
          if (PAGED ? !sees : l == 0.f)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = PAGED ? 0u : ~0u;
          if (kStaged) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
              *reinterpret_cast<uint4 *>(stg + lane * 128 + (((2 * q + e) ^ (lane & 7)) * 16)) =
                  make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
          } else if (my_out >= 0) {
            store32(a.o + static_cast<int64_t>(my_out) * D + 64 * h + q * 16, v);
          }
        }
        if (!kStaged) continue;
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int rr = (lane >> 3) + 4 * q, ch = lane & 7;
          const uint4 v = *reinterpret_cast<const uint4 *>(stg + rr * 128 + ((ch ^ (rr & 7)) * 16));
          const int out_row = __shfl_sync(~0u, my_out, rr);
          if (out_row >= 0)
            *reinterpret_cast<uint4 *>(a.o + static_cast<int64_t>(out_row) * D + 64 * h + ch * 8) =
                v;
        }
        __syncwarp();
      }
      if (!PAGED && a.lse != nullptr && my_out >= 0)
        a.lse[kPlainEnd ? static_cast<int64_t>(my_out % a.H) * a.T + my_out / a.H
                        : static_cast<int64_t>(head) * a.T + row] =
            (m + __log2f(l)) * 0.6931471805599453f;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (threadIdx.x == 0) {
    if (misc->abort) atomicExch(a.dev_status, kDevTimeout);
    // The last CTA to finish returns the counters to zero for the next launch.
    __threadfence();
    if (atomicAdd(a.sched + 1, 1) == static_cast<int>(gridDim.x) - 1) {
      a.sched[0] = 0;
      a.sched[1] = 0;
      __threadfence();
    }
  }
}

// Joins the partitions of the rows whose context was cut: gridDim.y blocks per
// sequence (which end at once if it was not), one warp per (token, head), four
// dimensions a lane.  By sequence, because a grid over all rows costs 40 us where few
// are cut; 4 us for 16 chunks of up to 6 tokens, 32 heads, of which the rows' loads
// are the smaller part and the launch and the chain of (max, sum) the larger.
// SPREAD (shared prefixes, where every row of a sharing sequence is joined, and long
// chunks): all tokens spread evenly over eight blocks an SM, a warp joining `merge_heads`
// heads of each.  By sequence the longest chunk's rows are the call's tail there (32 chunks up
// to 300 behind 4096 tokens: 173 us, 139 so), but with few rows it is 1 - 3 us quicker.
constexpr int kMergeSeqs = 1024;        // sequences that a block keeps in shared memory
template <int FORM, bool SPREAD>
__global__ void __launch_bounds__(256) paged_merge_kernel(const FormArgs<FORM> a) {
  constexpr int D = kDecodeHeadSize;
  // The next kernel of the stream may be scheduled: it waits for this grid.
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // Nothing in global memory is read ahead of the wait, the bounds included: only behind
  // it are another kernel's writes sure to be visible.  (Bounds read ahead of it took 1 us off
  // 16 drafts over up to 4096, 33.2 against 34.3.)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  Seq q;
  int cut = 1, pre = 0;                                  // partitions; those of the prefix
  if constexpr (FORM == kShared && !SPREAD) {
    const int4 x = a.seq[2 * blockIdx.x], y = a.seq[2 * blockIdx.x + 1];
    q = {x.x, x.y, x.z, x.w};
    cut = y.x, pre = y.y;
  } else if constexpr (FORM != kShared) {
    // The call's work, as number_items adds it up, and the sequence's partitions, by one
    // warp (every block asks L2 for the same few lines).
    __shared__ Seq shared_seq;
    __shared__ int shared_cut;
    if (threadIdx.x < 32) {
      const Seq q = global_seq<true>(a, blockIdx.x);
      const Work own = work_of<FORM>(a, q);
      int64_t work = 0, work_short = 0;
      for (int i = lane; i < a.S; i += 32) {
        const Work w = work_of<FORM>(a, global_seq<true>(a, i));
        work += static_cast<int64_t>(w.tiles) * w.blocks;
        if (FORM == kWindow && w.blocks == 1) work_short += w.tiles;
      }
      work = warp_sum(work);
      if (FORM == kWindow) {
        work_short = min(work, 8 * warp_sum(work_short));
        if (own.blocks == 1) work = work_short;
      }
      if (lane == 0) {
        shared_seq = q;
        shared_cut = parts_of(a, q, own.tiles, work, a.n_split);
      }
    }
    __syncthreads();
    q = shared_seq;
    cut = shared_cut;
  }
  if (!SPREAD && cut == 1 && pre == 0) return;           // written directly
  const int64_t stride = static_cast<int64_t>(a.T) * a.H;
  // Row `row` of the output: token i of the sequence.
  auto join = [&](int i, int64_t row) {
    // The block's last token sets the partitions' size, the row's own those it is in.
    const int block = i / (2 * a.tpb), last = min((block + 1) * 2 * a.tpb, q.n) - 1;
    const int gap =
        FORM == kWindow ? gap_of<FORM>(a, q.pos + block * 2 * a.tpb).skip * kCell : 0;
    const int size = part_size(tiles_for(1, q.pos + last - gap, q.kv_len - gap), cut);
    const int own = (tiles_for(1, q.pos + i - gap, q.kv_len - gap) + size - 1) / size;
    const int parts = own + pre;
    // Partition p's place: the prefix's lie behind the most that a context has.
    auto place = [&](int p) -> int64_t {
      return FORM == kShared && p >= own ? a.n_split + p - own : p;
    };
    auto part_row = [&](int p) {
      return *reinterpret_cast<const float4 *>(a.ws_o + (place(p) * stride + row) * D + lane * 4);
    };
    // kShared: the first partitions' rows are loaded ahead of the (max, sum) that weigh
    // them (64 requests behind 8192 tokens: 38.5 us, 40.6 without; but 16 drafts over up to
    // 4096, cut without a prefix, 33.8 so and 33.0 without).
    constexpr int kAhead = FORM == kShared ? 8 : 0;
    float4 ahead[kAhead + 1];
#pragma unroll
    for (int p = 0; p < kAhead; ++p)
      if (p < parts) ahead[p] = part_row(p);
    // 32 partitions at a time, lane p holding partition p's (max, sum): their rows'
    // loads do not wait for one another.
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p0 = 0; p0 < parts; p0 += 32) {
      const int n = min(32, parts - p0);
      float2 ml = make_float2(-INFINITY, 0.f);
      if (lane < n) ml = a.ws_ml[place(p0 + lane) * stride + row];
      float mx = ml.x;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, off));
      mx = fmaxf(mx, m);
      // No score so far but NaN, which a maximum passes over, or -inf: the sums are NaN,
      // which the row has to become, or 0.
      const bool none = mx == -INFINITY;
      const float f = none ? 0.f : ex2_approx(ml.x - mx), old = none ? 1.f : ex2_approx(m - mx);
      float sum = f * ml.y;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(~0u, sum, off);
      l = fmaf(l, old, sum);
      if (none) continue;
      o.x *= old, o.y *= old, o.z *= old, o.w *= old;
      m = mx;
      auto add = [&](int p, const float4 &v) {
        const float w = __shfl_sync(~0u, f, p);
        o.x = fmaf(w, v.x, o.x), o.y = fmaf(w, v.y, o.y);
        o.z = fmaf(w, v.z, o.z), o.w = fmaf(w, v.w, o.w);
      };
      if (p0 == 0)
#pragma unroll
        for (int p = 0; p < kAhead; ++p)
          if (p < n) add(p, ahead[p]);
      const float *src = a.ws_o + (p0 * stride + row) * D + lane * 4;
#pragma unroll 16
      for (int p = p0 == 0 ? kAhead : 0; p < n; ++p)
        add(p, FORM == kShared ? part_row(p0 + p)
                               : *reinterpret_cast<const float4 *>(src + p * stride * D));
    }
    const float inv = parts == 0 ? 0.f : 1.f / l;        // a query that sees no key: zeros
    uint2 w;
    w.x = pack_bf16x2(o.x * inv, o.y * inv);
    w.y = pack_bf16x2(o.z * inv, o.w * inv);
    *reinterpret_cast<uint2 *>(a.o + row * D + lane * 4) = w;
  };
  const int warp = threadIdx.x >> 5;
  if constexpr (SPREAD) {
    __shared__ int4 seqs[2 * kMergeSeqs];
    const bool kept = a.S <= kMergeSeqs;
    if (kept) {
      bool any = false;
      for (int i = threadIdx.x; i < 2 * a.S; i += 256) {
        const int4 x = seqs[i] = a.seq[i];
        any |= i % 2 == 1 && (x.x > 1 || x.y > 0);
      }
      if (!__syncthreads_or(any)) return;                // all written directly
    }
    const int4 *of = kept ? seqs : a.seq;
    const uint32_t parts = (a.H + a.merge_heads - 1) / a.merge_heads;   // of a token's heads
    const uint32_t units = a.T * parts;
    for (uint32_t x = blockIdx.x * 8 + warp; x < units; x += gridDim.x * 8) {
      const int tok = x / parts, h0 = x % parts * a.merge_heads;
      // The last sequence that begins at or before the token owns it, if any does.
      const int s = warp_search(a.S, tok, [&](int j) { return of[2 * j].x; });
      if (s < 0) continue;
      const int4 u = of[2 * s], v = of[2 * s + 1];
      q = {u.x, u.y, u.z, u.w};
      cut = v.x, pre = v.y;
      if (tok - q.begin >= q.n || (cut == 1 && pre == 0)) continue;
      for (int h = h0; h < min(h0 + a.merge_heads, a.H); ++h)
        join(tok - q.begin, static_cast<int64_t>(tok) * a.H + h);
    }
  } else {
    for (int x = blockIdx.y * 8 + warp; x < q.n * a.H; x += gridDim.y * 8)
      join(x / a.H, static_cast<int64_t>(q.begin) * a.H + x);
  }
}

// Numbers the items of a call with shared prefixes of many sequences (one block).
constexpr int kPlanThreads = 1024, kClasses = 32;
__global__ void __launch_bounds__(kPlanThreads) shared_plan_kernel(const SharedArgs a) {
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  using Plan = Planner<kPlanThreads, kSharedMaxGroups>;
  __shared__ Plan::Scratch scratch;
  __shared__ int firsts[kPlanThreads];                     // of the first entries
  __shared__ unsigned long long classes[kClasses];
  __shared__ int n_entries;
  const int tid = threadIdx.x;
  if (tid < kClasses) classes[tid] = 0;
  Plan plan(a, scratch);
  // Items by size, largest first, in classes of 1 .. 15 key tiles, then of half powers of
  // two; a class's counter holds its entries (high word) and items.
  auto class_of = [&](int size) {
    const int log = 31 - __clz(size);
    return kClasses - 1 -
           (size < 16 ? size : min(16 + 2 * (log - 4) + ((size >> (log - 1)) & 1), kClasses - 1));
  };
  auto count_of = [&](const PlanEntry &x) {
    return (1ull << 32) + static_cast<unsigned long long>(x.w.blocks * x.parts * a.Hk);
  };
  for (int s = tid; s < a.S + a.P; s += kPlanThreads) {
    const PlanEntry x = plan.entry_of(s);
    if (x.w.blocks > 0) atomicAdd(&classes[class_of(part_size(x.w.tiles, x.parts))], count_of(x));
  }
  __syncthreads();
  if (tid < kClasses) {
    const unsigned long long n = classes[tid];
    unsigned long long sum = n;
#pragma unroll
    for (int off = 1; off < kClasses; off <<= 1) {
      const unsigned long long below = __shfl_up_sync(~0u, sum, off);
      if (tid >= off) sum += below;
    }
    classes[tid] = sum - n;
    if (tid == kClasses - 1) {
      n_entries = static_cast<int>(sum >> 32);
      *a.head = n_entries;
      a.first[n_entries] = static_cast<int>(sum);
    }
  }
  __syncthreads();
  for (int s = tid; s < a.S + a.P; s += kPlanThreads) {
    const PlanEntry x = plan.entry_of(s);
    if (s < a.S) plan.put_seq(s, x);
    if (x.w.blocks == 0) continue;
    const unsigned long long at =
        atomicAdd(&classes[class_of(part_size(x.w.tiles, x.parts))], count_of(x));
    const int i = static_cast<int>(at >> 32);
    a.first[i] = static_cast<int>(at);
    if (i < kPlanThreads) firsts[i] = static_cast<int>(at);
    a.rec[2 * i] = make_int4(x.q.begin, x.q.n, x.q.kv_len, x.q.pos);
    a.rec[2 * i + 1] = make_int4(x.row, x.col, x.parts, x.slot);
  }
  __syncthreads();
  // The first item of each CTA, decoded.  (Every entry has an item: they are among the
  // first entries.)
  for (int w = tid; w < a.ctas && w < a.first[n_entries]; w += kPlanThreads) {
    int lo = 0, n = min(n_entries, kPlanThreads);
    while (n > 1) {
      const int half = n / 2;
      if (firsts[lo + half] <= w) lo += half, n -= half;
      else n = half;
    }
    Item it = {};
    Gap gap;
    decode_entry(a, a.rec[2 * lo], a.rec[2 * lo + 1], w - firsts[lo], it, gap);
    int4 x[4];
    memcpy(x, &it, sizeof it);
    x[3].w = gap.skip;
#pragma unroll
    for (int i = 0; i < 4; ++i) a.start[4 * w + i] = x[i];
  }
}

cudaError_t sm_count(int *n) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
  return e;
}

template <int D, bool F16, bool PAGED, int FORM>
cudaError_t launch(const CUtensorMap &tq, const KvMap<PAGED, FORM> &tk,
                   const KvMap<PAGED, FORM> &tv, const FormArgs<FORM> &a, cudaStream_t stream) {
  using C = Cfg<D, PAGED>;
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(fwd_packed_kernel<D, F16, PAGED, FORM>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, C::kAlloc);
  if (e != cudaSuccess) return e;
  int64_t n_items = static_cast<int64_t>(a.n_vblocks) * a.n_split * a.Hk;   // a bound
  if constexpr (is_shared(FORM)) {
    sms = a.ctas;
    n_items += (static_cast<int64_t>(a.T) / (2 * a.tpb) + a.P) * a.pre_split * a.Hk;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(n_items < sms ? n_items : sms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kAlloc;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, fwd_packed_kernel<D, F16, PAGED, FORM>, tq, tk, tv, a);
  if (e != cudaSuccess || !PAGED || (!is_shared(FORM) && a.n_split == 1)) return e;
  // Eight blocks an SM in all, spread over the sequences (at most kCachedSeqs; with
  // shared prefixes any number) or the tokens.
  cfg.gridDim = dim3(static_cast<unsigned>(a.S), static_cast<unsigned>(std::max(8 * sms / a.S, 1)));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  if constexpr (is_shared(FORM)) {
    if (a.merge_heads == 0) return cudaLaunchKernelEx(&cfg, paged_merge_kernel<kShared, false>, a);
    cfg.gridDim = dim3(static_cast<unsigned>(8 * sms));
    return cudaLaunchKernelEx(&cfg, paged_merge_kernel<kShared, true>, a);
  } else {
    return cudaLaunchKernelEx(&cfg, paged_merge_kernel<FORM, false>, a);
  }
}

template <int FORM>
cudaError_t launch_packed_form(const CUtensorMap &tq, const KvMap<false, FORM> &tk,
                               const KvMap<false, FORM> &tv, const FormArgs<FORM> &a, int d,
                               bool f16, cudaStream_t stream) {
  if (d == 64)
    return f16 ? launch<64, true, false, FORM>(tq, tk, tv, a, stream)
               : launch<64, false, false, FORM>(tq, tk, tv, a, stream);
  return f16 ? launch<128, true, false, FORM>(tq, tk, tv, a, stream)
             : launch<128, false, false, FORM>(tq, tk, tv, a, stream);
}

Args args_of(const PackedProblem &p, int *sched, int *dev_status, int fault_cta) {
  Args a{};
  a.o = static_cast<uint16_t *>(p.o);
  a.lse = p.lse;
  a.cu_seqlens = p.cu_seqlens;
  a.context_lens = p.context_lens;
  a.block_tables = p.block_tables;
  a.sched = sched;
  a.dev_status = dev_status;
  a.fault_cta = fault_cta;
  a.S = p.S, a.T = p.T, a.H = p.H, a.Hk = p.Hk, a.G = p.H / p.Hk;
  a.tpb = packed_tile_tokens(a.G);
  a.max_blocks = p.max_blocks, a.num_blocks = p.num_blocks;
  a.n_vblocks = packed_blocks(p.T, p.S, a.G);
  a.n_split = 1;
  a.causal = p.causal;
  a.scale_log2 = p.scale * 1.4426950408889634f;
  return a;
}

WindowArgs window_args(const Args &a, const PackedProblem &p) {
  WindowArgs w;
  static_cast<Args &>(w) = a;
  w.window = p.window, w.sinks = p.sinks;
  return w;
}

}  // namespace

int packed_tile_tokens(int group) { return BM / group; }

int packed_blocks(int T, int S, int group) { return T / (2 * packed_tile_tokens(group)) + S; }

cudaError_t launch_fwd_packed(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                              const PackedProblem &p, int d, bool f16, int *sched,
                              int *dev_status, int fault_cta, cudaStream_t stream) {
  const Args a = args_of(p, sched, dev_status, fault_cta);
  if (p.window == 0) return launch_packed_form<kAll>(tq, tk, tv, a, d, f16, stream);
  return launch_packed_form<kWindow>(tq, CellMaps{tk, *p.k_cells}, CellMaps{tv, *p.v_cells},
                                     window_args(a, p), d, f16, stream);
}

// The most partitions of a context, from what the host knows (the longest one's
// bound): as parts_of reckons for a sequence of one token that is alone, and no more
// than a workspace of 256 MB holds -- with that many rows the blocks fill the GPU.
// Beyond kCachedSeqs sequences, whose bounds and numbering do not fit the barrier area,
// nothing is cut: a long context among short ones is then one chain of its key tiles
// (131072 tokens among 1024s, 32 / 8 heads: 169 us with 112 sequences, 1350 with 113).
int paged_max_parts(int T, int S, int H, int Hk, int max_blocks, int window, int sinks) {
  if (S > kCachedSeqs) return 1;
  double tiles = (max_blocks + kTileBlocks - 1) / kTileBlocks;
  // With a window, a block's list of key tiles is that long at most.
  if (window > 0)
    tiles = std::fmin(tiles, std::ceil((window + 2.0 * packed_tile_tokens(H / Hk) + sinks +
                                        2 * kCell) / BN));
  const double least = std::fmax(4.0, std::sqrt(tiles * Hk / 152 * 2.5 / 0.7));
  const double room = 256e6 / (sizeof(float) * (kDecodeHeadSize + 2.0) * T * H);
  if (tiles < 1.5 * least) return 1;   // parts_of never cuts so few
  const double n = std::fmin(std::fmin(tiles / least + 1, room), 32767);
  return n < 1 ? 1 : static_cast<int>(n);
}

size_t paged_prefill_workspace_bytes(int T, int S, int H, int Hk, int max_blocks, int window,
                                     int sinks) {
  const int n = paged_max_parts(T, S, H, Hk, max_blocks, window, sinks);
  if (n == 1) return 0;
  return static_cast<size_t>(n) * T * H * (kDecodeHeadSize + 2) * sizeof(float);
}

cudaError_t launch_paged_prefill(const CUtensorMap &tq, const CUtensorMap &tk,
                                 const CUtensorMap &tv, const PackedProblem &p, float *workspace,
                                 int *sched, int *dev_status, int fault_cta,
                                 cudaStream_t stream) {
  Args a = args_of(p, sched, dev_status, fault_cta);
  const int n = paged_max_parts(p.T, p.S, p.H, p.Hk, p.max_blocks, p.window, p.sinks);
  if (n > 1) {
    a.n_split = n;
    a.ws_o = workspace;
    a.ws_ml = reinterpret_cast<float2 *>(workspace + static_cast<size_t>(n) * p.T * p.H *
                                                         kDecodeHeadSize);
  }
  if (p.window == 0) return launch<128, false, true, kAll>(tq, tk, tv, a, stream);
  return launch<128, false, true, kWindow>(tq, tk, tv, window_args(a, p), stream);
}

// Workspace of a call with shared prefixes: partial rows (at least one of a row's own
// context and one of its prefix, more as far as 256 MB reach), then the plan.
SharedLayout shared_layout(int T, int S, int P, int H, int Hk, int max_blocks) {
  SharedLayout l{};
  const double tiles = (max_blocks + kTileBlocks - 1) / kTileBlocks;
  const double least = std::fmax(4.0, std::sqrt(tiles * Hk / 152 * 2.5 / 0.7));
  const double room = 256e6 / 2 / (sizeof(float) * (kDecodeHeadSize + 2.0) * T * H);
  const double n = std::fmin(std::fmin(tiles / least + 1, room), 32767);
  l.split = n < 1 ? 1 : static_cast<int>(n);
  l.pre_split = P > 0 ? l.split : 0;
  const size_t rows = static_cast<size_t>(l.split + l.pre_split) * T * H;
  auto take = [&](size_t bytes) {
    const size_t at = l.bytes;
    l.bytes += (bytes + 15) / 16 * 16;
    return at;
  };
  const size_t entries = static_cast<size_t>(S) + P;
  l.rows = take(rows * kDecodeHeadSize * sizeof(float));
  l.sums = take(rows * sizeof(float2));
  l.rec = take(entries * 2 * sizeof(int4));
  l.seq = take(static_cast<size_t>(S) * 2 * sizeof(int4));
  l.first = take((entries + 1) * sizeof(int));
  l.head = take(sizeof(int));
  l.start = take(static_cast<size_t>(kSharedMaxCtas) * sizeof(int4) * 4);
  return l;
}

cudaError_t launch_paged_shared(const CUtensorMap &tq, const CUtensorMap &tk,
                                const CUtensorMap &tv, const PackedProblem &p,
                                const int *cu_groups, const int *prefix_lens, int P,
                                char *workspace, int *sched, int *dev_status, int fault_cta,
                                cudaStream_t stream) {
  const SharedLayout l = shared_layout(p.T, p.S, P, p.H, p.Hk, p.max_blocks);
  SharedArgs a;
  static_cast<Args &>(a) = args_of(p, sched, dev_status, fault_cta);
  a.n_split = l.split, a.pre_split = l.pre_split;
  a.ws_o = reinterpret_cast<float *>(workspace + l.rows);
  a.ws_ml = reinterpret_cast<float2 *>(workspace + l.sums);
  a.rec = reinterpret_cast<int4 *>(workspace + l.rec);
  a.seq = reinterpret_cast<int4 *>(workspace + l.seq);
  a.first = reinterpret_cast<int *>(workspace + l.first);
  a.head = reinterpret_cast<int *>(workspace + l.head);
  a.start = reinterpret_cast<int4 *>(workspace + l.start);
  a.cu_groups = cu_groups, a.prefix_lens = prefix_lens, a.P = P;
  cudaError_t e = sm_count(&a.ctas);
  if (e != cudaSuccess) return e;
  a.ctas = std::min(a.ctas, kSharedMaxCtas);
  // The merge spreads the tokens over its 64 warps an SM where they have two rows each and the
  // sequences eight tokens on average (with fewer, the longest is no tail).
  const int64_t rows = static_cast<int64_t>(p.T) * p.H, warps = 64 * a.ctas;
  a.merge_heads = rows >= 2 * warps && p.T / 8 >= p.S
                      ? static_cast<int>(std::clamp<int64_t>(rows / warps, 1, p.H))
                      : 0;
  if (p.S + P <= kCachedSeqs) return launch<128, false, true, kSharedFew>(tq, tk, tv, a, stream);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, shared_plan_kernel, a);
  if (e != cudaSuccess) return e;
  return launch<128, false, true, kShared>(tq, tk, tv, a, stream);
}

}  // namespace fattn
