// fwd_packed.cu -- exact attention of several queries per sequence for
// sequences of different lengths in one call, with grouped key/value heads,
// on the sm_103a tensor cores:
//   packed   prompts packed one after another, q [T, H, d], k and v [T, Hk, d],
//            sequence s in rows cu_seqlens[s] .. cu_seqlens[s+1] - 1, every
//            query against its own sequence's keys (causal or not);
//   paged    a chunk of new queries per sequence, q [T, H, d], against the
//            paged cache that holds the sequence's whole context (the chunk's
//            own keys included): query i of n sees keys 0 .. ctx - n + i.
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
//
// What bounds it: for long prompts the tensor pipe and the softmax chain (S out of
// TMEM, exponentials, P back) of a two-tile step, 1.4 us where the MMAs alone take
// 1.37; for chunks of one query tile that chain alone, 1.3 us a key tile; for a few
// tokens over long contexts the 16 copies of a paged key tile and HBM; for short
// prompts the start (5 us) and the chain of an SM's few items.  Measured: 8 prompts up
// to 4096 tokens, 32 / 8 heads, d = 128, causal, 182 us (1497 TFLOP/s); one of 16384,
// 8 / 1 heads, fp16, 330 us (1665); 32 prompts up to 200, 16 heads, d = 64, 17 us;
// chunks of 4 x 1024 tokens over 8192, 345 us (1494 TFLOP/s), up to 1024 over up to
// 16384, 94 us; 64 single tokens over 4096, 180 us (6.0 TB/s).
// Rounding: P to the element type before P V, O once at the end; scores, maxima, sums,
// partial rows and their merge are fp32.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstdint>

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

// Key tiles that `n` tokens, the last of which sees key `last` last, visit.
__device__ __forceinline__ int tiles_for(int n, int last, int kv_len) {
  return n > 0 ? (max(0, min(kv_len, last + 1)) + BN - 1) / BN : 0;
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

// Work of a sequence: key tiles of its last block, and blocks.
struct Work {
  int tiles, blocks;
};
__device__ __forceinline__ Work work_of(const Args &a, const Seq &q) {
  return {tiles_for(q.n, q.pos + q.n - 1, q.kv_len), (q.n + 2 * a.tpb - 1) / (2 * a.tpb)};
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
// number.)
__device__ __forceinline__ int parts_of(const Args &a, const Seq &q, int tiles, int64_t work) {
  constexpr float kFixed = 2.5f, kRow = 0.02f, kLeast = 4.f;
  if (a.n_split == 1) return 1;
  const float w = __fmul_rn(__ll2float_rn(work * a.Hk), 1.f / (152.f * 0.7f));
  const float c = __fmaf_rn(kRow, static_cast<float>(min(q.n, 2 * a.tpb) * a.G), kFixed);
  const float size = fmaxf(__fsqrt_rn(__fmul_rn(w, c)), kLeast);
  const float n = __fdiv_rn(static_cast<float>(tiles), size);
  return n < 1.5f ? 1 : min(__float2int_ru(n), a.n_split);
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
template <bool PAGED>
__device__ __forceinline__ void number_items(const Args &a, Misc *m) {
  const int lane = threadIdx.x & 31;
  auto seq = [&](int i) {
    return make_seq(a, PAGED, m->seq[i].x, m->seq[i + 1].x, m->seq[i].y);
  };
  int64_t work = 0;
  if (PAGED && a.n_split > 1) {
#pragma unroll 1
    for (int i = lane; i < a.S; i += 32) {
      const Work w = work_of(a, seq(i));
      work += static_cast<int64_t>(w.tiles) * w.blocks;
    }
    work = warp_sum(work);
  }
  // Key: key tiles of an item, then the index, so that no two are equal.
#pragma unroll 1
  for (int i = lane; i < a.S; i += 32) {
    const Seq q = seq(i);
    const int tiles = work_of(a, q).tiles;
    const int parts = PAGED ? parts_of(a, q, tiles, work) : 1;
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
    m->first[rank] = work_of(a, seq(i)).blocks * m->n_parts[i] * a.Hk;
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

// Item w of n_items (whole warp); false if it has no work.  m: the numbered
// sequences, or null.
template <bool PAGED>
__device__ __forceinline__ bool decode_item(const Args &a, const Misc *m, int n_items, int w,
                                            Item &it) {
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
  it.kv_len = q.kv_len;
  it.kv0 = PAGED ? s : q.begin;
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

// A wait that all lanes of the warp leave with one answer.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t ph, volatile int *abort_flag) {
  return __all_sync(~0u, mbar_wait(bar, ph, abort_flag));
}

__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t ph) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, ph) && globaltimer_ns() - t0 < kWaitLimitNs) {
  }
}

template <int D, bool F16, bool PAGED>
__global__ void __launch_bounds__(kThreads, 1)
    fwd_packed_kernel(const __grid_constant__ CUtensorMap tm_q,
                      const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const Args a) {
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
  const bool cached = a.S <= kCachedSeqs;
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
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
      }
      if (cached) {
        number_items<PAGED>(a, misc);
      }
      const Misc *numbered = cached ? misc : nullptr;
      const int n_items = cached ? misc->first[a.S] : a.n_vblocks * a.Hk;
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
      int nxt_id = 0;           // paged: block id of the item's block `lane`
      auto ids_of = [&](const Item &it, int tile) -> int {
        // Lane i: block i of the four key tiles from `tile` on; past the
        // context, a block that the cache does not have (reads as zeros).
        const int b = tile * kTileBlocks + lane;
        if (b >= (it.kv_len + kBlk - 1) / kBlk) return a.num_blocks;
        return a.block_tables[static_cast<int64_t>(it.kv0) * a.max_blocks + b];
      };
      auto find = [&]() {
        for (;;) {
          if (w >= n_items) {
            nxt.live = 0;
            return;
          }
          if (decode_item<PAGED>(a, numbered, n_items, w, nxt)) break;
          claim();
          w = claimed();
        }
        if (PAGED) nxt_id = ids_of(nxt, nxt.kt0);
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
      find();
      for (int k = 0; ok; ++k) {
        const Item it = nxt;
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
              if (j + 4 < n_max) ids_next = ids_of(it, tile + 4);
            }
            pb = __shfl_sync(~0u, ids, (j & 3) * kTileBlocks + (lane & 7));
          }
          if (!(ok = open_slot())) break;
          const uint32_t k_dst = s_base + C::kRing + (e % R) * C::kTileBytes;
          const uint32_t k_bar = bar(kBarFull + e % R);
          if (PAGED) {
            if (lane < kTileBlocks)
              tma_load_5d(k_dst + lane * 4096, &tm_k, 0, 0, 0, it.kvh, pb, k_bar);
          } else if (lane == 0) {
            for (int b = 0; b < C::kBoxes; ++b)
              tma_load_3d(k_dst + b * C::kBoxBytes, &tm_k, b * 64, it.kv0 + tile * BN, it.kvh,
                          k_bar);
          }
          ++e;
          if (j == 0 && !(ok = load_q(0) && load_q(1))) break;
          if (!(ok = open_slot())) break;
          const uint32_t v_dst = s_base + C::kRing + (e % R) * C::kTileBytes;
          const uint32_t v_bar = bar(kBarFull + e % R);
          if (PAGED) {
            if (lane < kTileBlocks)
              tma_load_4d(v_dst + lane * 4096, &tm_v, 0, 0, it.kvh, pb, v_bar);
          } else if (lane == 0) {
            for (int b = 0; b < C::kBoxes; ++b)
              tma_load_3d(v_dst + b * C::kBoxBytes, &tm_v, b * 64, it.kv0 + tile * BN, it.kvh,
                          v_bar);
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
        const int lim_j = lim - j * BN;
        if (__any_sync(~0u, lim_j < BN)) {
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
            uint4 *dst = reinterpret_cast<uint4 *>(a.ws_o + (base + my_out) * D + c * 32);
#pragma unroll
            for (int q = 0; q < 8; ++q)
              dst[q] = make_uint4(ov[4 * q], ov[4 * q + 1], ov[4 * q + 2], ov[4 * q + 3]);
          }
        }
        if (my_out >= 0) a.ws_ml[base + my_out] = make_float2(m, l);
        continue;
      }
      const float inv_l = 1.f / l;
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
        for (int q = 0; q < 8; ++q) {
          const uint32_t *c8 = &ov[q >> 2][(q & 3) * 8];
          uint4 v;
          v.x = pack2<F16>(__uint_as_float(c8[0]) * inv_l, __uint_as_float(c8[1]) * inv_l);
          v.y = pack2<F16>(__uint_as_float(c8[2]) * inv_l, __uint_as_float(c8[3]) * inv_l);
          v.z = pack2<F16>(__uint_as_float(c8[4]) * inv_l, __uint_as_float(c8[5]) * inv_l);
          v.w = pack2<F16>(__uint_as_float(c8[6]) * inv_l, __uint_as_float(c8[7]) * inv_l);
          // A row that sees no key is zero whatever its accumulator holds.  Packed, a
          // query sees itself at least: a sum of 0 means scores that are all -inf, NaN
          // (as inv_l makes it; without the select the compiler's registers cost 1%).
          if (PAGED ? !sees : l == 0.f)
            v = PAGED ? make_uint4(0u, 0u, 0u, 0u) : make_uint4(~0u, ~0u, ~0u, ~0u);
          if (!PAGED)
            *reinterpret_cast<uint4 *>(stg + lane * 128 + ((q ^ (lane & 7)) * 16)) = v;
          else if (my_out >= 0)
            *reinterpret_cast<uint4 *>(a.o + static_cast<int64_t>(my_out) * D + 64 * h + q * 8) = v;
        }
        if (PAGED) continue;
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
        a.lse[static_cast<int64_t>(my_out % a.H) * a.T + my_out / a.H] =
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
__global__ void __launch_bounds__(256) paged_merge_kernel(const Args a) {
  constexpr int D = kDecodeHeadSize;
  // The next kernel of the stream may be scheduled: it waits for this grid.
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // Nothing in global memory is read ahead of the wait, the bounds included: only behind
  // it are another kernel's writes sure to be visible.  (Bounds read ahead of it took 1 us off
  // 16 drafts over up to 4096, 33.2 against 34.3.)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // The call's work, as number_items adds it up, and the sequence's partitions, by one
  // warp (every block asks L2 for the same few lines).
  const int lane = threadIdx.x & 31;
  __shared__ Seq shared_seq;
  __shared__ int shared_cut;
  if (threadIdx.x < 32) {
    int64_t work = 0;
    for (int i = lane; i < a.S; i += 32) {
      const Work w = work_of(a, global_seq<true>(a, i));
      work += static_cast<int64_t>(w.tiles) * w.blocks;
    }
    work = warp_sum(work);
    const Seq q = global_seq<true>(a, blockIdx.x);
    if (lane == 0) {
      shared_seq = q;
      shared_cut = parts_of(a, q, work_of(a, q).tiles, work);
    }
  }
  __syncthreads();
  const Seq q = shared_seq;
  const int cut = shared_cut;
  if (cut == 1) return;                                  // written directly
  const int64_t stride = static_cast<int64_t>(a.T) * a.H;
  for (int x = blockIdx.y * 8 + (threadIdx.x >> 5); x < q.n * a.H; x += gridDim.y * 8) {
    const int i = x / a.H;                               // token of the sequence
    const int64_t row = static_cast<int64_t>(q.begin) * a.H + x;
    // The block's last token sets the partitions' size, the row's own those it is in.
    const int last = min((i / (2 * a.tpb) + 1) * 2 * a.tpb, q.n) - 1;
    const int size = part_size(tiles_for(1, q.pos + last, q.kv_len), cut);
    const int parts = (tiles_for(1, q.pos + i, q.kv_len) + size - 1) / size;
    // 32 partitions at a time, lane p holding partition p's (max, sum): their rows'
    // loads do not wait for one another.
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p0 = 0; p0 < parts; p0 += 32) {
      const int n = min(32, parts - p0);
      float2 ml = make_float2(-INFINITY, 0.f);
      if (lane < n) ml = a.ws_ml[(p0 + lane) * stride + row];
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
      const float *src = a.ws_o + (p0 * stride + row) * D + lane * 4;
#pragma unroll 16
      for (int p = 0; p < n; ++p) {
        const float4 v = *reinterpret_cast<const float4 *>(src + p * stride * D);
        const float w = __shfl_sync(~0u, f, p);
        o.x = fmaf(w, v.x, o.x), o.y = fmaf(w, v.y, o.y);
        o.z = fmaf(w, v.z, o.z), o.w = fmaf(w, v.w, o.w);
      }
    }
    const float inv = parts == 0 ? 0.f : 1.f / l;        // a query that sees no key: zeros
    uint2 w;
    w.x = pack_bf16x2(o.x * inv, o.y * inv);
    w.y = pack_bf16x2(o.z * inv, o.w * inv);
    *reinterpret_cast<uint2 *>(a.o + row * D + lane * 4) = w;
  }
}

cudaError_t sm_count(int *n) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
  return e;
}

template <int D, bool F16, bool PAGED>
cudaError_t launch(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, Args a,
                   cudaStream_t stream) {
  using C = Cfg<D, PAGED>;
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(fwd_packed_kernel<D, F16, PAGED>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, C::kAlloc);
  if (e != cudaSuccess) return e;
  const int64_t n_items = static_cast<int64_t>(a.n_vblocks) * a.n_split * a.Hk;   // a bound
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
  e = cudaLaunchKernelEx(&cfg, fwd_packed_kernel<D, F16, PAGED>, tq, tk, tv, a);
  if (e != cudaSuccess || !PAGED || a.n_split == 1) return e;
  // Eight blocks an SM in all, spread over the sequences (at most kCachedSeqs).
  cfg.gridDim = dim3(static_cast<unsigned>(a.S), static_cast<unsigned>(8 * sms / a.S));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, paged_merge_kernel, a);
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

}  // namespace

int packed_tile_tokens(int group) { return BM / group; }

int packed_blocks(int T, int S, int group) { return T / (2 * packed_tile_tokens(group)) + S; }

cudaError_t launch_fwd_packed(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                              const PackedProblem &p, int d, bool f16, int *sched,
                              int *dev_status, int fault_cta, cudaStream_t stream) {
  const Args a = args_of(p, sched, dev_status, fault_cta);
  if (d == 64)
    return f16 ? launch<64, true, false>(tq, tk, tv, a, stream)
               : launch<64, false, false>(tq, tk, tv, a, stream);
  return f16 ? launch<128, true, false>(tq, tk, tv, a, stream)
             : launch<128, false, false>(tq, tk, tv, a, stream);
}

// The most partitions of a context, from what the host knows (the longest one's
// bound): as parts_of reckons for a sequence of one token that is alone, and no more
// than a workspace of 256 MB holds -- with that many rows the blocks fill the GPU.
// Beyond kCachedSeqs sequences, whose bounds and numbering do not fit the barrier area,
// nothing is cut: a long context among short ones is then one chain of its key tiles
// (131072 tokens among 1024s, 32 / 8 heads: 169 us with 112 sequences, 1350 with 113).
int paged_max_parts(int T, int S, int H, int Hk, int max_blocks) {
  if (S > kCachedSeqs) return 1;
  const double tiles = (max_blocks + kTileBlocks - 1) / kTileBlocks;
  const double least = std::fmax(4.0, std::sqrt(tiles * Hk / 152 * 2.5 / 0.7));
  const double room = 256e6 / (sizeof(float) * (kDecodeHeadSize + 2.0) * T * H);
  const double n = std::fmin(std::fmin(tiles / least + 1, room), 32767);
  return n < 1 ? 1 : static_cast<int>(n);
}

size_t paged_prefill_workspace_bytes(int T, int S, int H, int Hk, int max_blocks) {
  const int n = paged_max_parts(T, S, H, Hk, max_blocks);
  if (n == 1) return 0;
  return static_cast<size_t>(n) * T * H * (kDecodeHeadSize + 2) * sizeof(float);
}

cudaError_t launch_paged_prefill(const CUtensorMap &tq, const CUtensorMap &tk,
                                 const CUtensorMap &tv, const PackedProblem &p, float *workspace,
                                 int *sched, int *dev_status, int fault_cta,
                                 cudaStream_t stream) {
  Args a = args_of(p, sched, dev_status, fault_cta);
  const int n = paged_max_parts(p.T, p.S, p.H, p.Hk, p.max_blocks);
  if (n > 1) {
    a.n_split = n;
    a.ws_o = workspace;
    a.ws_ml = reinterpret_cast<float2 *>(workspace + static_cast<size_t>(n) * p.T * p.H *
                                                         kDecodeHeadSize);
  }
  return launch<128, false, true>(tq, tk, tv, a, stream);
}

}  // namespace fattn
