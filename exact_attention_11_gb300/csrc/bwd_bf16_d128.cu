// bwd_bf16_d128.cu -- the main backward kernel for head dimension 128: the
// same arithmetic as bwd_main_kernel in bwd_bf16.cu (recomputation scheme of
// "FlashAttention: GPU 메모리 계층을 활용한 어텐션 최적화 분석", youngju.dev,
// section 7: P = exp(S - LSE), dV = P^T dO, dP = dO V^T, dS = P (dP - D),
// dQ = scale dS K, dK = scale dS^T Q), scheduled so that the tensor cores and
// the CUDA cores work at the same time.
//
// One CTA per (128-key block j, head) keeps K_j, V_j in shared memory and
// dV_j, dK_j (fp32) in TMEM.  Each 128-query step is split into two 64-query
// sub-tiles t = 0, 1, each owned by one group of four warps.  While group t
// turns S_t, dP_t into P_t, dS_t, the MMA warp works on the other sub-tile,
// so the two groups take turns ("ping-pong"), as the forward kernel's two
// query tiles do.  Per sub-tile (TMEM region R_t = [128t, 128t+128)):
//   S_t^T  = K_j Q_t^T  -> R_t[0,64)      dP_t^T = V_j dO_t^T -> R_t[64,128)
//   group t: P_t^T = exp2(S^T scale log2e - LSE2) and dS_t^T = P^T (dP^T - D)
//            as packed bf16 at R_t[0,32) and R_t[32,64); dS^T also to shared
//            memory (128-byte swizzle, keys as rows)
//   dQ_t'^T = K_j^T dS_t^T -> R_t[64,128) (lanes = d, columns = queries)
//   dV_j += P_t^T dO_t,  dK_j += dS_t^T Q_t            (A operands from TMEM)
//   group t reads dQ_t'^T out of TMEM and adds it to the fp32 dQ accumulator
//   with TMA reduces: each warp stages its 32 d x 64 queries as two
//   [query][d] boxes in its own quarter of the dS^T buffer, which dQ_t'^T has
//   finished reading and the group only writes again in its next element
//   step.
// The kernel is bound by shared-memory bandwidth (MMA operands, TMA writes,
// dS stores), so operands come from TMEM wherever the TMEM budget allows.
// MMA order per sub-tile: dQ'_t, dV_t, dK_t, then S_t, dP_t of the next step
// (after group t has released R_t), then the other sub-tile.  Q and dO
// arrive as 64-row halves through 4-slot rings, two steps ahead.
//
// The CTAs are persistent (one per SM): the producer claims (key block,
// head) items from a device-wide counter, heaviest first, and hands them to
// the other roles through a two-entry ring in shared memory.  Every barrier
// keeps counting across items.  At an item boundary the producer loads the
// next item's first Q and dO halves as soon as ring slots free up and its K
// and V once the last MMA of the current item has read theirs; the MMA warp
// starts the next item's first S and dP while the groups write the current
// item's dV and dK, and its first dV, dK products wait only for the groups
// to have read those accumulators out of TMEM.
//
// PACKED (fa_backward_packed): sequences of different lengths one after
// another, grouped key/value heads.  An item is (key block of a sequence, query
// head), found in the table that the preparation kernel wrote; inside it, key
// and query indices count from the sequence's start, and only the TMA
// coordinates and output rows add the sequence's place.  A tile that the
// sequence ends in also holds the next one's rows: a warp of the producer
// warpgroup clears them in shared memory (K, V, Q and dO: a zero weight does not
// cancel a NaN) before the MMA warp may use the tile.  The dQ accumulator is
// padded to whole blocks per sequence, so that no tile's rows fall on another
// sequence's.  The query heads of a group are items of their own, as a group
// would make the causal kernel's heaviest items too long to balance; they add
// their dK, dV to fp32 accumulators with TMA reduces, or, with one query head
// per key/value head, store them as the dense kernel does.
// kWindow (fa_backward_packed_window): an item comes with the query blocks that it
// visits; a query sees a key if it is at most window - 1 behind or among the first
// `sinks` (bwd_tile.cuh's masks by bits, in the blocks that either border crosses).
// kWindowGroups: an item may have all query heads of its key/value head, one after another:
// K and V are loaded once, dK and dV add up in TMEM and are stored.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "bwd_tile.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace fattn {
namespace {

constexpr int D = 128;
constexpr int BM = 128;      // keys per CTA
constexpr int BQ = 128;      // queries per step
constexpr int BH_ = 64;      // queries per sub-tile
constexpr int kSlots = 4;    // Q / dO half-tile ring depth
constexpr int kThreads = 384;
constexpr uint32_t kRegsLoad = 104, kRegsGroup = 200;
static_assert(kRegsLoad + 2 * kRegsGroup == 3 * 168,
              "the warpgroup register split must use exactly the launch budget");
constexpr uint32_t kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f;

// Shared memory (offsets from a 1024-byte aligned base; the kernel checks
// that the dynamic shared memory it is given starts on such a boundary).
constexpr int kTile = BM * D * 2;          // 32 KB: K or V
constexpr int kHalf = BH_ * D * 2;         // 16 KB: a 64-row half of Q or dO
constexpr int kHalfBox = BH_ * 128;        // 8 KB: 64 rows x 128 bytes (64 of d)
constexpr int kKeyBox = BM * 128;          // 16 KB: 128 rows x 128 bytes
constexpr int kOffK = 0;
constexpr int kOffV = kOffK + kTile;
constexpr int kOffQ = kOffV + kTile;                 // kSlots halves
constexpr int kOffDO = kOffQ + kSlots * kHalf;       // kSlots halves
constexpr int kOffDS = kOffDO + kSlots * kHalf;      // 2 x 16 KB (per sub-tile)
constexpr int kDSBytes = BM * BH_ * 2;               // 16 KB
constexpr int kOffVec = kOffDS + 2 * kDSBytes;       // kSlots x [LSE2 64 | D 64] f32
constexpr int kVecBytes = 2 * BH_ * 4;               // 512 B
constexpr int kOffBar = kOffVec + kSlots * kVecBytes;
constexpr int kSmemBytes = kOffBar + 512;
static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");

constexpr int kRowBoxes = D / 64;                     // 128-byte boxes per row

enum : int {
  kBarKV = 0,
  kBarQFull = 1,        // + slot
  kBarQEmpty = 5,       // + slot
  kBarDOFull = 9,       // + slot
  kBarDOEmpty = 13,     // + slot
  kBarSFull = 17,       // + t
  kBarPReady = 19,      // + t, 4 warps
  kBarDQFull = 21,      // + t
  kBarTmemFree = 23,    // + t, 4 warps: dQ'_t read out of TMEM
  kBarKVDone = 25,      // every MMA of the item is complete (K, V free; dV, dK final)
  kBarDrain = 26,
  kBarEpiDone = 27,     // 8 warps: the item's dV, dK have been read out of TMEM
  kBarItemFull = 28,    // + ring slot (2)
  kBarItemEmpty = 30,   // + ring slot (2)
  kBarFix = 32,         // + slot, PACKED: a ragged half of Q and dO has been cleared
  kBarKVFix = 36,       // PACKED: a ragged key block has been cleared
  kNumBars = 38         // even: Misc, which follows, holds 16-byte values
};
// Arrivals that free an item-ring slot: the MMA thread and the 8 group warps
// (PACKED: and the clearing warp).
constexpr int kItemConsumers = 1 + 8;

struct Misc {
  uint32_t tmem_base;
  int abort;
  int item[2];
  int4 seq[2];          // PACKED: the item's entry of the block table
  int4 range[2];        // WINDOW: first query block, their number, first head, heads
};
static_assert(kNumBars * 8 + sizeof(Misc) <= 512 && kNumBars % 2 == 0, "barrier area");

__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t ph, volatile int *abort_flag) {
  return __all_sync(~0u, mbar_wait(bar, ph, abort_flag));
}

__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t ph) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, ph) && globaltimer_ns() - t0 < kWaitLimitNs) {
  }
}

// Status latched when the dynamic shared memory does not start on a 1024-byte
// boundary (the layout above assumes it; the kernel then does nothing).
constexpr int kDevBadSmemBase = -2;

// An item: key block jb of head bh (items heaviest first: under the causal
// mask key block 0 is visited by every query block).  Indices of keys and
// queries count from the sequence's first row, which is row0 of the tensors
// (PACKED; else 0); N is its length.
struct BwdItem {
  int jb, bh, k0, i_first, n_steps, n_halves, N;
  int kvh, row0, blk0;   // PACKED: key/value head, first row, first padded block
  int per;               // kWindowGroups: steps of a query head
  __device__ void decode(int w, int BH, int n_qb, int causal, int N_) {
    jb = w / BH;
    bh = kvh = w - jb * BH;
    N = N_;
    row0 = blk0 = 0;
    steps(n_qb, causal);
  }
  // Entry w / H of the table, e = (first row, length, first padded block, key block).
  __device__ void decode_packed(int w, const int4 &e, int H, int G, int causal) {
    const int blk = w / H;
    bh = w - blk * H;
    kvh = bh / G;
    row0 = e.x;
    N = e.y;
    blk0 = e.z;
    jb = e.w;
    steps((N + BQ - 1) / BQ, causal);
  }
  __device__ void set_steps(int first, int n) {
    i_first = first;
    n_steps = n;
    n_halves = 2 * n;
  }
  __device__ void set_range(const int4 &r, int G) {
    i_first = r.x;
    per = r.y;
    bh = r.z;
    kvh = bh / G;
    n_steps = per * r.w;
    n_halves = 2 * n_steps;
  }
  __device__ void steps(int n_qb, int causal) {
    k0 = jb * BM;
    i_first = causal ? jb : 0;
    n_steps = n_qb - i_first;
    n_halves = 2 * n_steps;
  }
};

// What the kernel runs on: [B, H, N, d] tensors, packed sequences, or packed sequences
// with a window, whose items have one query head, or some of them all heads of a group
// (two kernels: in one, items of one head took 3 - 5% longer).
enum : int { kDense = 0, kPacked = 1, kWindow = 2, kWindowGroups = 3 };
template <int KIND>
using Extra = std::conditional_t<KIND >= kWindow, BwdWindow, BwdPacked>;

template <int KIND>
__global__ void __launch_bounds__(kThreads, 1)
    bwd_pipe_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                    const __grid_constant__ CUtensorMap tm_dq,
                    const float *__restrict__ vecs,
                    __nv_bfloat16 *__restrict__ dk, __nv_bfloat16 *__restrict__ dv, int N, int BH,
                    float scale, int causal, int *__restrict__ sched, int fault_cta,
                    int *__restrict__ dev_status, const __grid_constant__ CUtensorMap tm_dk,
                    const __grid_constant__ CUtensorMap tm_dv, const Extra<KIND> pk) {
  constexpr bool PACKED = KIND != kDense, WINDOW = KIND >= kWindow, GROUPS = KIND == kWindowGroups;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t s_base = smem_u32(smem);
  if ((s_base & 1023u) != 0) {
    if (threadIdx.x == 0) atomicExch(dev_status, kDevBadSmemBase);
    return;
  }
  const uint32_t bars = s_base + kOffBar;
  auto bar = [&](int i) { return bars + 8u * i; };
  Misc *misc = reinterpret_cast<Misc *>(smem + kOffBar + 8 * kNumBars);
  volatile int *abort_flag = &misc->abort;
  // PACKED: BH is the number of query heads; vecs and the accumulators count
  // padded blocks.
  const int n_qb = PACKED ? pk.n_blocks : (N + BQ - 1) / BQ;
  int n_items = n_qb * BH;
  if constexpr (WINDOW) n_items = pk.entries * BH;

  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    mbar_init(bar(kBarKV), 1);
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(bar(kBarQFull + s), 1);
      mbar_init(bar(kBarQEmpty + s), PACKED ? 2 : 1);   // PACKED: and the clearing warp
      mbar_init(bar(kBarDOFull + s), 1);
      mbar_init(bar(kBarDOEmpty + s), PACKED ? 2 : 1);
      if (PACKED) mbar_init(bar(kBarFix + s), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(kBarSFull + t), 1);
      mbar_init(bar(kBarPReady + t), 4);
      mbar_init(bar(kBarDQFull + t), 1);
      mbar_init(bar(kBarTmemFree + t), 4);
      mbar_init(bar(kBarItemFull + t), 1);
      mbar_init(bar(kBarItemEmpty + t), kItemConsumers + (PACKED ? 1 : 0));
    }
    if (PACKED) mbar_init(bar(kBarKVFix), 1);
    mbar_init(bar(kBarKVDone), PACKED ? 2 : 1);
    mbar_init(bar(kBarDrain), 1);
    mbar_init(bar(kBarEpiDone), 8);
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
  // A programmatic dependent of the preparation kernel: its set-up above
  // overlaps that kernel's tail; no global memory is touched before this wait.
  // The dQ kernel may be scheduled once every block of this one is past it.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // Consumer side of the item ring: waits for entry k and frees it (one
  // arrival per warp, or the lone MMA thread).
  auto fetch_item = [&](int k, int &w, BwdItem &it, bool whole_warp) -> bool {
    const int slot = k & 1;
    if (!mbar_wait(bar(kBarItemFull + slot), (k >> 1) & 1, abort_flag)) return false;
    w = *reinterpret_cast<volatile int *>(&misc->item[slot]);
    if (PACKED) {
      const volatile int *e = reinterpret_cast<const volatile int *>(&misc->seq[slot]);
      it.decode_packed(w, make_int4(e[0], e[1], e[2], e[3]), BH, pk.group, causal);
      const volatile int *r = reinterpret_cast<const volatile int *>(&misc->range[slot]);
      if (GROUPS) it.set_range(make_int4(r[0], r[1], r[2], r[3]), pk.group);
      else if (WINDOW) it.set_steps(r[0], r[1]);
    } else {
      it.decode(w, BH, n_qb, causal, N);
    }
    if (whole_warp) __syncwarp();
    if (!whole_warp || (threadIdx.x & 31) == 0) mbar_arrive(bar(kBarItemEmpty + slot));
    return true;
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLoad));
    if (warp == 0 && elect_one()) {
      // ---------------------------------------------------------- TMA producer
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
      tma_prefetch_desc(&tm_do);
      int nq = 0, ndo = 0, nkv = 0;   // halves (and K/V pairs) issued so far
      bool ok = true;
      // kWindowGroups: the first entry and item of those with all heads of a group, the first
      // behind them; and the number of items.
      int from = 0, to = 0, n_from = 0, n_to = 0, n_used = 0;
      if constexpr (WINDOW && !GROUPS) n_used = pk.count[0] * BH;
      if constexpr (GROUPS) {
        const int4 count = *reinterpret_cast<const int4 *>(pk.count);
        from = count.y;
        to = from + count.z;
        n_from = from * BH;
        n_to = n_from + count.z * pk.kv_heads;
        n_used = n_to + (count.x - to) * BH;
      }
      auto claim = [&]() { return static_cast<int>(gridDim.x) + atomicAdd(sched, 1); };
      for (int k = 0; ok; ++k) {
        const int islot = k & 1;
        if (!(ok = mbar_wait(bar(kBarItemEmpty + islot), ((k >> 1) & 1) ^ 1, abort_flag))) break;
        // The CTA's own first item, then claimed ones.
        int w = k == 0 ? static_cast<int>(blockIdx.x) : claim();
        int4 entry = make_int4(0, 0, 0, 0);
        int4 range = make_int4(0, 0, 0, 0);
        if (PACKED) {
          auto in_table = [&](int x) { return WINDOW && x >= n_used ? n_items : x; };
          int at = 0;
          auto entry_of = [&](int x) {
            if (!GROUPS || x < n_from) at = x / BH;
            else if (x < n_to) at = from + (x - n_from) / pk.kv_heads;
            else at = to + (x - n_to) / BH;
            return at;
          };
          w = in_table(w);
          // Entries of length 0 end a sorted table, else are passed over.
          while (w < n_items && (entry = pk.table[entry_of(w)]).y == 0)
            w = pk.sorted ? n_items : in_table(claim());
          if constexpr (WINDOW)
            if (w < n_items) {
              const int2 blocks = pk.range[at];
              const bool all = GROUPS && at >= from && at < to;
              const int head = all ? (w - n_from - (at - from) * pk.kv_heads) * pk.group
                                   : at < from ? w - at * BH : w - n_to - (at - to) * BH;
              range = make_int4(blocks.x, blocks.y, head, all ? pk.group : 1);
            }
          // (Offsets that decrease leave entries unwritten: whatever they hold, the
          // item stays inside the tensors.)
          entry.x = min(max(entry.x, 0), pk.tokens - 1);
          entry.y = min(max(entry.y, 1), pk.tokens - entry.x);
          const int n_kb = (entry.y + BM - 1) / BM;
          entry.z = min(max(entry.z, 0), max(pk.n_blocks - n_kb, 0));
          entry.w = min(max(entry.w, 0), n_kb - 1);
          misc->seq[islot] = entry;
          if (WINDOW) {
            range.x = min(max(range.x, 0), n_kb - 1);
            range.y = min(max(range.y, 1), n_kb - range.x);
            misc->range[islot] = range;
          }
        }
        misc->item[islot] = w;
        mbar_arrive(bar(kBarItemFull + islot));
        if (w >= n_items) break;
        BwdItem it;
        if (PACKED) {
          it.decode_packed(w, entry, BH, pk.group, causal);
          if (GROUPS) it.set_range(range, pk.group);
          else if (WINDOW) it.set_steps(range.x, range.y);
        } else
          it.decode(w, BH, n_qb, causal, N);
        const int h_base = nq;
        int first_h = 0, head = it.bh;   // the head, and the half that it begins with
        // Q / dO half h of the item (with its [LSE2 | D] vectors on QFull).
        auto load_half = [&](int h) -> bool {
          const int g = h_base + h, slot = g % kSlots, use = g / kSlots;
          if (GROUPS && h - first_h == 2 * it.per) first_h = h, ++head;
          const int qb = it.i_first + ((h - first_h) >> 1);
          const int qrow = qb * BQ + (h & 1) * BH_;
          if (!mbar_wait(bar(kBarQEmpty + slot), (use & 1) ^ 1, abort_flag)) return false;
          mbar_arrive_expect_tx(bar(kBarQFull + slot), kHalf + kVecBytes);
          for (int b = 0; b < 2; ++b)
            tma_load_3d(s_base + kOffQ + slot * kHalf + b * kHalfBox, &tm_q, b * 64,
                        it.row0 + qrow, head, bar(kBarQFull + slot));
          const float *vsrc =
              vecs + (static_cast<int64_t>(head) * n_qb + it.blk0 + qb) * (2 * BQ) + (h & 1) * BH_;
          bulk_load(s_base + kOffVec + slot * kVecBytes, vsrc, BH_ * 4, bar(kBarQFull + slot));
          bulk_load(s_base + kOffVec + slot * kVecBytes + BH_ * 4, vsrc + BQ, BH_ * 4,
                    bar(kBarQFull + slot));
          nq = g + 1;
          if (!mbar_wait(bar(kBarDOEmpty + slot), (use & 1) ^ 1, abort_flag)) return false;
          mbar_arrive_expect_tx(bar(kBarDOFull + slot), kHalf);
          for (int b = 0; b < 2; ++b)
            tma_load_3d(s_base + kOffDO + slot * kHalf + b * kHalfBox, &tm_do, b * 64,
                        it.row0 + qrow, head, bar(kBarDOFull + slot));
          ndo = g + 1;
          return true;
        };
        // The first two halves as soon as ring slots free up; K and V once
        // the previous item's last MMA has read them.
        for (int h = 0; h < 2 && h < it.n_halves && ok; ++h) ok = load_half(h);
        if (!ok) break;
        if (static_cast<int>(blockIdx.x) == fault_cta) {
          // Failure-path test: stop here, as if the K and V copies were lost;
          // the MMA warp's bounded wait for them runs out.
          ok = false;
          break;
        }
        if (k > 0 && !(ok = mbar_wait(bar(kBarKVDone), (k - 1) & 1, abort_flag))) break;
        mbar_arrive_expect_tx(bar(kBarKV), 2 * kTile);
        for (int b = 0; b < 2; ++b) {
          tma_load_3d(s_base + kOffK + b * kKeyBox, &tm_k, b * 64, it.row0 + it.k0, it.kvh, bar(kBarKV));
          tma_load_3d(s_base + kOffV + b * kKeyBox, &tm_v, b * 64, it.row0 + it.k0, it.kvh, bar(kBarKV));
        }
        nkv = k + 1;
        for (int h = 2; h < it.n_halves && ok; ++h) ok = load_half(h);
      }
      if (!ok) {
        if (nkv > 0) drain_wait(bar(kBarKV), (nkv - 1) & 1);
        for (int g = (nq > kSlots ? nq - kSlots : 0); g < nq; ++g)
          drain_wait(bar(kBarQFull + g % kSlots), (g / kSlots) & 1);
        for (int g = (ndo > kSlots ? ndo - kSlots : 0); g < ndo; ++g)
          drain_wait(bar(kBarDOFull + g % kSlots), (g / kSlots) & 1);
      }
    } else if (warp == 1 && elect_one()) {
      // ---------------------------------------------------------- MMA issuer
      // Fully unrolled issue with 32-bit descriptor words: a rolled loop
      // costs the issuing thread about 60 cycles per MMA, more than an
      // M = 128, N = 64 MMA takes on the tensor core.
      constexpr uint32_t idesc_s = idesc_bf16_f32(BM, BH_, false);        // S^T, dP^T
      constexpr uint32_t idesc_q = idesc_bf16_f32(D, BH_, true, true);    // dQ'^T
      constexpr uint32_t idesc_g = idesc_bf16_f32(BM, D, true);           // dV, dK
      const uint32_t k_kmaj = sdesc_lo(s_base + kOffK, 16);
      const uint32_t v_kmaj = sdesc_lo(s_base + kOffV, 16);
      const uint32_t k_mn = sdesc_lo(s_base + kOffK, kKeyBox);   // K^T, M = d
      const uint32_t q_kmaj = sdesc_lo(s_base + kOffQ, 16);
      const uint32_t q_mn = sdesc_lo(s_base + kOffQ, kHalfBox);  // N = d
      const uint32_t do_kmaj = sdesc_lo(s_base + kOffDO, 16);
      const uint32_t do_mn = sdesc_lo(s_base + kOffDO, kHalfBox);
      const uint32_t ds_mn = sdesc_lo(s_base + kOffDS, kDSBytes); // dS^T as B
      // S_t^T = K Q_t^T and dP_t^T = V dO_t^T of ring half g into R_{h & 1}.
      auto issue_sdp = [&](int h, int g) {
        const uint32_t R = tmem + 128u * (h & 1);
        const uint32_t so = static_cast<uint32_t>((g % kSlots) * kHalf) >> 4;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t ok_ = static_cast<uint32_t>((kk >> 2) * kKeyBox + (kk & 3) * 32) >> 4;
          const uint32_t oh = static_cast<uint32_t>((kk >> 2) * kHalfBox + (kk & 3) * 32) >> 4;
          mma_ss_lo(R, k_kmaj + ok_, q_kmaj + so + oh, idesc_s, kk > 0 ? 1u : 0u);
          mma_ss_lo(R + 64, v_kmaj + ok_, do_kmaj + so + oh, idesc_s, kk > 0 ? 1u : 0u);
        }
        mma_commit(bar(kBarSFull + (h & 1)));
      };
      // Half h of an item (ring half g): Q and dO have landed and, where the
      // sequence ends inside the half or before it, have been cleared.
      uint32_t fix_parity = 0;   // bit: ring slot
      int kv_fixes = 0;
      int first_h = 0;           // kWindowGroups: the half that the last one's head begins with
      auto wait_half = [&](const BwdItem &it, int h, int g) -> bool {
        const int slot = g % kSlots;
        if (!mbar_wait(bar(kBarQFull + slot), (g / kSlots) & 1, abort_flag)) return false;
        if (!mbar_wait(bar(kBarDOFull + slot), (g / kSlots) & 1, abort_flag)) return false;
        if (GROUPS && h - first_h == 2 * it.per) first_h = h;
        if (PACKED && (it.i_first * BQ + (h - first_h + 1) * BH_ > it.N)) {
          if (!mbar_wait(bar(kBarFix + slot), (fix_parity >> slot) & 1, abort_flag)) return false;
          fix_parity ^= 1u << slot;
        }
        return true;
      };
      bool ok = true;
      int g0 = 0;       // ring halves of the earlier items
      int steps = 0;    // steps (per sub-tile) of the earlier items
      for (int k = 0; ok; ++k) {
        int w;
        BwdItem it;
        if (!(ok = fetch_item(k, w, it, false)) || w >= n_items) break;
        first_h = 0;
        if (!(ok = mbar_wait(bar(kBarKV), k & 1, abort_flag))) break;
        if (PACKED && it.k0 + BM > it.N) {
          if (!(ok = mbar_wait(bar(kBarKVFix), kv_fixes & 1, abort_flag))) break;
          ++kv_fixes;
        }
        // The item's first S_t, dP_t: R_t must have been read out (the dQ'_t
        // of the previous item's last step).
        for (int h = 0; h < 2 && h < it.n_halves && ok; ++h) {
          const int g = g0 + h;
          if (steps > 0 && !(ok = mbar_wait(bar(kBarTmemFree + h), (steps - 1) & 1, abort_flag)))
            break;
          if (!(ok = wait_half(it, h, g))) break;
          tc_fence_after();
          issue_sdp(h, g);
        }
        for (int h = 0; h < it.n_halves && ok; ++h) {
          const int t = h & 1, st = steps + (h >> 1), g = g0 + h, slot = g % kSlots;
          const uint32_t R = tmem + 128u * t;
          if (!(ok = mbar_wait(bar(kBarPReady + t), st & 1, abort_flag))) break;
          tc_fence_after();
          // dQ_t'^T = K^T dS_t^T: M = d, N = 64 queries, K = 128 keys.
          const uint32_t dso = static_cast<uint32_t>(t * kDSBytes) >> 4;
#pragma unroll
          for (int kk = 0; kk < BM / 16; ++kk) {
            const uint32_t off = static_cast<uint32_t>(kk * 2048) >> 4;
            mma_ss_lo(R + 64, k_mn + off, ds_mn + dso + off, idesc_q, kk > 0 ? 1u : 0u);
          }
          mma_commit(bar(kBarDQFull + t));
          // The previous item's dV, dK must have left TMEM before the first
          // product of this one overwrites them.
          if (h == 0 && k > 0) {
            if (!(ok = mbar_wait(bar(kBarEpiDone), (k - 1) & 1, abort_flag))) break;
            tc_fence_after();
          }
          // dV += P_t^T dO_t, dK += dS_t^T Q_t (A operands from TMEM); K = 64
          // queries.
          const uint32_t so = static_cast<uint32_t>(slot * kHalf) >> 4;
#pragma unroll
          for (int kk = 0; kk < BH_ / 16; ++kk) {
            const uint32_t ob = so + (static_cast<uint32_t>(kk * 2048) >> 4);
            const uint32_t acc = (h > 0 || kk > 0) ? 1u : 0u;
            mma_ts_lo(tmem + 256, R + kk * 8, do_mn + ob, idesc_g, acc);
            mma_ts_lo(tmem + 256 + D, R + 32 + kk * 8, q_mn + ob, idesc_g, acc);
          }
          mma_commit(bar(kBarQEmpty + slot));
          mma_commit(bar(kBarDOEmpty + slot));
          const int h2 = h + 2;
          if (h2 < it.n_halves) {
            const int g2 = g0 + h2;
            if (!(ok = mbar_wait(bar(kBarTmemFree + t), st & 1, abort_flag))) break;
            if (!(ok = wait_half(it, h2, g2))) break;
            tc_fence_after();
            issue_sdp(h2, g2);
          }
        }
        if (ok) mma_commit(bar(kBarKVDone));
        g0 += it.n_halves;
        steps += it.n_steps;
      }
      mma_commit(bar(kBarDrain));
      drain_wait(bar(kBarDrain), 0);
    } else if (PACKED && warp == 2) {
      // ------------------------------------------- rows past the sequence's end
      // Follows every copy and takes part in freeing the ring slots, so that no
      // barrier can run a phase past its wait.
      const int lane = threadIdx.x & 31;
      // Rows from `keep` on of a tile of `rows` 128-byte rows (box by box).
      auto clear = [&](int off, int rows, int keep) {
        for (int i = lane; i < (rows - keep) * 8; i += 32)
#pragma unroll
          for (int b = 0; b < kRowBoxes; ++b)
            *reinterpret_cast<uint4 *>(smem + off + b * rows * 128 + (keep + (i >> 3)) * 128 +
                                       (i & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
      };
      bool ok = true;
      int g = 0;
      for (int k = 0; ok; ++k) {
        int w;
        BwdItem it;
        if (!(ok = fetch_item(k, w, it, true)) || w >= n_items) break;
        int first_h = 0;
        auto half = [&](int h) -> bool {
          const int slot = g % kSlots;
          const uint32_t ph = (g / kSlots) & 1;
          if (!wait_warp(bar(kBarQFull + slot), ph, abort_flag)) return false;
          if (!wait_warp(bar(kBarDOFull + slot), ph, abort_flag)) return false;
          // (rows of the sequence)
          if (GROUPS && h - first_h == 2 * it.per) first_h = h;
          const int keep = it.N - it.i_first * BQ - (h - first_h) * BH_;
          if (keep < BH_) {
            clear(kOffQ + slot * kHalf, BH_, max(keep, 0));
            clear(kOffDO + slot * kHalf, BH_, max(keep, 0));
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kBarFix + slot));
          }
          if (lane == 0) {
            mbar_arrive(bar(kBarQEmpty + slot));
            mbar_arrive(bar(kBarDOEmpty + slot));
          }
          ++g;
          return true;
        };
        // In the order of the copies: two halves, K and V, the other halves.
        for (int h = 0; h < 2 && ok; ++h) ok = half(h);
        if (!ok || !(ok = wait_warp(bar(kBarKV), k & 1, abort_flag))) break;
        if (it.k0 + BM > it.N) {
          clear(kOffK, BM, it.N - it.k0);
          clear(kOffV, BM, it.N - it.k0);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBarKVFix));
        }
        if (lane == 0) mbar_arrive(bar(kBarKVDone));   // (with the item's last MMA)
        for (int h = 2; h < it.n_halves && ok; ++h) ok = half(h);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsGroup));
    // ------------------------- groups: P, dS, dQ' read-out and reduce, epilogue
    const int t = (warp - 4) >> 2;            // sub-tile of this group
    const int quarter = warp & 3;             // TMEM lanes 32*quarter .. +31
    const int lane = threadIdx.x & 31;
    const int r = quarter * 32 + lane;        // key row of S^T, dP^T; d row of dQ'^T
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t R = tmem + lane_off + 128u * t;
    const uint64_t c2 = f2(scale * kLog2e, scale * kLog2e);
    uint8_t *ds_buf = smem + kOffDS + t * kDSBytes;
    // This warp's quarter of the dS^T buffer: staging of its dQ' boxes and
    // of its dV / dK rows.
    uint8_t *stg = ds_buf + quarter * 4096;
    const uint32_t stg_u32 = s_base + kOffDS + t * kDSBytes + quarter * 4096;
    bool ok = true;
    int g0 = 0, steps = 0;
    for (int k = 0; ok; ++k) {
      int w;
      BwdItem it;
      if (!(ok = fetch_item(k, w, it, true)) || w >= n_items) break;
      const int key = it.k0 + r;
      int first_i = 0;          // kWindowGroups: the step that head it.bh begins with
      for (int i = 0; i < it.n_steps && ok; ++i) {
        const int h = 2 * i + t, st = steps + i, g = g0 + h, slot = g % kSlots;
        if (GROUPS && i - first_i == it.per) first_i = i, ++it.bh;
        const int q0 = (it.i_first + i - first_i) * BQ + t * BH_;   // first query of the sub-tile
        if (!(ok = wait_warp(bar(kBarSFull + t), st & 1, abort_flag))) break;
        // [LSE2 | D] of the sub-tile came with Q_t on QFull, which S_t needed.
        if (!(ok = wait_warp(bar(kBarQFull + slot), (g / kSlots) & 1, abort_flag))) break;
        tc_fence_after();
        const float *vec = reinterpret_cast<const float *>(smem + kOffVec + slot * kVecBytes);
        // Masking is needed only where a key of this warp is past N or, on the
        // diagonal block, later than a query (warp-uniform).
        const bool diag = causal && (q0 < it.k0 + BM) && (q0 + BH_ > it.k0);
        bool masked = diag || (it.k0 + quarter * 32 + 31 >= it.N);
        uint64_t see = 0;
        if constexpr (WINDOW) {
          // ... or, unless it is one of the first, too far before one.
          const int key_w = it.k0 + quarter * 32;
          masked |= q0 + BH_ - 1 - key_w >= pk.window && key_w + 31 >= pk.sinks;
          if (masked) see = bwd_tile::near_queries(key, q0, it.N, pk.window, pk.sinks);
        }
        if (masked)
          bwd_tile::chunks<WINDOW ? 2 : 1>(R, vec, ds_buf, r, key, q0, it.N, diag, see, c2);
        else
          bwd_tile::chunks<0>(R, vec, ds_buf, r, key, q0, it.N, diag, see, c2);
        tmem_wait_st();
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarPReady + t));

        // dQ_t'^T row d = r: 64 query columns, read out, then R_t is released.
        if (!(ok = wait_warp(bar(kBarDQFull + t), st & 1, abort_flag))) break;
        tc_fence_after();
        uint32_t g0v[32], g1v[32];
        tmem_ld32(R + 64, g0v);
        tmem_ld32(R + 96, g1v);
        tmem_wait_ld(g0v);
        tmem_wait_ld(g1v);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarTmemFree + t));
        // Add into the row-major accumulator with TMA reduces: this warp's
        // quarter of the dS^T buffer (its own key rows, free now that dQ'^T,
        // which read it, is complete) stages one 32-query x 32-d box at a time
        // as [query][d] fp32 rows with the 128-byte swizzle.
#pragma unroll
        for (int bx = 0; bx < 2; ++bx) {
          if (bx == 1) {
            if (lane == 0) bulk_wait_read_all();
            __syncwarp();
          }
#pragma unroll
          for (int qq = 0; qq < 32; ++qq)
            *reinterpret_cast<uint32_t *>(stg + qq * 128 + ((((lane >> 2) ^ (qq & 7))) << 4) +
                                          (lane & 3) * 4) = bx ? g1v[qq] : g0v[qq];
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_reduce_add_3d(&tm_dq, stg_u32, 32 * quarter, it.blk0 * BQ + q0 + 32 * bx, it.bh);
            bulk_commit();
          }
        }
        // The next element phase writes dS^T rows over the staging area.
        if (lane == 0) bulk_wait_read_all();
        __syncwarp();
      }
      if (!ok) break;

      // Epilogue: group 0 writes dV_j, group 1 dK_j = scale * (dS^T Q), as
      // bf16 rows (rows >= N are not stored).  Both 64-column halves are
      // read out of TMEM first, so the MMA warp may start the next item's
      // products into them while the rows are stored.
      if (!(ok = wait_warp(bar(kBarKVDone), k & 1, abort_flag))) break;
      tc_fence_after();
      // Rows are D values apart; PACKED: [row][key/value head].
      const int64_t row_step = PACKED ? static_cast<int64_t>(pk.kv_heads) * D : D;
      __nv_bfloat16 *base =
          (t ? dk : dv) + (PACKED ? it.row0 * row_step + it.kvh * D : static_cast<int64_t>(it.bh) * N * D);
      const float mul = t ? scale : 1.f;
      const uint32_t col = t ? 256u + D : 256u;
      uint32_t v[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(tmem + lane_off + col + 32 * c, v[c]);
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_wait_ld(v[c]);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarEpiDone));
      bool shared = PACKED && pk.group > 1;
      if constexpr (GROUPS) shared = it.n_steps == it.per;
      if constexpr (WINDOW) shared = shared || it.k0 < pk.split;
      if (shared) {
        // Another query head of the group (kWindow: or another item of the block of
        // first keys) adds to the same rows: fp32 boxes of
        // 32 rows x 32 columns into the accumulator (dK there still unscaled).
        // Rows past the sequence fall on its padding.
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (c > 0) {
            if (lane == 0) bulk_wait_read_all();
            __syncwarp();
          }
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint4 *>(stg + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                make_uint4(v[c][4 * j], v[c][4 * j + 1], v[c][4 * j + 2], v[c][4 * j + 3]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_reduce_add_3d(t ? &tm_dk : &tm_dv, stg_u32, 32 * c,
                              it.blk0 * BQ + it.k0 + quarter * 32, it.kvh);
            bulk_commit();
          }
        }
        if (lane == 0) bulk_wait_read_all();
        __syncwarp();
        g0 += it.n_halves;
        steps += it.n_steps;
        continue;
      }
      // The rows leave through this warp's staging quarter, 64 columns at a
      // time: the warp packs its 32 rows into 4 KB (16-byte chunks swizzled by
      // the row) and reads them back so that eight lanes store one row's 128
      // contiguous bytes.
      const int key_w = key - lane;   // this warp's first key row
#pragma unroll
      for (int hh = 0; hh < D / 64; ++hh) {
#pragma unroll
        for (int kq = 0; kq < 8; ++kq) {
          const uint32_t *c8 = &v[2 * hh + (kq >> 2)][(kq & 3) * 8];
          uint4 x;
          x.x = pack_bf16x2(__uint_as_float(c8[0]) * mul, __uint_as_float(c8[1]) * mul);
          x.y = pack_bf16x2(__uint_as_float(c8[2]) * mul, __uint_as_float(c8[3]) * mul);
          x.z = pack_bf16x2(__uint_as_float(c8[4]) * mul, __uint_as_float(c8[5]) * mul);
          x.w = pack_bf16x2(__uint_as_float(c8[6]) * mul, __uint_as_float(c8[7]) * mul);
          *reinterpret_cast<uint4 *>(stg + lane * 128 + ((kq ^ (lane & 7)) * 16)) = x;
        }
        __syncwarp();
#pragma unroll
        for (int kq = 0; kq < 8; ++kq) {
          const int rr = (lane >> 3) + 4 * kq, ch = lane & 7;
          const uint4 x = *reinterpret_cast<const uint4 *>(stg + rr * 128 + ((ch ^ (rr & 7)) * 16));
          if (key_w + rr < it.N)
            *reinterpret_cast<uint4 *>(base + (key_w + rr) * row_step + 64 * hh +
                                       ch * 8) = x;
        }
        __syncwarp();
      }
      g0 += it.n_halves;
      steps += it.n_steps;
    }
  }

  if (warp >= 4 && (threadIdx.x & 31) == 0) bulk_wait_all();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (threadIdx.x == 0) {
    if (misc->abort) atomicExch(dev_status, kDevTimeout);
    // The last CTA to finish puts the launch's work counters back to zero.
    __threadfence();
    if (atomicAdd(sched + 1, 1) == static_cast<int>(gridDim.x) - 1) {
      sched[0] = 0;
      sched[1] = 0;
      __threadfence();
    }
  }
}

template <int KIND>
cudaError_t launch_main(const CUtensorMap &tq64, const CUtensorMap &tk, const CUtensorMap &tv,
                        const CUtensorMap &tdo64, const CUtensorMap &tdq, const float *vecs,
                        void *dk, void *dv, int BH, int N, float scale, int causal, int *sched,
                        int fault_cta, int *dev_status, cudaStream_t stream,
                        const CUtensorMap &tdk, const CUtensorMap &tdv, const Extra<KIND> &pk) {
  cudaError_t e = cudaFuncSetAttribute(bwd_pipe_kernel<KIND>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  int dev = 0, n_sm = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
    return e;
  long long n_items = KIND == kDense ? (N + BQ - 1) / BQ : pk.n_blocks;
  if constexpr (KIND >= kWindow) n_items = pk.entries;
  n_items *= BH;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(n_items < n_sm ? n_items : n_sm));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, bwd_pipe_kernel<KIND>, tq64, tk, tv, tdo64, tdq, vecs,
                            reinterpret_cast<__nv_bfloat16 *>(dk),
                            reinterpret_cast<__nv_bfloat16 *>(dv), N, BH, scale, causal, sched,
                            fault_cta, dev_status, tdk, tdv, pk);
}

}  // namespace

cudaError_t launch_bwd_main_d128(const CUtensorMap &tq64, const CUtensorMap &tk,
                                 const CUtensorMap &tv, const CUtensorMap &tdo64,
                                 const CUtensorMap &tdq, const float *vecs, void *dk, void *dv,
                                 int BH, int N, float scale, int causal, int *sched,
                                 int fault_cta, int *dev_status, cudaStream_t stream) {
  return launch_main<kDense>(tq64, tk, tv, tdo64, tdq, vecs, dk, dv, BH, N, scale, causal, sched,
                            fault_cta, dev_status, stream, tdq, tdq, BwdPacked{});
}

cudaError_t launch_bwd_packed_main_d128(const CUtensorMap &tq64, const CUtensorMap &tk,
                                        const CUtensorMap &tv, const CUtensorMap &tdo64,
                                        const CUtensorMap &tdq, const CUtensorMap &tdk,
                                        const CUtensorMap &tdv, const float *vecs, void *dk,
                                        void *dv, int H, const BwdPacked &pk, float scale,
                                        int causal, int *sched, int *dev_status, int fault_cta,
                                        cudaStream_t stream) {
  return launch_main<kPacked>(tq64, tk, tv, tdo64, tdq, vecs, dk, dv, H, 0, scale, causal, sched,
                           fault_cta, dev_status, stream, tdk, tdv, pk);
}

cudaError_t launch_bwd_window_main_d128(const CUtensorMap &tq64, const CUtensorMap &tk,
                                        const CUtensorMap &tv, const CUtensorMap &tdo64,
                                        const CUtensorMap &tdq, const CUtensorMap &tdk,
                                        const CUtensorMap &tdv, const float *vecs, void *dk,
                                        void *dv, int H, const BwdWindow &pk, float scale,
                                        int *sched, int *dev_status, int fault_cta,
                                        cudaStream_t stream) {
  auto launch = pk.grouping ? launch_main<kWindowGroups> : launch_main<kWindow>;
  return launch(tq64, tk, tv, tdo64, tdq, vecs, dk, dv, H, 0, scale, 1, sched, fault_cta,
                dev_status, stream, tdk, tdv, pk);
}

}  // namespace fattn
