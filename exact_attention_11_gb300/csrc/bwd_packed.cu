// bwd_packed.cu -- gradients of the packed forward (fwd_packed.cu, bf16): what
// runs before and after the main kernels of bwd_bf16_d128.cu / bwd_bf16_d64.cu
// (their PACKED form).  The mathematics is that of bwd_bf16.cu, sequence by
// sequence; with grouped heads, dK and dV of a key/value head are the sums over
// the query heads that use it.
//
//   packed_prep_kernel   per padded 128-row block (sequence s starts at block
//                        cu_seqlens[s] / 128 + s: no prefix sum over lengths, at
//                        most one unused block per sequence): its entry in the
//                        block table, [-LSE2 x 128 | -D x 128] of every query
//                        head, and zeros in the fp32 accumulators.  The table goes
//                        by length, longest sequence first, so that the main
//                        kernel's items come heaviest first
//   main kernel          one item per (key block, query head)
//   packed_out_kernel    dQ = scale * accumulator (and dK, dV where heads share
//                        them), rounded to bf16 into the packed rows
// Both side kernels are bound by HBM: they read o and dO once, write and read
// the fp32 accumulators once and write the gradients once.
//
// Measured (16 query / 4 key/value heads): 4 documents of 5498 tokens in all, d = 128,
// causal: 21 + 161 + 15 us, 197 for the call (the main kernel 1112 TFLOP/s, the side
// kernels 5.4 and 6.7 TB/s); 16 documents of 2168 tokens, d = 64: 8 + 31 + 6, 45 us, of
// which the main kernel's start and tail are half.  An item per query head and not per
// group: with two to sixteen steps of a group an item, 50 - 59 us and 213 - 215.
// With a window (fa_backward_packed_window) a key block's item visits the query blocks
// that see it only, which the table gives with it; what bounds it and how it rounds stay:
// 4 documents of 10560 tokens in all, window 1024, 4 first tokens: 258 us for the call (720
// TFLOP/s of visible pairs; the main kernel takes 2.2 us a step of 128 x 128 pairs, of which
// the window leaves 0.89); 16 of 2168 tokens, d = 64, window 256: 8 + 28 + 6, 37 us.
// With a window items are alike and, in long calls, many: there most have all query heads of a
// key/value head, load K and V once and store dK and dV, whose sums over heads stay in TMEM
// (281 -> 258 us for the 4 documents; 3 of up to 4300, 32 / 8 heads, window 208: 203 -> 162).
// Rounding: P and dS to bf16 before their products, as the dense kernels; sums and
// accumulators fp32; each gradient once.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "kernels.h"
#include "packed.cuh"
#include "ptx.cuh"

namespace fattn {
namespace {

constexpr int BQ = 128;
// Up to this many sequences the table is sorted (each block compares its sequence
// with all others); beyond, it goes by block number, unused blocks in between.
constexpr int kSortedSeqs = 2048;
constexpr int kSms = 152;     // of an sm_103a GPU
constexpr int kStart = 3;     // an item's start and end, in steps (2 and 4: no change)
constexpr float kLog2e = 1.4426950408889634f;
// All keys up to a query's own (or all); a window; a window, and items that may have all heads
// of a group.
enum : int { kAll = 0, kWindow = 1, kGroups = 2 };

struct SideArgs {
  const __nv_bfloat16 *o, *dout;
  const float *lse;             // [H][T]
  const int *cu_seqlens;
  float *dq_acc;                // [H][rows][D], rows = n_blocks * 128
  float *dk_acc, *dv_acc;       // [Hk][rows][D], null when no heads are shared
  float *vecs;                  // [H][n_blocks][2][128]
  int4 *table;
  __nv_bfloat16 *dq, *dk, *dv;
  int S, T, H, Hk, n_blocks;
  float scale;
  // A window: the main kernel's query blocks per entry of the table, and their count.
  int2 *range;
  int4 *count;
  int *stored;
  int entries, split, whole, window, sinks;
};

// A window: key block jb is seen by the query blocks from its own to `reach` further;
// if it holds first tokens, by all later ones too.  In sequences of more than `whole`
// blocks, an SM's share of the call's steps (beside items with all heads of a group, half of
// it), those are items of their own (entries of
// kFar query blocks or more): one item of the whole sequence would end the call alone
// (one document of 16384, 8 heads, window 512: 185 us, 354 in one item; but four of 8192,
// whose items fit in: 631, 622 so).  Far parts of four blocks: 190, 633 us, but 0.98 - 0.99 of
// the time over three times 40 mixes of short and long documents; of sixteen 1.01 - 1.02.
constexpr int kFar = 8;
__host__ __device__ __forceinline__ int reach(int window) {
  return (BQ - 2 + window) / BQ;
}
__host__ __device__ __forceinline__ int far_steps(int window) {
  const int r = reach(window) + 1;
  return r > kFar ? r : kFar;
}
// Entries for the far query blocks of key block jb, of a sequence of `blocks`.
__device__ __forceinline__ int far_entries(const SideArgs &a, int jb, int blocks) {
  const int step = far_steps(a.window);
  if (jb * BQ >= a.split || blocks <= a.whole) return 0;
  return (max(blocks - 1 - jb - reach(a.window), 0) + step - 1) / step;
}
__device__ __forceinline__ int far_entries(const SideArgs &a, int blocks) {
  int n = 0;
  if (blocks > a.whole)
    for (int jb = 0; jb < blocks && jb * BQ < a.split; ++jb) n += far_entries(a, jb, blocks);
  return n;
}

__device__ __forceinline__ int first_block(const SideArgs &a, int s) {
  return clampi(a.cu_seqlens[s], 0, a.T) / BQ + s;
}

// One block of 256 threads per (padded block, head); heads H .. H + Hk - 1
// stand for the key/value heads' accumulators.
template <int D, int KIND>
__global__ void __launch_bounds__(256) packed_prep_kernel(const SideArgs a) {
  constexpr bool WINDOW = KIND != kAll, GROUPS = KIND == kGroups;
  // The main kernel may be scheduled once every block of this one has begun.
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int L = D / 8;                 // threads per row, eight values each
  constexpr int kRows = 256 / L;
  const int heads = a.H + (a.dk_acc != nullptr ? a.Hk : 0);
  const int blk = blockIdx.x / heads, h = blockIdx.x - blk * heads;
  const int s = warp_search(a.S, blk, [&](int i) { return first_block(a, i); });
  int begin = 0, n = 0, local = 0;
  if (s >= 0) {
    begin = clampi(a.cu_seqlens[s], 0, a.T);
    n = clampi(a.cu_seqlens[s + 1], begin, a.T) - begin;
    local = blk - begin / BQ - s;
  }
  const bool live = s >= 0 && local * BQ < n;
  // A window: the entry's query blocks, up to the last that sees the key block (all
  // of them, where it holds first tokens and nothing is split off).
  auto put_range = [&](int at, int last) {
    if (WINDOW) a.range[at] = make_int2(local, max(last - local + 1, 1));
  };
  const int blocks = (n + BQ - 1) / BQ;
  const int last = WINDOW ? min(local + reach(a.window), blocks - 1) : 0;
  __shared__ int sum[GROUPS ? 48 : WINDOW ? 32 : 8];
  __shared__ float sum_lost[GROUPS ? 8 : 1];
  __shared__ int most[GROUPS ? 8 : 1];
  if (h == 0 && a.S > kSortedSeqs) {
    if (threadIdx.x == 0) {
      a.table[blk] = live ? make_int4(begin, n, blk - local, local) : make_int4(0, 0, 0, 0);
      put_range(blk, local * BQ < a.sinks ? blocks - 1 : last);
      if (WINDOW && blk == 0) *a.count = make_int4(a.n_blocks, 0, 0, 0);
    }
  } else if (h == 0 || (GROUPS && h >= a.H)) {
    // The block's place in the table: behind the blocks of longer sequences (of
    // equal ones, those before it); an unused block, behind all used ones.
    int before = 0;
    // A window: entries of all sequences, far ones, and those of first tokens, which come
    // first.
    int used = 0, far_before = 0, far = 0, split_before = 0, split = 0;
    const int n_split = (a.split + BQ - 1) / BQ;
    float lost = 0.f;                        // steps that the last blocks have less than the others
    int longest = 0;                         // blocks of a sequence
    for (int j = threadIdx.x; j < a.S; j += 256) {
      const int b = clampi(a.cu_seqlens[j], 0, a.T);
      const int len = clampi(a.cu_seqlens[j + 1], b, a.T) - b;
      const int blocks = (len + BQ - 1) / BQ;
      const bool longer = len > n || (len == n && j < s);
      if (live)
        before += longer ? blocks : 0;
      else   // all used blocks, less those numbered before this one
        before += blocks - clampi(blk - b / BQ - j, 0, blocks);
      if (WINDOW) {
        const int f = far_entries(a, blocks);
        used += blocks, far += f, far_before += longer ? f : 0;
        if (GROUPS) {
          const int c = min(blocks, n_split);
          split += c, split_before += longer ? c : 0;
          const float r = static_cast<float>(reach(a.window)), b = static_cast<float>(blocks);
          lost += b > r ? r * (r + 1.f) * 0.5f : b * (r + 1.f) - b * (b + 1.f) * 0.5f;
          longest = max(longest, blocks);
        }
      }
    }
    auto add_up = [&](auto x, auto *sum) {
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(~0u, x, off);
      if ((threadIdx.x & 31) == 0) sum[threadIdx.x >> 5] = x;
    };
    add_up(before, sum);
    if constexpr (WINDOW) {
      add_up(used, sum + 8);
      add_up(far_before, sum + 16);
      add_up(far, sum + 24);
      if (GROUPS) {
        add_up(split_before, sum + 32);
        add_up(split, sum + 40);
        add_up(lost, sum_lost);
        longest = __reduce_max_sync(~0u, longest);
        if ((threadIdx.x & 31) == 0) most[threadIdx.x >> 5] = longest;
      }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      auto total = [&](const auto *x) {
        auto n = x[0];
        for (int u = 1; u < 8; ++u) n += x[u];
        return n;
      };
      before = total(sum);
      int place = live ? before + local : before + blk;
      if constexpr (GROUPS) {
        split = total(sum + 40);
        split_before = total(sum + 32);
        if (live)
          place = local < n_split ? split_before + local
                                  : place + split - split_before - min(blocks, n_split);
      }
      // (Offsets that decrease may lead anywhere: stay inside the table.)
      const int at = clampi(place, 0, a.n_blocks - 1);
      if (h == 0 && (!WINDOW || live))
        a.table[at] = live ? make_int4(begin, n, blk - local, local) : make_int4(0, 0, 0, 0);
      if constexpr (WINDOW) {
        // The used entries come first, then the far ones.
        used = total(sum + 8);
        const int far_all = total(sum + 24), all = clampi(used + far_all, 0, a.entries);
        const int from = clampi(split, 0, all), rest = clampi(used, from, all) - from;
        int grouped = 0;
        if (GROUPS) {
          // Items with all heads of a group load K and V once and need no sums of dK and dV
          // in memory, but are few and long: if an SM's share of the call is one and a half
          // of them or more (in steps; kStart: an item's start), they go first, and what
          // comes last in items of one head takes the SMs most of one of them.  (One or two
          // of them for the share: no change over 40 mixes; at the end a half 0.99 of the time
          // for the 4 documents, a whole one 1.03.)
          for (int u = 1; u < 8; ++u) most[0] = max(most[0], most[u]);
          const float steps = static_cast<float>(reach(a.window)) + 1.f;
          const float share =
              (static_cast<float>(all) * (steps + kStart) - total(sum_lost)) * a.H / kSms;
          const float item = fminf(steps, static_cast<float>(most[0])) * (a.H / a.Hk) + kStart;
          const float last = 0.75f * kSms * item / ((item - kStart) + kStart * (a.H / a.Hk));
          if (1.5f * item <= share)
            grouped = clampi(rest + min(far_all, static_cast<int>(last) / a.Hk) -
                                 static_cast<int>(last) / a.Hk, 0, rest);
        }
        // Its items have all heads of a group, which then store dK and dV.
        if (GROUPS) {
          sum[0] = live && at >= from && at < from + grouped && local >= n_split;
          if (h == 0) a.stored[blk] = sum[0];
        }
        if (h == 0 && blk == 0) *a.count = make_int4(all, from, grouped, 0);
        if (h == 0 && live) {
          const bool to_end = local * BQ < a.sinks && (a.split == 0 || blocks <= a.whole);
          put_range(at, to_end ? blocks - 1 : last);
          // (Only blocks of first tokens have far entries, at most eight: the loop is that
          // short.  Over all blocks before, one document of 2^20 tokens took 387 us here, 77 so.)
          const int step = far_steps(a.window), n_far = far_entries(a, local, blocks);
          int to = used + total(sum + 16);
          if (n_far > 0)
            for (int jb = 0; jb < local; ++jb) to += far_entries(a, jb, blocks);
          for (int f = 0; f < n_far; ++f) {
            const int first = last + 1 + f * step, x = clampi(to + f, 0, a.entries - 1);
            a.table[x] = make_int4(begin, n, blk - local, local);
            a.range[x] = make_int2(first, min(step, blocks - first));
          }
        }
      }
    }
  }
  if (!live) return;
  if (GROUPS && h >= a.H) {
    __syncthreads();
    if (sum[0]) return;
  }
  const int row_in = threadIdx.x / L, part = threadIdx.x % L;
  const int64_t rows = static_cast<int64_t>(a.n_blocks) * BQ;
  const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kRounds = BQ / kRows;
  if (h >= a.H) {
    if (WINDOW && a.H == a.Hk && local * BQ >= a.split) return;   // stored, not added up
#pragma unroll
    for (int u = 0; u < kRounds; ++u) {
      const int64_t at =
          ((h - a.H) * rows + static_cast<int64_t>(blk) * BQ + u * kRows + row_in) * D + part * 8;
      reinterpret_cast<float4 *>(a.dk_acc + at)[0] = z;
      reinterpret_cast<float4 *>(a.dk_acc + at)[1] = z;
      reinterpret_cast<float4 *>(a.dv_acc + at)[0] = z;
      reinterpret_cast<float4 *>(a.dv_acc + at)[1] = z;
    }
    return;
  }
  // Every round's loads go out before the first is used.
  uint4 x[kRounds], y[kRounds];
  float lse[kRounds];
#pragma unroll
  for (int u = 0; u < kRounds; ++u) {
    const int i = local * BQ + u * kRows + row_in;
    if (i >= n) continue;
    const int64_t at = (static_cast<int64_t>(begin + i) * a.H + h) * D + part * 8;
    x[u] = *reinterpret_cast<const uint4 *>(a.o + at);
    y[u] = *reinterpret_cast<const uint4 *>(a.dout + at);
    lse[u] = a.lse[static_cast<int64_t>(h) * a.T + begin + i];
  }
  float *vec = a.vecs + (static_cast<int64_t>(h) * a.n_blocks + blk) * (2 * BQ);
#pragma unroll
  for (int u = 0; u < kRounds; ++u) {
    const int r = u * kRows + row_in;
    const bool real = local * BQ + r < n;
    float acc = 0.f;
    if (real) {
      const uint32_t xw[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      const uint32_t yw[4] = {y[u].x, y[u].y, y[u].z, y[u].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc = fmaf(__uint_as_float(xw[e] << 16), __uint_as_float(yw[e] << 16), acc);
        acc = fmaf(__uint_as_float(xw[e] & 0xffff0000u), __uint_as_float(yw[e] & 0xffff0000u), acc);
      }
      float *q = a.dq_acc + (h * rows + static_cast<int64_t>(blk) * BQ + r) * D + part * 8;
      reinterpret_cast<float4 *>(q)[0] = z;
      reinterpret_cast<float4 *>(q)[1] = z;
    }
#pragma unroll
    for (int off = L / 2; off > 0; off >>= 1) acc += __shfl_xor_sync(~0u, acc, off);
    if (part == 0) {
      vec[r] = real ? -lse[u] * kLog2e : -INFINITY;
      vec[BQ + r] = real ? -acc : 0.f;
    }
  }
}

// One block per token: its rows of every head, eight values a thread.
template <int D, int KIND>
__global__ void __launch_bounds__(256) packed_out_kernel(const SideArgs a) {
  constexpr bool WINDOW = KIND != kAll, GROUPS = KIND == kGroups;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int L = D / 8;
  const int tok = blockIdx.x;
  // The last sequence that begins at or before the token owns it, if any does.
  const int s = warp_search(a.S, tok, [&](int i) { return clampi(a.cu_seqlens[i], 0, a.T); });
  if (s < 0 || tok >= clampi(a.cu_seqlens[s + 1], 0, a.T)) return;
  const int begin = clampi(a.cu_seqlens[s], 0, a.T);
  const int64_t rows = static_cast<int64_t>(a.n_blocks) * BQ;
  const int64_t acc_row = static_cast<int64_t>(begin / BQ + s) * BQ + tok - begin;
  bool shared = a.dk_acc != nullptr;
  if (WINDOW && a.H == a.Hk) shared = shared && (tok - begin) / BQ * BQ < a.split;
  if (GROUPS) shared = a.stored[begin / BQ + s + (tok - begin) / BQ] == 0;
  const int n = (a.H + (shared ? 2 * a.Hk : 0)) * L;
  for (int i = threadIdx.x; i < n; i += 256) {
    int h = i / L;
    const int c = i % L * 8;
    const float *acc = a.dq_acc;
    __nv_bfloat16 *out = a.dq;
    int heads = a.H;
    float mul = a.scale;
    if (h >= a.H) {
      h -= a.H;
      heads = a.Hk;
      const bool is_v = h >= a.Hk;
      if (is_v) h -= a.Hk;
      acc = is_v ? a.dv_acc : a.dk_acc;
      out = is_v ? a.dv : a.dk;
      mul = is_v ? 1.f : a.scale;
    }
    const float4 *p = reinterpret_cast<const float4 *>(acc + (h * rows + acc_row) * D + c);
    const float4 x = p[0], y = p[1];
    *reinterpret_cast<uint4 *>(out + (static_cast<int64_t>(tok) * heads + h) * D + c) =
        make_uint4(pack_bf16x2(x.x * mul, x.y * mul), pack_bf16x2(x.z * mul, x.w * mul),
                   pack_bf16x2(y.x * mul, y.y * mul), pack_bf16x2(y.z * mul, y.w * mul));
  }
}

template <int D, int KIND>
cudaError_t launch_d(const PackedGradMaps &m, const PackedGrad &p, const SideArgs &a, int *sched,
                     int *dev_status, int fault_cta, cudaStream_t stream) {
  const int heads = p.H + (a.dk_acc != nullptr ? p.Hk : 0);
  packed_prep_kernel<D, KIND><<<static_cast<unsigned>(a.n_blocks * heads), 256, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  BwdWindow pk;
  pk.table = a.table;
  pk.tokens = a.T;
  pk.sorted = a.S <= kSortedSeqs;
  pk.n_blocks = a.n_blocks;
  pk.group = p.H / p.Hk;
  pk.kv_heads = p.Hk;
  if (KIND != kAll) {
    pk.sorted = 0;   // (an entry of length 0 does not end it: the count does)
    pk.range = a.range, pk.count = reinterpret_cast<const int *>(a.count);
    pk.entries = a.entries, pk.split = a.split;
    pk.window = a.window, pk.sinks = a.sinks, pk.grouping = KIND == kGroups;
    auto main_kernel = D == 128 ? launch_bwd_window_main_d128 : launch_bwd_window_main_d64;
    e = main_kernel(m.q, m.k, m.v, m.dout, m.dq_acc, m.dk_acc, m.dv_acc, a.vecs, p.dk, p.dv, p.H,
                    pk, p.scale, sched, dev_status, fault_cta, stream);
  } else {
    auto main_kernel = D == 128 ? launch_bwd_packed_main_d128 : launch_bwd_packed_main_d64;
    e = main_kernel(m.q, m.k, m.v, m.dout, m.dq_acc, m.dk_acc, m.dv_acc, a.vecs, p.dk, p.dv, p.H,
                    pk, p.scale, p.causal, sched, dev_status, fault_cta, stream);
  }
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.T));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, packed_out_kernel<D, KIND>, a);
}

}  // namespace

PackedGradLayout packed_grad_layout(int T, int S, int H, int Hk, int d, int window, int sinks) {
  PackedGradLayout l{};
  l.n_blocks = T / BQ + S;
  l.entries = l.n_blocks;
  // Up to eight blocks of first tokens are split: with more there are items enough, and
  // their far parts would fill the table.  Only the longest sequences have far parts.
  if (window > 0 && window < T && S <= kSortedSeqs && sinks <= 8 * BQ) {
    l.split = sinks;
    const long long most = T / (BQ * (reach(window) + 1)) + 1;   // sequences with far parts
    l.entries += (sinks + BQ - 1) / BQ *
                 (T / (BQ * far_steps(window)) + 2 * std::min<long long>(S, most) + 1);
  }
  l.shared = H != Hk || l.split > 0;
  const size_t rows = static_cast<size_t>(l.n_blocks) * BQ;
  const size_t shared = l.shared ? rows * Hk * d : 0;
  l.dk_acc = rows * H * d;
  l.dv_acc = l.dk_acc + shared;
  l.vecs = l.dv_acc + shared;
  l.table = l.vecs + static_cast<size_t>(l.n_blocks) * H * 2 * BQ;
  l.range = l.table + static_cast<size_t>(l.entries) * 4;
  l.count = l.range + (window > 0 ? (static_cast<size_t>(l.entries) * 2 + 3) / 4 * 4 : 0);
  l.stored = l.count + (window > 0 ? 4 : 0);
  l.bytes = sizeof(float) * (l.stored + (window > 0 ? l.n_blocks : 0));
  return l;
}

cudaError_t launch_bwd_packed(const PackedGradMaps &m, const PackedGrad &p, float *ws, int *sched,
                              int *dev_status, int fault_cta, cudaStream_t stream) {
  const PackedGradLayout l = packed_grad_layout(p.T, p.S, p.H, p.Hk, p.d, p.window, p.sinks);
  SideArgs a{};
  a.o = static_cast<const __nv_bfloat16 *>(p.o);
  a.dout = static_cast<const __nv_bfloat16 *>(p.dout);
  a.lse = p.lse;
  a.cu_seqlens = p.cu_seqlens;
  a.dq_acc = ws;
  a.dk_acc = l.shared ? ws + l.dk_acc : nullptr;
  a.dv_acc = l.shared ? ws + l.dv_acc : nullptr;
  a.vecs = ws + l.vecs;
  a.table = reinterpret_cast<int4 *>(ws + l.table);
  a.dq = static_cast<__nv_bfloat16 *>(p.dq);
  a.dk = static_cast<__nv_bfloat16 *>(p.dk);
  a.dv = static_cast<__nv_bfloat16 *>(p.dv);
  a.S = p.S, a.T = p.T, a.H = p.H, a.Hk = p.Hk, a.n_blocks = l.n_blocks;
  a.scale = p.scale;
  if (p.window > 0) {
    a.range = reinterpret_cast<int2 *>(ws + l.range);
    a.count = reinterpret_cast<int4 *>(ws + l.count);
    a.stored = reinterpret_cast<int *>(ws + l.stored);
    a.entries = static_cast<int>(l.entries), a.split = l.split;
    a.window = p.window, a.sinks = p.sinks;
    const long long blocks = p.T / BQ, steps = reach(p.window) + 1;
    const long long share = blocks * steps * p.H / kSms;         // an SM's, in steps
    // An SM's share is twice an item with all heads of a group, if all tokens are one
    // sequence's (whose last blocks have less steps): packed_prep_kernel, which knows the
    // lengths, decides.  (From one and a half here: calls that it then left to items of one
    // head took 3 - 5% longer in the kernel for both.)
    const long long cut = std::min(steps, blocks), group = p.H / p.Hk;
    const long long most = (blocks * (steps + kStart) - cut * (cut - 1) / 2) * p.H / kSms;
    const bool groups = group > 1 && p.S <= kSortedSeqs && (p.sinks == 0 || l.split > 0) &&
                 2 * (group * std::min(steps, blocks + 1) + kStart) <= most;
    a.whole = static_cast<int>(std::min(groups ? std::max(steps, share / 2) : share, 1ll << 30));
    auto launch = p.d == 128 ? (groups ? launch_d<128, kGroups> : launch_d<128, kWindow>)
                             : (groups ? launch_d<64, kGroups> : launch_d<64, kWindow>);
    return launch(m, p, a, sched, dev_status, fault_cta, stream);
  }
  return p.d == 128 ? launch_d<128, kAll>(m, p, a, sched, dev_status, fault_cta, stream)
                    : launch_d<64, kAll>(m, p, a, sched, dev_status, fault_cta, stream);
}

}  // namespace fattn
