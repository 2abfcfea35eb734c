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
// Rounding: P and dS to bf16 before their products, as the dense kernels; sums and
// accumulators fp32; each gradient once.
#include <cuda_runtime.h>

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
constexpr float kLog2e = 1.4426950408889634f;

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
};

__device__ __forceinline__ int first_block(const SideArgs &a, int s) {
  return clampi(a.cu_seqlens[s], 0, a.T) / BQ + s;
}

// One block of 256 threads per (padded block, head); heads H .. H + Hk - 1
// stand for the key/value heads' accumulators.
template <int D>
__global__ void __launch_bounds__(256) packed_prep_kernel(const SideArgs a) {
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
  if (h == 0 && a.S > kSortedSeqs) {
    if (threadIdx.x == 0)
      a.table[blk] = live ? make_int4(begin, n, blk - local, local) : make_int4(0, 0, 0, 0);
  } else if (h == 0) {
    // The block's place in the table: behind the blocks of longer sequences (of
    // equal ones, those before it); an unused block, behind all used ones.
    int before = 0;
    for (int j = threadIdx.x; j < a.S; j += 256) {
      const int b = clampi(a.cu_seqlens[j], 0, a.T);
      const int len = clampi(a.cu_seqlens[j + 1], b, a.T) - b;
      const int blocks = (len + BQ - 1) / BQ;
      if (live)
        before += (len > n || (len == n && j < s)) ? blocks : 0;
      else   // all used blocks, less those numbered before this one
        before += blocks - clampi(blk - b / BQ - j, 0, blocks);
    }
    __shared__ int sum[8];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) before += __shfl_xor_sync(~0u, before, off);
    if ((threadIdx.x & 31) == 0) sum[threadIdx.x >> 5] = before;
    __syncthreads();
    if (threadIdx.x == 0) {
      before = 0;
      for (int u = 0; u < 8; ++u) before += sum[u];
      // (Offsets that decrease may lead anywhere: stay inside the table.)
      const int at = clampi(live ? before + local : before + blk, 0, a.n_blocks - 1);
      a.table[at] = live ? make_int4(begin, n, blk - local, local) : make_int4(0, 0, 0, 0);
    }
  }
  if (!live) return;
  const int row_in = threadIdx.x / L, part = threadIdx.x % L;
  const int64_t rows = static_cast<int64_t>(a.n_blocks) * BQ;
  const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kRounds = BQ / kRows;
  if (h >= a.H) {
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
template <int D>
__global__ void __launch_bounds__(256) packed_out_kernel(const SideArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int L = D / 8;
  const int tok = blockIdx.x;
  // The last sequence that begins at or before the token owns it, if any does.
  const int s = warp_search(a.S, tok, [&](int i) { return clampi(a.cu_seqlens[i], 0, a.T); });
  if (s < 0 || tok >= clampi(a.cu_seqlens[s + 1], 0, a.T)) return;
  const int begin = clampi(a.cu_seqlens[s], 0, a.T);
  const int64_t rows = static_cast<int64_t>(a.n_blocks) * BQ;
  const int64_t acc_row = static_cast<int64_t>(begin / BQ + s) * BQ + tok - begin;
  const int n = (a.H + (a.dk_acc != nullptr ? 2 * a.Hk : 0)) * L;
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

template <int D>
cudaError_t launch_d(const PackedGradMaps &m, const PackedGrad &p, const SideArgs &a, int *sched,
                     int *dev_status, int fault_cta, cudaStream_t stream) {
  const int heads = p.H + (a.dk_acc != nullptr ? p.Hk : 0);
  packed_prep_kernel<D><<<static_cast<unsigned>(a.n_blocks * heads), 256, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  BwdPacked pk;
  pk.table = a.table;
  pk.tokens = a.T;
  pk.sorted = a.S <= kSortedSeqs;
  pk.n_blocks = a.n_blocks;
  pk.group = p.H / p.Hk;
  pk.kv_heads = p.Hk;
  auto main_kernel = D == 128 ? launch_bwd_packed_main_d128 : launch_bwd_packed_main_d64;
  e = main_kernel(m.q, m.k, m.v, m.dout, m.dq_acc, m.dk_acc, m.dv_acc, a.vecs, p.dk, p.dv, p.H, pk,
                  p.scale, p.causal, sched, dev_status, fault_cta, stream);
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
  return cudaLaunchKernelEx(&cfg, packed_out_kernel<D>, a);
}

}  // namespace

PackedGradLayout packed_grad_layout(int T, int S, int H, int Hk, int d) {
  PackedGradLayout l;
  l.n_blocks = T / BQ + S;
  const size_t rows = static_cast<size_t>(l.n_blocks) * BQ;
  const size_t shared = H != Hk ? rows * Hk * d : 0;
  l.dk_acc = rows * H * d;
  l.dv_acc = l.dk_acc + shared;
  l.vecs = l.dv_acc + shared;
  l.table = l.vecs + static_cast<size_t>(l.n_blocks) * H * 2 * BQ;
  l.bytes = sizeof(float) * (l.table + static_cast<size_t>(l.n_blocks) * 4);
  return l;
}

cudaError_t launch_bwd_packed(const PackedGradMaps &m, const PackedGrad &p, float *ws, int *sched,
                              int *dev_status, int fault_cta, cudaStream_t stream) {
  const PackedGradLayout l = packed_grad_layout(p.T, p.S, p.H, p.Hk, p.d);
  SideArgs a{};
  a.o = static_cast<const __nv_bfloat16 *>(p.o);
  a.dout = static_cast<const __nv_bfloat16 *>(p.dout);
  a.lse = p.lse;
  a.cu_seqlens = p.cu_seqlens;
  a.dq_acc = ws;
  a.dk_acc = p.H != p.Hk ? ws + l.dk_acc : nullptr;
  a.dv_acc = p.H != p.Hk ? ws + l.dv_acc : nullptr;
  a.vecs = ws + l.vecs;
  a.table = reinterpret_cast<int4 *>(ws + l.table);
  a.dq = static_cast<__nv_bfloat16 *>(p.dq);
  a.dk = static_cast<__nv_bfloat16 *>(p.dk);
  a.dv = static_cast<__nv_bfloat16 *>(p.dv);
  a.S = p.S, a.T = p.T, a.H = p.H, a.Hk = p.Hk, a.n_blocks = l.n_blocks;
  a.scale = p.scale;
  return p.d == 128 ? launch_d<128>(m, p, a, sched, dev_status, fault_cta, stream)
                    : launch_d<64>(m, p, a, sched, dev_status, fault_cta, stream);
}

}  // namespace fattn
