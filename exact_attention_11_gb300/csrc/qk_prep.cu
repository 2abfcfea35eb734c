// qk_prep.cu -- what a layer does to its queries and keys before attention,
// in one pass over them: the RMS norm of each head and the rotary position
// embedding, with the result written densely or, for serving, the keys and
// values written into the paged cache; and the backward pass.
//
// Per row x of d values (one token, one head), with weight w (optional):
//     r = 1 / sqrt(mean(x^2) + eps),   y = x r w   (y = x without a weight)
// and per rotated pair i < rot / 2 of y, at angle t = position * inv_freq[i]:
//     (a, b) -> mscale (a cos t - b sin t, b cos t + a sin t).
// Pairs are (i, i + rot/2) ("half" layout) or (2i, 2i + 1) (interleaved);
// values past rot pass through.  Backward, with g = R(-t) dy:
//     dw = sum over rows of g x r,   dx = r (w g - x r^2 mean(w g x)).
//
// Angles.  position * inv_freq of a far position has lost its fraction of a
// turn in fp32 (2^24 steps in all) and FP64 is slow on this GPU.  A turn is
// therefore a 64-bit fixed-point fraction: each block turns inv_freq / 2 pi
// into round(2^64 frac) once, and position * that, in wrapping 64-bit integer
// arithmetic, is the exact angle modulo a turn (error < |position| 2^-64
// turns beside inv_freq's own rounding).  Its top 32 bits go to sincospif.
//
// Bound by HBM bytes: every value is read once and written once, 16 bytes a
// load.  A thread owns two 8-value chunks of a row, chosen so that both
// members of every pair are its own (half layout: chunk l and chunk
// l + rot/16; interleaved: any two), so the rotation needs no exchange and
// the norm's sum one butterfly over d/16 lanes.  The rows of a warp are
// consecutive tokens of one head, so the 16-byte pieces of a key that the
// cache keeps 16 tokens wide fill whole sectors.  The cosines of a token
// serve all its heads: a block takes kTok tokens and computes them once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"

namespace fattn {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;   // rot / 2 at d = 256
constexpr int kMaxTok = 4;       // tokens per block
constexpr int kCacheBlock = kDecodeBlockSize;

// Eight consecutive values of type T <-> fp32.
template <typename T>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16> {
  uint4 w;
  __device__ void load(const void *p) { w = *reinterpret_cast<const uint4 *>(p); }
  __device__ void get(float (&f)[8]) const {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(v[i] << 16);
      f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
    }
  }
  __device__ static void store(void *p, const float (&f)[8]) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                               pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  }
};
template <>
struct Chunk<__half> {
  uint4 w;
  __device__ void load(const void *p) { w = *reinterpret_cast<const uint4 *>(p); }
  __device__ void get(float (&f)[8]) const {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&v[i]));
      f[2 * i] = x.x;
      f[2 * i + 1] = x.y;
    }
  }
  __device__ static void store(void *p, const float (&f)[8]) {
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      v[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(v[0], v[1], v[2], v[3]);
  }
};
template <>
struct Chunk<float> {
  float4 a, b;
  __device__ void load(const void *p) {
    a = reinterpret_cast<const float4 *>(p)[0];
    b = reinterpret_cast<const float4 *>(p)[1];
  }
  __device__ void get(float (&f)[8]) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
  __device__ static void store(void *p, const float (&f)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
};

// The two chunks that thread l of a row's D/16 owns.  Half layout: chunk l of
// the rotated part with its partner l + rot/16, then the chunks past rot two
// by two; interleaved: two by two.
template <int D>
__device__ __forceinline__ void chunks_of(int l, int rot, bool half, int &c0, int &c1) {
  const int n = rot >> 4;   // pairs of chunks in the rotated part
  if (half && l < n) {
    c0 = l;
    c1 = l + n;
  } else {
    c0 = 2 * l;
    c1 = 2 * l + 1;
  }
}

// Angle table of a token: in either layout thread l of a row rotates pairs
// 8 l .. 8 l + 7, if those are below rot / 2.  It reads them as four float4
// (cos, sin, cos, sin); the four are L apart, so that a row's lanes read
// consecutive 16-byte words.
template <int L>
struct Table {
  static constexpr int kStride = 4 * L + 4;   // float4 per token (the 4: bank spread)
  __device__ static int at(int pair) {        // in float2
    return (((pair & 7) >> 1) * L + (pair >> 3)) * 2 + (pair & 1);
  }
};

// Rotates thread l's two chunks by its angles; `dir` = 1 forward, -1 backward.
template <int L>
__device__ __forceinline__ void rotate(float (&a)[8], float (&b)[8], int l, int rot, bool half,
                                       const float4 *cs, float dir) {
  if (l * 16 >= rot) return;
#pragma unroll
  for (int j2 = 0; j2 < 4; ++j2) {
    const float4 t = cs[j2 * L + l];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const float c = u ? t.z : t.x, s = dir * (u ? t.w : t.y);
      const int j = 2 * j2 + u;
      float &pa = half ? a[j] : (j < 4 ? a[(2 * j) & 7] : b[(2 * j) & 7]);
      float &pb = half ? b[j] : (j < 4 ? a[(2 * j + 1) & 7] : b[(2 * j + 1) & 7]);
      const float x = pa, y = pb;
      pa = x * c - y * s;
      pb = y * c + x * s;
    }
  }
}

// inv_freq (radians per position) as a 64-bit fraction of a turn.
__device__ __forceinline__ uint64_t turn_fraction(double inv_freq) {
  const double t = inv_freq * 0.15915494309189533577;   // 1 / (2 pi)
  return static_cast<uint64_t>((t - floor(t)) * 18446744073709551616.0);
}

// (cos, sin) of tokens t0 .. t0 + n - 1, times mscale, into their tables.
template <int L>
__device__ __forceinline__ void fill_table(float4 *cs, const uint64_t *frac, const int *positions,
                                           int t0, int n, int pairs, float mscale) {
  for (int i = threadIdx.x; i < n * pairs; i += kThreads) {
    const int t = i / pairs, p = i - t * pairs;
    const uint64_t turns =
        static_cast<uint64_t>(static_cast<int64_t>(positions[t0 + t])) * frac[p];
    // Signed top half: the angle in [-1/2, 1/2) turns, in units of 2^-32.
    const float x = static_cast<float>(static_cast<int32_t>(turns >> 32)) * 0x1p-31f;
    float s, c;
    sincospif(x, &s, &c);
    reinterpret_cast<float2 *>(cs + t * Table<L>::kStride)[Table<L>::at(p)] =
        make_float2(c * mscale, s * mscale);
  }
}

template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int off = LANES / 2; off > 0; off >>= 1) v += __shfl_xor_sync(~0u, v, off);
  return v;
}

struct PrepArgs {
  const void *q, *k, *v, *qw, *kw;
  const int *positions;
  const double *inv_freq;
  const long long *slots;       // null: dense keys
  void *q_out, *k_out;          // k_out: dense keys, or the key cache
  void *v_cache;
  int T, H, Hk, rot, half;
  int64_t q_stride, k_stride, v_stride, n_slots;
  float eps, mscale;
  int tok_shift;                // log2 of the tokens per block (1, 2 or 4)
  int row_blocks;               // blocks that share a token tile's rows
  int qk_blocks;                // blocks of the q / k part; the rest transpose V
};

// A block's values of V: kCacheBlock tokens of one head, transposed through
// shared memory into the cache's [dimension][token] rows.  A run of tokens in
// consecutive slots leaves as the widest aligned stores (16, 8, 4 or 2
// bytes): whole cache blocks of a prompt as 16-byte stores, a decode step's
// lone tokens as 2-byte ones.
constexpr int kValueRow = kDecodeHeadSize * 2 + 4;   // bytes; the 4 spread rows over the banks
constexpr int kValueBytes = kCacheBlock * (kValueRow + 12) + 4;
__device__ void write_values(const PrepArgs &a, int unit, uint8_t *smem) {
  constexpr int D = kDecodeHeadSize;
  constexpr int kRow = kValueRow;
  long long *slot = reinterpret_cast<long long *>(smem + kCacheBlock * kRow);
  int *width = reinterpret_cast<int *>(slot + kCacheBlock);
  const int h = unit % a.Hk, t0 = unit / a.Hk * kCacheBlock;
  const int n = min(kCacheBlock, a.T - t0);
  const int t = threadIdx.x >> 4, c = threadIdx.x & 15;
  if (t < n) {
    const uint4 x = *reinterpret_cast<const uint4 *>(
        reinterpret_cast<const uint16_t *>(a.v) + static_cast<int64_t>(t0 + t) * a.v_stride +
        h * D + c * 8);
    uint32_t *row = reinterpret_cast<uint32_t *>(smem + t * kRow + c * 16);
    row[0] = x.x, row[1] = x.y, row[2] = x.z, row[3] = x.w;
  }
  if (threadIdx.x < 32) {
    // Token i's run: the largest aligned group of 8, 4 or 2 slots around its
    // own that consecutive tokens of the tile fill.
    const int i = threadIdx.x;
    long long s = i < n ? a.slots[t0 + i] : -1;
    if (s < 0 || s >= a.n_slots) s = -1;
    const long long after = __shfl_down_sync(~0u, s, 1);   // by every lane, before the test
    const uint32_t next = __ballot_sync(~0u, s >= 0 && after == s + 1);
    int w = 1;
    bool leads = s >= 0;
    for (int x = 2; x <= 8; x <<= 1) {
      const int j = i - static_cast<int>(s & (x - 1));
      if (s < 0 || j < 0) continue;
      const uint32_t need = ((1u << (x - 1)) - 1u) << j;   // j's neighbours up to j + x - 1
      if (j + x <= kCacheBlock && (next & need) == need) {
        w = x;
        leads = j == i;
      }
    }
    const uint32_t m = __ballot_sync(~0u, i < kCacheBlock && leads);
    if (i < kCacheBlock) {
      slot[i] = s;
      width[i] = w;
    }
    if (i == 0) width[kCacheBlock] = static_cast<int>(m);
  }
  __syncthreads();
  // Two threads per dimension, each with every other run.
  const int d = threadIdx.x >> 1;
  const uint16_t *col = reinterpret_cast<const uint16_t *>(smem) + d;
  auto at = [&](int i) { return static_cast<uint32_t>(col[i * (kRow / 2)]); };
  int turn = 0;
  for (uint32_t runs = width[kCacheBlock]; runs != 0; runs &= runs - 1, ++turn) {
    if ((turn & 1) != (threadIdx.x & 1)) continue;
    const int i = __ffs(runs) - 1;
    uint16_t *dst = reinterpret_cast<uint16_t *>(a.v_cache) +
                    ((slot[i] / kCacheBlock * a.Hk + h) * D + d) * kCacheBlock +
                    slot[i] % kCacheBlock;
    const int w = width[i];
    if (w == 8) {
      *reinterpret_cast<uint4 *>(dst) =
          make_uint4(at(i) | at(i + 1) << 16, at(i + 2) | at(i + 3) << 16,
                     at(i + 4) | at(i + 5) << 16, at(i + 6) | at(i + 7) << 16);
    } else if (w == 4) {
      *reinterpret_cast<uint2 *>(dst) =
          make_uint2(at(i) | at(i + 1) << 16, at(i + 2) | at(i + 3) << 16);
    } else if (w == 2) {
      *reinterpret_cast<uint32_t *>(dst) = at(i) | at(i + 1) << 16;
    } else {
      *dst = static_cast<uint16_t>(at(i));
    }
  }
}

template <typename T, int D, bool CACHE>
__global__ void __launch_bounds__(kThreads) qk_prep_kernel(const PrepArgs a) {
  constexpr int L = D / 16;            // threads per row
  constexpr int kRows = kThreads / L;  // rows a block takes at a time
  constexpr int kTable = kMaxTok * Table<L>::kStride * 16;
  __shared__ __align__(16) uint8_t smem[CACHE && kTable < kValueBytes ? kValueBytes : kTable];
  __shared__ uint64_t frac[kMaxPairs];
  float4 *cs = reinterpret_cast<float4 *>(smem);
  if (CACHE && static_cast<int>(blockIdx.x) >= a.qk_blocks) {
    write_values(a, blockIdx.x - a.qk_blocks, smem);
    return;
  }
  const int tile = blockIdx.x / a.row_blocks, part = blockIdx.x - tile * a.row_blocks;
  const int tok = 1 << a.tok_shift;
  const int t0 = tile * tok, n_tok = min(tok, a.T - t0);
  const int rows = (a.H + a.Hk) * tok;   // token fastest
  const int l = threadIdx.x % L;
  const bool half = a.half != 0;
  int c0, c1;
  chunks_of<D>(l, a.rot, half, c0, c1);
  auto source = [&](int row) -> const T * {
    const int h = row >> a.tok_shift, t = t0 + (row & (tok - 1));
    return h < a.H ? reinterpret_cast<const T *>(a.q) + t * a.q_stride + h * D
                   : reinterpret_cast<const T *>(a.k) + t * a.k_stride + (h - a.H) * D;
  };
  // The first rows are on their way while the angles are computed.
  int row = part * kRows + threadIdx.x / L;
  const int step = kRows * a.row_blocks;
  auto live = [&](int r) { return r < rows && (r & (tok - 1)) < n_tok; };
  Chunk<T> x0, x1;
  if (live(row)) {
    const T *p = source(row);
    x0.load(p + c0 * 8);
    x1.load(p + c1 * 8);
  }
  const int pairs = a.rot >> 1;
  for (int i = threadIdx.x; i < pairs; i += kThreads) frac[i] = turn_fraction(a.inv_freq[i]);
  __syncthreads();
  fill_table<L>(cs, frac, a.positions, t0, n_tok, pairs, a.mscale);
  __syncthreads();
  // Every lane of a warp makes the same number of rounds (the row sum's
  // shuffles), so the loop runs on the warp's first row.
  for (int first = row - (threadIdx.x % 32) / L; first < rows; first += step, row += step) {
    const bool on = live(row);
    float f0[8] = {}, f1[8] = {};
    if (on) {
      x0.get(f0);
      x1.get(f1);
    }
    const int h = row >> a.tok_shift, tt = row & (tok - 1), t = t0 + tt;
    if (live(row + step)) {
      const T *p = source(row + step);
      x0.load(p + c0 * 8);
      x1.load(p + c1 * 8);
    }
    const T *w = reinterpret_cast<const T *>(h < a.H ? a.qw : a.kw);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(f0[i], f0[i], fmaf(f1[i], f1[i], s));
    s = row_sum<L>(s);
    if (!on) continue;
    if (w != nullptr) {
      const float r = rsqrtf(s * (1.f / D) + a.eps);
      Chunk<T> w0, w1;
      float g0[8], g1[8];
      w0.load(w + c0 * 8);
      w1.load(w + c1 * 8);
      w0.get(g0);
      w1.get(g1);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        f0[i] *= r * g0[i];
        f1[i] *= r * g1[i];
      }
    }
    rotate<L>(f0, f1, l, a.rot, half, cs + tt * Table<L>::kStride, 1.f);
    if (h < a.H) {
      T *o = reinterpret_cast<T *>(a.q_out) + (static_cast<int64_t>(t) * a.H + h) * D;
      Chunk<T>::store(o + c0 * 8, f0);
      Chunk<T>::store(o + c1 * 8, f1);
    } else if (CACHE) {
      const long long slot = a.slots[t];
      if (slot < 0 || slot >= a.n_slots) continue;
      T *o = reinterpret_cast<T *>(a.k_out) +
             (slot / kCacheBlock * a.Hk + (h - a.H)) * (D * kCacheBlock) +
             slot % kCacheBlock * 8;
      Chunk<T>::store(o + c0 * (8 * kCacheBlock), f0);
      Chunk<T>::store(o + c1 * (8 * kCacheBlock), f1);
    } else {
      T *o = reinterpret_cast<T *>(a.k_out) + (static_cast<int64_t>(t) * a.Hk + h - a.H) * D;
      Chunk<T>::store(o + c0 * 8, f0);
      Chunk<T>::store(o + c1 * 8, f1);
    }
  }
}

struct PrepGradArgs {
  const void *dyq, *dyk, *q, *k, *qw, *kw;
  const int *positions;
  const double *inv_freq;
  void *dq, *dk;
  float *partial;               // [grid][2][D], null when neither side has a weight
  int T, H, Hk, rot, half;
  int64_t q_stride, k_stride;
  float eps, mscale;
  int tiles;                    // token tiles of kMaxTok
};

// Backward: persistent blocks take every gridDim.x-th tile of kMaxTok tokens.
// A thread always owns the same 16 columns of a row, so the weights'
// gradients are register sums over its rows, joined over the block at the
// end and over the blocks by a second kernel, in an order that depends on
// the sizes alone.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) qk_prep_grad_kernel(const PrepGradArgs a) {
  constexpr int L = D / 16;
  constexpr int kRows = kThreads / L;
  __shared__ __align__(16) float4 cs[kMaxTok * Table<L>::kStride];
  __shared__ uint64_t frac[kMaxPairs];
  __shared__ float sums[kThreads / 32][2][D];
  const int l = threadIdx.x % L, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool half = a.half != 0;
  int c0, c1;
  chunks_of<D>(l, a.rot, half, c0, c1);
  const int pairs = a.rot >> 1;
  for (int i = threadIdx.x; i < pairs; i += kThreads) frac[i] = turn_fraction(a.inv_freq[i]);
  float dw[2][16];
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int i = 0; i < 16; ++i) dw[u][i] = 0.f;
  for (int tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
    const int t0 = tile * kMaxTok, n_tok = min(kMaxTok, a.T - t0);
    __syncthreads();   // frac is ready; the last tile's table has been read
    fill_table<L>(cs, frac, a.positions, t0, n_tok, pairs, a.mscale);
    __syncthreads();
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const int heads = side ? a.Hk : a.H;
      const int64_t stride = side ? a.k_stride : a.q_stride;
      const T *dy = reinterpret_cast<const T *>(side ? a.dyk : a.dyq);
      const T *xs = reinterpret_cast<const T *>(side ? a.k : a.q);
      const T *w = reinterpret_cast<const T *>(side ? a.kw : a.qw);
      T *dx = reinterpret_cast<T *>(side ? a.dk : a.dq);
      float w0[8], w1[8];
      if (w != nullptr) {
        Chunk<T> b0, b1;
        b0.load(w + c0 * 8);
        b1.load(w + c1 * 8);
        b0.get(w0);
        b1.get(w1);
      }
      const int rows = heads * kMaxTok;
      int row = threadIdx.x / L;
      for (int first = row - lane / L; first < rows; first += kRows, row += kRows) {
        const int h = row / kMaxTok, tt = row % kMaxTok;
        const bool on = row < rows && tt < n_tok;
        const int64_t t = t0 + tt;
        float g0[8] = {}, g1[8] = {}, x0[8] = {}, x1[8] = {};
        if (on) {
          Chunk<T> b0, b1, b2, b3;
          const T *p = dy + (t * heads + h) * D;
          b0.load(p + c0 * 8);
          b1.load(p + c1 * 8);
          if (w != nullptr) {
            const T *px = xs + t * stride + h * D;
            b2.load(px + c0 * 8);
            b3.load(px + c1 * 8);
            b2.get(x0);
            b3.get(x1);
          }
          b0.get(g0);
          b1.get(g1);
          rotate<L>(g0, g1, l, a.rot, half, cs + tt * Table<L>::kStride, -1.f);
        }
        if (w != nullptr) {
          float ss = 0.f, wgx = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            ss = fmaf(x0[i], x0[i], fmaf(x1[i], x1[i], ss));
            wgx = fmaf(w0[i] * g0[i], x0[i], fmaf(w1[i] * g1[i], x1[i], wgx));
          }
          ss = row_sum<L>(ss);
          wgx = row_sum<L>(wgx);
          const float r = rsqrtf(ss * (1.f / D) + a.eps);
          const float m = r * r * (wgx * (1.f / D));
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dw[side][i] = fmaf(g0[i] * x0[i], r, dw[side][i]);
            dw[side][8 + i] = fmaf(g1[i] * x1[i], r, dw[side][8 + i]);
            g0[i] = r * (w0[i] * g0[i] - x0[i] * m);
            g1[i] = r * (w1[i] * g1[i] - x1[i] * m);
          }
        }
        if (on) {
          T *o = dx + (t * heads + h) * D;
          Chunk<T>::store(o + c0 * 8, g0);
          Chunk<T>::store(o + c1 * 8, g1);
        }
      }
    }
  }
  if (a.partial == nullptr) return;
  // Lanes l, l + L, ... of a warp hold the same columns.
#pragma unroll
  for (int side = 0; side < 2; ++side)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float v = dw[side][i];
#pragma unroll
      for (int off = L; off < 32; off <<= 1) v += __shfl_xor_sync(~0u, v, off);
      if (lane < L) sums[warp][side][(i < 8 ? c0 : c1) * 8 + (i & 7)] = v;
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
    float v = 0.f;
#pragma unroll
    for (int u = 0; u < kThreads / 32; ++u) v += sums[u][i / D][i % D];
    a.partial[static_cast<int64_t>(blockIdx.x) * 2 * D + i] = v;
  }
}

// Joins the blocks' weight gradients: a block per 32 columns, 32 strands of
// partials each, summed in a fixed order.
__global__ void __launch_bounds__(1024)
    qk_prep_grad_join_kernel(const float *__restrict__ partial, int n, int D,
                             float *__restrict__ dqw, float *__restrict__ dkw) {
  __shared__ float s[32][33];
  const int col = blockIdx.x * 32 + threadIdx.x;
  float v = 0.f;
  for (int i = threadIdx.y; i < n; i += 32) v += partial[static_cast<int64_t>(i) * 2 * D + col];
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y != 0) return;
  v = 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i) v += s[i][threadIdx.x];
  float *out = col < D ? dqw : dkw;
  if (out != nullptr) out[col < D ? col : col - D] = v;
}

int num_sms(cudaError_t *e) {
  int dev = 0, n = 0;
  if ((*e = cudaGetDevice(&dev)) == cudaSuccess)
    *e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n;
}

template <typename T, int D, bool CACHE>
cudaError_t launch_prep_d(PrepArgs a, cudaStream_t stream) {
  constexpr int kRows = kThreads * 16 / D;
  cudaError_t e;
  const int sms = num_sms(&e);
  if (e != cudaSuccess) return e;
  const int heads = a.H + a.Hk;
  // Four tokens a block share the angles' cost and give the key cache 64-byte
  // runs; with too few tokens to fill the GPU, one token a block, and its
  // heads over several blocks, so that every load is in flight at once.
  a.tok_shift = 2;
  static_assert(kMaxTok == 4, "tok_shift");
  while (a.tok_shift > 0 && (static_cast<int64_t>(a.T) >> a.tok_shift) < 4 * sms) --a.tok_shift;
  const int tok = 1 << a.tok_shift;
  const int tiles = static_cast<int>((static_cast<int64_t>(a.T) + tok - 1) / tok);
  const int rounds = (heads * tok + kRows - 1) / kRows;
  a.row_blocks = 1;
  while (a.row_blocks < rounds && static_cast<int64_t>(tiles) * a.row_blocks < 4 * sms)
    ++a.row_blocks;
  const int64_t qk = static_cast<int64_t>(tiles) * a.row_blocks;
  const int64_t vb =
      CACHE ? (static_cast<int64_t>(a.T) + kCacheBlock - 1) / kCacheBlock * a.Hk : 0;
  if (qk + vb > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  a.qk_blocks = static_cast<int>(qk);
  qk_prep_kernel<T, D, CACHE><<<static_cast<unsigned>(qk + vb), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_prep_t(const PrepArgs &a, int d, cudaStream_t stream) {
  switch (d) {
    case 64: return launch_prep_d<T, 64, false>(a, stream);
    case 128: return launch_prep_d<T, 128, false>(a, stream);
    default: return launch_prep_d<T, 256, false>(a, stream);
  }
}

// Blocks of the backward: up to four per SM, each with at least one tile.
int grad_blocks(int T, int sms) {
  const int tiles = (T + kMaxTok - 1) / kMaxTok;
  return tiles < 4 * sms ? tiles : 4 * sms;
}

template <typename T, int D>
cudaError_t launch_grad_d(const PrepGradArgs &a, float *dqw, float *dkw, cudaStream_t stream) {
  cudaError_t e;
  const int sms = num_sms(&e);
  if (e != cudaSuccess) return e;
  const int blocks = grad_blocks(a.T, sms);
  qk_prep_grad_kernel<T, D><<<blocks, kThreads, 0, stream>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess || a.partial == nullptr) return e;
  qk_prep_grad_join_kernel<<<2 * D / 32, dim3(32, 32), 0, stream>>>(a.partial, blocks, D, dqw,
                                                                    dkw);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_grad_t(const PrepGradArgs &a, int d, float *dqw, float *dkw,
                          cudaStream_t stream) {
  switch (d) {
    case 64: return launch_grad_d<T, 64>(a, dqw, dkw, stream);
    case 128: return launch_grad_d<T, 128>(a, dqw, dkw, stream);
    default: return launch_grad_d<T, 256>(a, dqw, dkw, stream);
  }
}

}  // namespace

cudaError_t launch_qk_prep(ElemType type, const QkPrep &p, void *q_out, void *k_out,
                           cudaStream_t stream) {
  PrepArgs a{};
  a.q = p.q, a.k = p.k, a.qw = p.q_weight, a.kw = p.k_weight;
  a.positions = p.positions, a.inv_freq = p.inv_freq;
  a.q_out = q_out, a.k_out = k_out;
  a.T = p.T, a.H = p.H, a.Hk = p.Hk, a.rot = p.rot, a.half = !p.interleaved;
  a.q_stride = p.q_stride, a.k_stride = p.k_stride;
  a.eps = p.eps, a.mscale = p.mscale;
  switch (type) {
    case ElemType::kBf16: return launch_prep_t<__nv_bfloat16>(a, p.d, stream);
    case ElemType::kF16: return launch_prep_t<__half>(a, p.d, stream);
    default: return launch_prep_t<float>(a, p.d, stream);
  }
}

cudaError_t launch_qk_prep_cache(const QkPrep &p, const void *v, int64_t v_stride,
                                 const long long *slots, int64_t n_slots, void *q_out,
                                 void *k_cache, void *v_cache, cudaStream_t stream) {
  PrepArgs a{};
  a.q = p.q, a.k = p.k, a.v = v, a.qw = p.q_weight, a.kw = p.k_weight;
  a.positions = p.positions, a.inv_freq = p.inv_freq, a.slots = slots;
  a.q_out = q_out, a.k_out = k_cache, a.v_cache = v_cache;
  a.T = p.T, a.H = p.H, a.Hk = p.Hk, a.rot = p.rot, a.half = !p.interleaved;
  a.q_stride = p.q_stride, a.k_stride = p.k_stride, a.v_stride = v_stride, a.n_slots = n_slots;
  a.eps = p.eps, a.mscale = p.mscale;
  return launch_prep_d<__nv_bfloat16, kDecodeHeadSize, true>(a, stream);
}

size_t qk_prep_grad_workspace_bytes(int T, int d) {
  // The most blocks any launch uses (the grid follows the SM count).
  return sizeof(float) * 2 * static_cast<size_t>(d) * static_cast<size_t>(grad_blocks(T, 256));
}

cudaError_t launch_qk_prep_grad(ElemType type, const QkPrep &p, const void *dq_out,
                                const void *dk_out, void *dq, void *dk, float *dqw, float *dkw,
                                float *workspace, cudaStream_t stream) {
  PrepGradArgs a{};
  a.dyq = dq_out, a.dyk = dk_out, a.q = p.q, a.k = p.k, a.qw = p.q_weight, a.kw = p.k_weight;
  a.positions = p.positions, a.inv_freq = p.inv_freq, a.dq = dq, a.dk = dk;
  a.partial = (dqw != nullptr || dkw != nullptr) ? workspace : nullptr;
  a.T = p.T, a.H = p.H, a.Hk = p.Hk, a.rot = p.rot, a.half = !p.interleaved;
  a.q_stride = p.q_stride, a.k_stride = p.k_stride;
  a.eps = p.eps, a.mscale = p.mscale;
  a.tiles = static_cast<int>((static_cast<int64_t>(p.T) + kMaxTok - 1) / kMaxTok);
  switch (type) {
    case ElemType::kBf16: return launch_grad_t<__nv_bfloat16>(a, p.d, dqw, dkw, stream);
    case ElemType::kF16: return launch_grad_t<__half>(a, p.d, dqw, dkw, stream);
    default: return launch_grad_t<float>(a, p.d, dqw, dkw, stream);
  }
}

}  // namespace fattn
