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
// therefore a 64-bit fixed-point fraction: inv_freq / 2 pi becomes 2^64 frac, and
// position * that, in wrapping 64-bit integer arithmetic, is the exact angle modulo
// a turn (error < |position| 2^-64 turns beside inv_freq's own rounding).  Its top
// 32 bits go to sincospif.
//
// Bound by HBM bytes: every value is read once and written once, 16 bytes a
// load.  What stands between a kernel like this and that bound is its instruction
// count, so:
//  * A thread owns two 8-value chunks of a row, chosen so that both members of
//    every pair are its own (half layout: chunk l and chunk l + rot/16;
//    interleaved: any two): the rotation needs no exchange, and the norm's sum one
//    butterfly over d/16 lanes.
//  * Chunks are unpacked into first and second members, two values to a packed
//    fp32 register, whatever the layout: one rotation code for both, at two values
//    an instruction.
//  * A thread's token stays the same from round to round (rows go token first), so
//    its addresses advance by a constant.
// The rows of a warp are consecutive tokens of one head, so the 16-byte pieces of a
// key that the cache keeps 16 tokens wide fill whole sectors.  The cosines of a
// token serve all its heads: a block takes up to kMaxTok tokens and computes them
// once.
//
// Measured, bf16 unless said: into the cache, 32 + 8 heads, d = 128: 64 tokens 4.7 us
// (launch and two dependent loads), 4099 tokens 24.4 us (4.1 TB/s; V's transposition 3
// us of it); dense fp16, 16384 tokens, 16 + 16 heads, d = 64: 26.6 us (5.1 TB/s; a copy
// by the same loads and stores runs 13% faster); backward, 8192 tokens, 32 + 8 heads:
// 54.5 us (4.6 TB/s).  Neither DRAM (28% and 52% busy into the cache and backward) nor
// the issue slots (55% and 50%) are full: what is left is latency, into the cache a
// block's angle table, barrier and first rows in series, backward the rows that 24 warps
// an SM keep in flight.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"

namespace fattn {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTok = 8;       // tokens per block
constexpr int kCacheBlock = kDecodeBlockSize;

// Two chunks of eight consecutive values, as they lie in memory.
template <typename T>
struct Chunks {
  uint4 c[2];
  __device__ __forceinline__ void load(const T *p, int c0, int c1) {
    c[0] = *reinterpret_cast<const uint4 *>(p + c0 * 8);
    c[1] = *reinterpret_cast<const uint4 *>(p + c1 * 8);
  }
};
template <>
struct Chunks<float> {
  uint4 c[4];
  __device__ __forceinline__ void load(const float *p, int c0, int c1) {
    const uint4 *x = reinterpret_cast<const uint4 *>(p + c0 * 8);
    const uint4 *y = reinterpret_cast<const uint4 *>(p + c1 * 8);
    c[0] = x[0], c[1] = x[1], c[2] = y[0], c[3] = y[1];
  }
};

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);   // two values, low half first
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  return pack_bf16x2(lo, hi);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// The 16 values of a thread as eight pairs: the first members a, the second members
// b, two pairs to a packed register.  HALF: a is chunk 0, b is chunk 1; interleaved:
// chunk 0 holds pairs 0 .. 3, chunk 1 pairs 4 .. 7.
struct Pairs {
  uint64_t a[4], b[4];
};
template <typename T, bool HALF>
__device__ __forceinline__ Pairs unpack(const Chunks<T> &x) {
  Pairs p;
  if constexpr (sizeof(T) == 4) {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(x.c);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = HALF ? 2 * i : 4 * i;   // first member of pair 2 i
      p.a[i] = f2(__uint_as_float(w[e]), __uint_as_float(w[HALF ? e + 1 : e + 2]));
      p.b[i] = f2(__uint_as_float(w[HALF ? e + 8 : e + 1]), __uint_as_float(w[HALF ? e + 9 : e + 3]));
    }
  } else {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(x.c);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (HALF) {
        const float2 u = unpack2<T>(w[i]), v = unpack2<T>(w[4 + i]);
        p.a[i] = f2(u.x, u.y);
        p.b[i] = f2(v.x, v.y);
      } else {
        const float2 u = unpack2<T>(w[2 * i]), v = unpack2<T>(w[2 * i + 1]);
        p.a[i] = f2(u.x, v.x);
        p.b[i] = f2(u.y, v.y);
      }
    }
  }
  return p;
}
// Rounds once and stores the two chunks at their places c0, c1 of a row; `step`:
// values between chunks (8 in a dense row).
template <typename T, bool HALF>
__device__ __forceinline__ void store(T *row, int c0, int c1, int step, const Pairs &p) {
  constexpr int kWords = sizeof(T) == 4 ? 16 : 8;
  uint32_t w[kWords];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = f2_split(p.a[i]), b = f2_split(p.b[i]);
    if constexpr (sizeof(T) == 4) {
      const int e = HALF ? 2 * i : 4 * i;
      w[e] = __float_as_uint(a.x);
      w[HALF ? e + 1 : e + 2] = __float_as_uint(a.y);
      w[HALF ? e + 8 : e + 1] = __float_as_uint(b.x);
      w[HALF ? e + 9 : e + 3] = __float_as_uint(b.y);
    } else if (HALF) {
      w[i] = pack2<T>(a.x, a.y);
      w[4 + i] = pack2<T>(b.x, b.y);
    } else {
      w[2 * i] = pack2<T>(a.x, b.x);
      w[2 * i + 1] = pack2<T>(a.y, b.y);
    }
  }
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int v = 0; v < kWords / 8; ++v)
      reinterpret_cast<uint4 *>(row + (u ? c1 : c0) * step)[v] =
          make_uint4(w[u * (kWords / 2) + 4 * v], w[u * (kWords / 2) + 4 * v + 1],
                     w[u * (kWords / 2) + 4 * v + 2], w[u * (kWords / 2) + 4 * v + 3]);
}
__device__ __forceinline__ float sum2(uint64_t v) {
  const float2 x = f2_split(v);
  return x.x + x.y;
}
__device__ __forceinline__ float sum_squares(const Pairs &p) {
  uint64_t s = fmul2(p.a[0], p.a[0]), t = fmul2(p.b[0], p.b[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    s = ffma2(p.a[i], p.a[i], s);
    t = ffma2(p.b[i], p.b[i], t);
  }
  return sum2(fadd2(s, t));
}

// The two chunks that thread l of a row's D/16 owns.  Half layout: chunk l of
// the rotated part with its partner l + rot/16, then the chunks past rot two
// by two; interleaved: two by two.
template <bool HALF>
__device__ __forceinline__ void chunks_of(int l, int rot, int &c0, int &c1) {
  const int n = rot >> 4;   // pairs of chunks in the rotated part
  c0 = HALF && l < n ? l : 2 * l;
  c1 = HALF && l < n ? l + n : 2 * l + 1;
}

// Angle table of a token: in either layout thread l of a row rotates pairs
// 8 l .. 8 l + 7, if those are below rot / 2, with four float4 of its own (eight
// cosines, eight sines); the four are L apart, so that a row's lanes read
// consecutive 16-byte words.
template <int L>
struct Table {
  static constexpr int kStride = 4 * L + 4;   // float4 per token (the 4: bank spread)
  __device__ static int at(int pair) {        // the cosine, in floats
    return (((pair & 7) >> 2) * L + (pair >> 3)) * 4 + (pair & 3);
  }
  static constexpr int kSine = 2 * L * 4;     // from a cosine to its sine
};
struct Angles {
  uint64_t c[4], s[4];
};
template <int L>
__device__ __forceinline__ Angles read_angles(const float4 *table, int l) {
  Angles t;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float4 c = table[j * L + l], s = table[(2 + j) * L + l];
    t.c[2 * j] = f2(c.x, c.y), t.c[2 * j + 1] = f2(c.z, c.w);
    t.s[2 * j] = f2(s.x, s.y), t.s[2 * j + 1] = f2(s.z, s.w);
  }
  return t;
}
__device__ __forceinline__ uint64_t neg2(uint64_t v) { return v ^ 0x8000000080000000ull; }
// (a, b) -> (a c - b s, b c + a s); backward: by the opposite angles.
template <bool BACK>
__device__ __forceinline__ void rotate(Pairs &p, const Angles &t) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t a = p.a[i], b = p.b[i], ns = neg2(t.s[i]);
    p.a[i] = ffma2(a, t.c[i], fmul2(b, BACK ? t.s[i] : ns));
    p.b[i] = ffma2(b, t.c[i], fmul2(a, BACK ? ns : t.s[i]));
  }
}

// inv_freq (radians per position) as a 64-bit fraction of a turn, round-off below
// 2^-53 of it, in integers: with inv_freq = m 2^(e - 52), the product of m and
// 2^66 / 2 pi shifted right by 54 - e.
__device__ __forceinline__ uint64_t turn_fraction(double inv_freq) {
  constexpr uint64_t kScale = 11743562013128004906ull;   // 2^66 / (2 pi)
  const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(inv_freq));
  const int e = static_cast<int>(bits >> 52 & 0x7ff) - 1023;
  const uint64_t m = (bits & 0xfffffffffffffull) | 0x10000000000000ull;
  const uint64_t lo = m * kScale, hi = __umul64hi(m, kScale);
  const int shift = 54 - e;
  uint64_t f = 0;
  if (shift >= 128) {
    f = 0;                                  // (zero and subnormal frequencies too)
  } else if (shift >= 64) {
    f = hi >> (shift - 64);
  } else if (shift > 0) {
    f = lo >> shift | hi << (64 - shift);
  } else if (shift > -64) {
    f = lo << -shift;
  }
  return bits >> 63 ? 0 - f : f;
}

// (cos, sin) of tokens t0 .. t0 + n - 1, times mscale, into their tables.
template <int L>
__device__ __forceinline__ void fill_table(float4 *cs, const double *inv_freq,
                                           const int *positions, int64_t t0, int n, int pairs,
                                           float mscale) {
  for (int i = threadIdx.x; i < n * pairs; i += kThreads) {
    const int t = i / pairs, p = i - t * pairs;
    const int position = positions[t0 + t];
    const uint64_t turns =
        static_cast<uint64_t>(static_cast<int64_t>(position)) * turn_fraction(inv_freq[p]);
    // Signed top half: the angle in [-1/2, 1/2) turns, in units of 2^-32.
    const float x = static_cast<float>(static_cast<int32_t>(turns >> 32)) * 0x1p-31f;
    float s, c;
    sincospif(x, &s, &c);
    float *dst = reinterpret_cast<float *>(cs + t * Table<L>::kStride) + Table<L>::at(p);
    dst[0] = c * mscale;
    dst[Table<L>::kSine] = s * mscale;
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
  int T, H, Hk, rot;
  int64_t q_stride, k_stride, v_stride, n_slots;
  float eps, mscale;
  int tok_shift;                // log2 of the tokens per block (1 .. kMaxTok)
  int row_blocks;               // blocks that share a token tile's rounds of rows
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

template <typename T, int D, bool HALF, bool CACHE>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 3 : 6) qk_prep_kernel(const PrepArgs a) {
  constexpr int L = D / 16;            // threads per row
  constexpr int kRows = kThreads / L;  // rows a block takes in a round
  static_assert(kRows % kMaxTok == 0, "a thread keeps its token");
  constexpr int kTable = kMaxTok * Table<L>::kStride * 16;
  __shared__ __align__(16) uint8_t smem[CACHE && kTable < kValueBytes ? kValueBytes : kTable];
  float4 *cs = reinterpret_cast<float4 *>(smem);
  if (CACHE && static_cast<int>(blockIdx.x) >= a.qk_blocks) {
    write_values(a, blockIdx.x - a.qk_blocks, smem);
    return;
  }
  const int tile = blockIdx.x / a.row_blocks, part = blockIdx.x - tile * a.row_blocks;
  const int tok = 1 << a.tok_shift;
  const int t0 = tile * tok, n_tok = min(tok, a.T - t0);
  const int l = threadIdx.x % L;
  int c0, c1;
  chunks_of<HALF>(l, a.rot, c0, c1);
  // This thread's token, and its head in a side's round r: h0 + r * heads.
  const int tt = threadIdx.x / L & (tok - 1), h0 = threadIdx.x / L >> a.tok_shift;
  const int heads = kRows >> a.tok_shift;
  const int64_t t = t0 + tt;
  const bool own = tt < n_tok;
  // The block's rounds: every row_blocks-th of the queries' and then the keys'.
  const int q_rounds = (a.H + heads - 1) / heads, k_rounds = (a.Hk + heads - 1) / heads;
  const int k_first = q_rounds <= part ? part - q_rounds
                                       : (a.row_blocks - (q_rounds - part) % a.row_blocks) % a.row_blocks;
  const T *q = reinterpret_cast<const T *>(a.q) + t * a.q_stride;
  const T *k = reinterpret_cast<const T *>(a.k) + t * a.k_stride;
  // (The queries' first rows are on their way while the angles are computed.)
  const int pairs = a.rot >> 1;
  bool ready = false;
  const bool turns = l * 16 < a.rot;
  // The rounds of one side; `put` stores a row's result.  (Angles and weights are
  // read again in each, from shared memory and L1: holding them takes 90 registers and
  // leaves two blocks an SM where 40 let six take turns, 38 us against 24 for 4099
  // tokens of 32 + 8 heads.)
  auto side = [&](const T *src, const T *weight, int n_heads, int first, int rounds,
                  auto &&put) {
    Chunks<T> x;
    if (own && first < rounds && h0 + first * heads < n_heads)
      x.load(src + (h0 + first * heads) * D, c0, c1);
    if (!ready) {
      fill_table<L>(cs, a.inv_freq, a.positions, t0, n_tok, pairs, a.mscale);
      __syncthreads();
      ready = true;
    }
    for (int r = first; r < rounds; r += a.row_blocks) {
      const int h = h0 + r * heads;
      const bool on = own && h < n_heads;
      Pairs v{};
      if (on) v = unpack<T, HALF>(x);
      const int next = h + heads * a.row_blocks;
      if (own && next < n_heads) x.load(src + next * D, c0, c1);
      if (weight != nullptr) {
        // (Every lane of the warp takes part in the sum.)
        const float rs = rsqrtf(row_sum<L>(sum_squares(v)) * (1.f / D) + a.eps);
        const uint64_t rs2 = f2(rs, rs);
        Chunks<T> c;
        c.load(weight, c0, c1);
        const Pairs w = unpack<T, HALF>(c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v.a[i] = fmul2(fmul2(v.a[i], rs2), w.a[i]);
          v.b[i] = fmul2(fmul2(v.b[i], rs2), w.b[i]);
        }
      }
      if (!on) continue;
      if (turns) rotate<false>(v, read_angles<L>(cs + tt * Table<L>::kStride, l));
      put(h, v);
    }
  };
  side(q, reinterpret_cast<const T *>(a.qw), a.H, part, q_rounds, [&](int h, const Pairs &v) {
    store<T, HALF>(reinterpret_cast<T *>(a.q_out) + (t * a.H + h) * D, c0, c1, 8, v);
  });
  T *k_row = reinterpret_cast<T *>(a.k_out);
  bool keep = true;
  if (CACHE) {
    // Element c of a cached key is at [head][c / 8][token][c % 8] of its block.
    const long long slot = own ? a.slots[t] : -1;
    keep = slot >= 0 && slot < a.n_slots;
    k_row += slot / kCacheBlock * a.Hk * (D * kCacheBlock) + slot % kCacheBlock * 8;
  } else {
    k_row += t * a.Hk * D;
  }
  side(k, reinterpret_cast<const T *>(a.kw), a.Hk, k_first, k_rounds,
       [&](int h, const Pairs &v) {
         if (!CACHE || keep)
           store<T, HALF>(k_row + h * (CACHE ? D * kCacheBlock : D), c0, c1,
                          CACHE ? 8 * kCacheBlock : 8, v);
       });
}

struct PrepGradArgs {
  const void *dyq, *dyk, *q, *k, *qw, *kw;
  const int *positions;
  const double *inv_freq;
  void *dq, *dk;
  float *partial;               // [blocks][D], the queries' blocks first; null without weights
  int T, H, Hk, rot;
  int64_t q_stride, k_stride;
  float eps, mscale;
  int q_blocks, k_blocks;       // blocks of either side
};

// Blocks of the backward on an SM.  Three of 80 registers, with angles and weights
// read again for every row: 54 us for 8192 tokens of 32 + 8 heads, bf16, against 62
// for two of 126 that hold them.  (fp32 rows take 16 registers more.)
template <typename T>
constexpr int kGradBlocks = sizeof(T) == 4 ? 2 : 3;

// Backward: a block works on one side only (so that one set of sums lives in
// registers), persistent over every q_blocks-th (k_blocks-th) tile of
// kMaxTok tokens.  A thread always owns the same 16 columns of a row, so the
// weights' gradients are register sums over its rows, joined over the block at the
// end and over the blocks by a second kernel, in an order that depends on the sizes
// and the SM count alone.
template <typename T, int D, bool HALF>
__global__ void __launch_bounds__(kThreads, kGradBlocks<T>) qk_prep_grad_kernel(const PrepGradArgs a) {
  constexpr int L = D / 16;
  constexpr int kRows = kThreads / L;
  constexpr int kHeads = kRows / kMaxTok;   // heads per round
  __shared__ __align__(16) float4 cs[2][kMaxTok * Table<L>::kStride];   // by tile parity
  __shared__ float sums[kThreads / 32][D];
  // The kernel that joins the blocks' sums may be scheduled; it waits for this one.
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int l = threadIdx.x % L, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int c0, c1;
  chunks_of<HALF>(l, a.rot, c0, c1);
  const bool is_k = static_cast<int>(blockIdx.x) >= a.q_blocks;
  const int block = is_k ? blockIdx.x - a.q_blocks : blockIdx.x;
  const int blocks = is_k ? a.k_blocks : a.q_blocks;
  const int n_heads = is_k ? a.Hk : a.H;
  const int64_t stride = is_k ? a.k_stride : a.q_stride;
  const T *dy = reinterpret_cast<const T *>(is_k ? a.dyk : a.dyq);
  const T *xs = reinterpret_cast<const T *>(is_k ? a.k : a.q);
  const T *weight = reinterpret_cast<const T *>(is_k ? a.kw : a.qw);
  T *dx = reinterpret_cast<T *>(is_k ? a.dk : a.dq);
  const bool norm = weight != nullptr;
  const int pairs = a.rot >> 1;
  const int tt = threadIdx.x / L & (kMaxTok - 1), h0 = threadIdx.x / L / kMaxTok;
  const bool turns = l * 16 < a.rot;
  Pairs dw{};
  // Rows of the tile from token t0: this thread's first is loaded a tile ahead.
  Chunks<T> y, x;
  auto load = [&](int64_t t0, int h) {
    const int64_t t = t0 + tt;
    if (t >= a.T || h >= n_heads) return;
    y.load(dy + (t * n_heads + h) * D, c0, c1);
    if (norm) x.load(xs + t * stride + h * D, c0, c1);
  };
  const int64_t step = static_cast<int64_t>(blocks) * kMaxTok;
  load(static_cast<int64_t>(block) * kMaxTok, h0);
  int parity = 0;
  for (int64_t t0 = static_cast<int64_t>(block) * kMaxTok; t0 < a.T; t0 += step, parity ^= 1) {
    const int n_tok = static_cast<int>(min(static_cast<int64_t>(kMaxTok), a.T - t0));
    // (The table of two tiles before has been read: a barrier lies between.)
    fill_table<L>(cs[parity], a.inv_freq, a.positions, t0, n_tok, pairs, a.mscale);
    __syncthreads();
    const bool own = tt < n_tok;
    for (int hr = 0; hr < n_heads; hr += kHeads) {
      const int h = hr + h0;
      const bool on = own && h < n_heads;
      Pairs g{}, v{};
      if (on) {
        g = unpack<T, HALF>(y);
        if (norm) v = unpack<T, HALF>(x);
      }
      // The next row: of this tile, or the first of the next.
      if (hr + kHeads < n_heads)
        load(t0, h + kHeads);
      else
        load(t0 + step, h0);
      if (turns && on) rotate<true>(g, read_angles<L>(cs[parity] + tt * Table<L>::kStride, l));
      if (norm) {
        // ss = sum x^2, wgx = sum w g x
        uint64_t d0 = 0, d1 = 0, wg[8];
        Chunks<T> c;
        c.load(weight, c0, c1);
        const Pairs w = unpack<T, HALF>(c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          wg[i] = fmul2(w.a[i], g.a[i]);
          wg[4 + i] = fmul2(w.b[i], g.b[i]);
          d0 = ffma2(wg[i], v.a[i], d0);
          d1 = ffma2(wg[4 + i], v.b[i], d1);
        }
        const float ss = row_sum<L>(sum_squares(v));
        const float wgx = row_sum<L>(sum2(fadd2(d0, d1)));
        // (Without a row here: nothing, where 0 * rsqrt(eps = 0) would be NaN.  r * r
        // alone could overflow.)
        const float r = on ? rsqrtf(ss * (1.f / D) + a.eps) : 0.f;
        const float m = -r * (r * (wgx * (1.f / D)));
        const uint64_t r2 = f2(r, r), m2 = f2(m, m);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          dw.a[i] = ffma2(fmul2(g.a[i], v.a[i]), r2, dw.a[i]);
          dw.b[i] = ffma2(fmul2(g.b[i], v.b[i]), r2, dw.b[i]);
          g.a[i] = fmul2(r2, ffma2(v.a[i], m2, wg[i]));
          g.b[i] = fmul2(r2, ffma2(v.b[i], m2, wg[4 + i]));
        }
      }
      if (on) store<T, HALF>(dx + ((t0 + tt) * n_heads + h) * D, c0, c1, 8, g);
    }
  }
  if (a.partial == nullptr) return;
  // Lanes l, l + L, ... of a warp hold the same columns: pair j's first member is
  // column col_a(j) of the head, its second col_b(j).
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 fa = f2_split(dw.a[j >> 1]), fb = f2_split(dw.b[j >> 1]);
    float va = j & 1 ? fa.y : fa.x, vb = j & 1 ? fb.y : fb.x;
#pragma unroll
    for (int off = L; off < 32; off <<= 1) {
      va += __shfl_xor_sync(~0u, va, off);
      vb += __shfl_xor_sync(~0u, vb, off);
    }
    if (lane < L) {
      const int base = (j < 4 ? c0 : c1) * 8 + 2 * (j & 3);   // interleaved
      sums[warp][HALF ? c0 * 8 + j : base] = va;
      sums[warp][HALF ? c1 * 8 + j : base + 1] = vb;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < D; i += kThreads) {
    float v = 0.f;
#pragma unroll
    for (int u = 0; u < kThreads / 32; ++u) v += sums[u][i];
    a.partial[static_cast<int64_t>(blockIdx.x) * D + i] = v;
  }
}

// Joins the blocks' weight gradients: a block per 32 columns of a side, 32 strands
// of partials each, summed in a fixed order.
__global__ void __launch_bounds__(1024)
    qk_prep_grad_join_kernel(const float *__restrict__ partial, int q_blocks, int k_blocks, int D,
                             float *__restrict__ dqw, float *__restrict__ dkw) {
  __shared__ float s[32][33];
  const bool is_k = static_cast<int>(blockIdx.x) >= D / 32;
  const int col = (is_k ? blockIdx.x - D / 32 : blockIdx.x) * 32 + threadIdx.x;
  const int n = is_k ? k_blocks : q_blocks;
  const float *src = partial + static_cast<int64_t>(is_k ? q_blocks : 0) * D + col;
  float *out = is_k ? dkw : dqw;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (out == nullptr) return;
  float v = 0.f;
#pragma unroll 8
  for (int i = threadIdx.y; i < n; i += 32) v += src[static_cast<int64_t>(i) * D];
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y != 0) return;
  v = 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i) v += s[i][threadIdx.x];
  out[col] = v;
}

int num_sms(cudaError_t *e) {
  int dev = 0, n = 0;
  if ((*e = cudaGetDevice(&dev)) == cudaSuccess)
    *e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n;
}

template <typename T, int D, bool CACHE>
cudaError_t launch_prep_d(PrepArgs a, bool half, cudaStream_t stream) {
  constexpr int kRows = kThreads * 16 / D;
  cudaError_t e;
  const int sms = num_sms(&e);
  if (e != cudaSuccess) return e;
  // Eight tokens a block share the angles' cost and give the key cache 128-byte
  // runs; with too few tokens to fill the GPU, fewer down to one a block, and its
  // rounds of rows over several blocks, so that every load is in flight at once.
  a.tok_shift = 3;
  static_assert(kMaxTok == 8, "tok_shift");
  while (a.tok_shift > 0 && (static_cast<int64_t>(a.T) >> a.tok_shift) < 4 * sms) --a.tok_shift;
  const int tok = 1 << a.tok_shift, heads = kRows / tok;
  const int tiles = static_cast<int>((static_cast<int64_t>(a.T) + tok - 1) / tok);
  const int rounds = (a.H + heads - 1) / heads + (a.Hk + heads - 1) / heads;
  a.row_blocks = 1;
  while (a.row_blocks < rounds && static_cast<int64_t>(tiles) * a.row_blocks < 4 * sms)
    ++a.row_blocks;
  const int64_t qk = static_cast<int64_t>(tiles) * a.row_blocks;
  const int64_t vb =
      CACHE ? (static_cast<int64_t>(a.T) + kCacheBlock - 1) / kCacheBlock * a.Hk : 0;
  if (qk + vb > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  a.qk_blocks = static_cast<int>(qk);
  const unsigned grid = static_cast<unsigned>(qk + vb);
  if (half)
    qk_prep_kernel<T, D, true, CACHE><<<grid, kThreads, 0, stream>>>(a);
  else
    qk_prep_kernel<T, D, false, CACHE><<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_prep_t(const PrepArgs &a, int d, bool half, cudaStream_t stream) {
  switch (d) {
    case 64: return launch_prep_d<T, 64, false>(a, half, stream);
    case 128: return launch_prep_d<T, 128, false>(a, half, stream);
    default: return launch_prep_d<T, 256, false>(a, half, stream);
  }
}

// Blocks of one side of the backward: at most one per tile of tokens.
int grad_blocks(int T, int most) {
  const int tiles = static_cast<int>((static_cast<int64_t>(T) + kMaxTok - 1) / kMaxTok);
  return tiles < most ? tiles : most;
}

template <typename T, int D>
cudaError_t launch_grad_d(PrepGradArgs a, bool half, float *dqw, float *dkw, cudaStream_t stream) {
  cudaError_t e;
  const int sms = num_sms(&e);
  if (e != cudaSuccess) return e;
  // The sides share the blocks by their heads' rounds.
  constexpr int kHeads = kThreads * 16 / D / kMaxTok;
  const int qr = (a.H + kHeads - 1) / kHeads, kr = (a.Hk + kHeads - 1) / kHeads;
  const int all = kGradBlocks<T> * sms;
  int kb = all * kr / (qr + kr);
  if (kb < 1) kb = 1;
  a.k_blocks = grad_blocks(a.T, kb);
  a.q_blocks = grad_blocks(a.T, all - kb);
  const int grid = a.q_blocks + a.k_blocks;
  if (half)
    qk_prep_grad_kernel<T, D, true><<<grid, kThreads, 0, stream>>>(a);
  else
    qk_prep_grad_kernel<T, D, false><<<grid, kThreads, 0, stream>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess || a.partial == nullptr) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * D / 32);
  cfg.blockDim = dim3(32, 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, qk_prep_grad_join_kernel, static_cast<const float *>(a.partial),
                            a.q_blocks, a.k_blocks, D, dqw, dkw);
}

template <typename T>
cudaError_t launch_grad_t(const PrepGradArgs &a, int d, bool half, float *dqw, float *dkw,
                          cudaStream_t stream) {
  switch (d) {
    case 64: return launch_grad_d<T, 64>(a, half, dqw, dkw, stream);
    case 128: return launch_grad_d<T, 128>(a, half, dqw, dkw, stream);
    default: return launch_grad_d<T, 256>(a, half, dqw, dkw, stream);
  }
}

}  // namespace

cudaError_t launch_qk_prep(ElemType type, const QkPrep &p, void *q_out, void *k_out,
                           cudaStream_t stream) {
  PrepArgs a{};
  a.q = p.q, a.k = p.k, a.qw = p.q_weight, a.kw = p.k_weight;
  a.positions = p.positions, a.inv_freq = p.inv_freq;
  a.q_out = q_out, a.k_out = k_out;
  a.T = p.T, a.H = p.H, a.Hk = p.Hk, a.rot = p.rot;
  a.q_stride = p.q_stride, a.k_stride = p.k_stride;
  a.eps = p.eps, a.mscale = p.mscale;
  switch (type) {
    case ElemType::kBf16: return launch_prep_t<__nv_bfloat16>(a, p.d, !p.interleaved, stream);
    case ElemType::kF16: return launch_prep_t<__half>(a, p.d, !p.interleaved, stream);
    default: return launch_prep_t<float>(a, p.d, !p.interleaved, stream);
  }
}

cudaError_t launch_qk_prep_cache(const QkPrep &p, const void *v, int64_t v_stride,
                                 const long long *slots, int64_t n_slots, void *q_out,
                                 void *k_cache, void *v_cache, cudaStream_t stream) {
  PrepArgs a{};
  a.q = p.q, a.k = p.k, a.v = v, a.qw = p.q_weight, a.kw = p.k_weight;
  a.positions = p.positions, a.inv_freq = p.inv_freq, a.slots = slots;
  a.q_out = q_out, a.k_out = k_cache, a.v_cache = v_cache;
  a.T = p.T, a.H = p.H, a.Hk = p.Hk, a.rot = p.rot;
  a.q_stride = p.q_stride, a.k_stride = p.k_stride, a.v_stride = v_stride, a.n_slots = n_slots;
  a.eps = p.eps, a.mscale = p.mscale;
  return launch_prep_d<__nv_bfloat16, kDecodeHeadSize, true>(a, !p.interleaved, stream);
}

size_t qk_prep_grad_workspace_bytes(int T, int d) {
  // Both sides' blocks, for up to 256 SMs.
  return sizeof(float) * 2 * static_cast<size_t>(d) * static_cast<size_t>(grad_blocks(T, 3 * 256));
}

cudaError_t launch_qk_prep_grad(ElemType type, const QkPrep &p, const void *dq_out,
                                const void *dk_out, void *dq, void *dk, float *dqw, float *dkw,
                                float *workspace, cudaStream_t stream) {
  PrepGradArgs a{};
  a.dyq = dq_out, a.dyk = dk_out, a.q = p.q, a.k = p.k, a.qw = p.q_weight, a.kw = p.k_weight;
  a.positions = p.positions, a.inv_freq = p.inv_freq, a.dq = dq, a.dk = dk;
  a.partial = (dqw != nullptr || dkw != nullptr) ? workspace : nullptr;
  a.T = p.T, a.H = p.H, a.Hk = p.Hk, a.rot = p.rot;
  a.q_stride = p.q_stride, a.k_stride = p.k_stride;
  a.eps = p.eps, a.mscale = p.mscale;
  switch (type) {
    case ElemType::kBf16: return launch_grad_t<__nv_bfloat16>(a, p.d, !p.interleaved, dqw, dkw, stream);
    case ElemType::kF16: return launch_grad_t<__half>(a, p.d, !p.interleaved, dqw, dkw, stream);
    default: return launch_grad_t<float>(a, p.d, !p.interleaved, dqw, dkw, stream);
  }
}

}  // namespace fattn
