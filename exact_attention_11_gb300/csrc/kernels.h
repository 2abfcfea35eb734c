// kernels.h -- launchers shared between the C ABI (api.cu) and the kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace fattn {

constexpr int kDecodeHeadSize = 128;
constexpr int kDecodeBlockSize = 16;
constexpr int kDecodePartitionTokens = 512;

cudaError_t launch_fwd_f32(const float *q, const float *k, const float *v, float *o, float *lse,
                           int BH, int N, int d, float scale, int causal, cudaStream_t stream);

// q, k, v tensor maps: 3-D views {d, N, B*H} of the bf16 inputs, 64 x 128 x 1
// boxes with the 128-byte swizzle.  `sched` points to two ints (the item
// counter and the finished-CTA counter) that are zero before the launch; the
// kernel leaves them zero.  Launches that may run at the same time need
// different `sched` slots.
constexpr int kFwdSchedSlots = 32768;
// fault_cta >= 0 makes that CTA's producer stop after its first Q loads (the
// failure-path test); -1 in normal use.
// f16 selects fp16 Q, K, V, O (tensor maps of CU_TENSOR_MAP_DATA_TYPE_FLOAT16).
// mask (bf16 only, causal 0, N a multiple of 16): uint8, key j visible to row i
// of head bh iff mask[bh * mask_bh_stride + i * N + j] != 0; mask_ranges,
// mask_flags and mask_bits: its tile summary from launch_mask_summary.
cudaError_t launch_fwd_bf16(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                            void *o, float *lse, int BH, int N, int d, float scale, int causal,
                            int *sched, int *dev_status, int fault_cta, cudaStream_t stream,
                            bool f16 = false, const uint8_t *mask = nullptr,
                            int64_t mask_bh_stride = 0, const int2 *mask_ranges = nullptr,
                            const uint8_t *mask_flags = nullptr, const uint4 *mask_bits = nullptr);

// Tile summary of a boolean mask (mask_tiles.cu) for mask_heads heads (1 when
// the mask is shared): per 128 x 128 block a flag (0 nothing visible, 1
// partly, 2 everything), per pair of query tiles the key tiles to process
// (int2 {kv0 | n_a << 16, n_b}, see mask_tiles.cu), per row of each block its
// 128 visibility bits (16 bytes).  ws: mask_summary_bytes(mask_heads, N)
// bytes of 16-byte aligned device memory; *flags, *ranges and *bits point
// into it.
size_t mask_summary_bytes(int mask_heads, int N);
cudaError_t launch_mask_summary(const uint8_t *mask, int64_t bh_stride, int N, int mask_heads,
                                void *ws, uint8_t **flags, const int2 **ranges,
                                const uint4 **bits, cudaStream_t stream);

// Head dimension 256 (fwd_d256.cu), bf16 or (f16) fp16: tq and tk as for
// launch_fwd_bf16 (64 x 128 x 1 boxes), tv with 64 x 64 x 1 boxes.
cudaError_t launch_fwd_d256(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                            void *o, float *lse, int BH, int N, float scale, int causal,
                            int *sched, int *dev_status, cudaStream_t stream, bool f16);

// FP8 forward (fwd_bf16.cu, d = 128): tq, tk are E4M3 maps {128, N, B*H}
// with 128 x 128 x 1 boxes, tvt the E4M3 map {Npad, 128, B*H} of V^T, same
// boxes; all with the 128-byte swizzle.  q_scale, k_scale: one fp32 per
// 128-row block of each head; v_scale: one per head.  o is bf16.  fault_cta
// as for launch_fwd_bf16.
cudaError_t launch_fwd_fp8(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tvt,
                           const float *q_scale, const float *k_scale, const float *v_scale,
                           void *o, float *lse, int BH, int N, float scale, int causal,
                           int *sched, int *dev_status, int fault_cta, cudaStream_t stream);

// FP8 block quantization (fp8_quant.cu, d = 128); v_amax: the workspace of
// fp8_quant_workspace_bytes(BH, N) bytes; signs: 128 fp32 +-1 values or null.
size_t fp8_quant_workspace_bytes(int BH, int N);
cudaError_t launch_fp8_quantize(const void *q, const void *k, const void *v, const float *signs,
                                void *q8, void *k8, void *vt8, float *q_scale, float *k_scale,
                                float *v_scale, float *v_amax, int BH, int N, int n_pad,
                                float rot_factor, int *dev_status, cudaStream_t stream);

// Backward: workspace = fp32 dQ accumulator (row-major [BH][N][d] inside
// B*H*Npad*d floats, Npad = N rounded up to 128), then [-LSE2 | -D] (2 x 128
// fp32) per 128-query block: 4 * B*H*Npad*(d + 2) bytes.  tq and tdo (the map
// of dO) are bf16 maps like the forward's but with boxes of
// bwd_qdo_box_rows(d) rows; tk, tv as in the forward; tdq is the fp32 map of
// the accumulator (boxes of 32 x 32 x 1, 128-byte swizzle).
inline int bwd_qdo_box_rows(int) { return 64; }
size_t bwd_workspace_bytes(int BH, int N, int d);
cudaError_t launch_bwd_bf16(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                            const CUtensorMap &tdo, const CUtensorMap &tdq, const void *o,
                            const void *dout, const float *lse, void *dq, void *dk, void *dv,
                            int BH, int N, int d, float scale, int causal, float *ws,
                            int *sched, int fault_cta, int *dev_status, cudaStream_t stream);

// The d = 128 main kernel (bwd_bf16_d128.cu); vecs = the [-LSE2 | -D]
// blocks, tdq = the fp32 map of the row-major dQ accumulator (TMA reduces);
// sched = a pair of work counters kept at zero (persistent CTAs).
cudaError_t launch_bwd_main_d128(const CUtensorMap &tq64, const CUtensorMap &tk,
                                 const CUtensorMap &tv, const CUtensorMap &tdo64,
                                 const CUtensorMap &tdq, const float *vecs, void *dk, void *dv,
                                 int BH,
                                 int N, float scale, int causal, int *sched, int fault_cta,
                                 int *dev_status, cudaStream_t stream);

// The d = 64 main kernel (bwd_bf16_d64.cu); tdq = the accumulator's fp32 map
// (its dQ' tiles are added with TMA reduces); sched as for d = 128.
cudaError_t launch_bwd_main_d64(const CUtensorMap &tq64, const CUtensorMap &tk,
                                const CUtensorMap &tv, const CUtensorMap &tdo64,
                                const CUtensorMap &tdq, const float *vecs, void *dk, void *dv,
                                int BH, int N, float scale, int causal, int *sched,
                                int fault_cta, int *dev_status, cudaStream_t stream);

// The main kernels for packed sequences: `table` holds for every 128-row key block,
// longest sequence first, its sequence's first row, length and first padded block
// (sequence s starts at block cu_seqlens[s] / 128 + s) and its number in the
// sequence; entries of length 0 end it (or, not `sorted`, lie in between).  The accumulators' maps have n_blocks * 128 rows per head; tdk, tdv
// are used when group > 1.  tq64, tdo64, tk, tv: maps {d, T, heads} of the
// packed tensors.
struct BwdPacked {
  const int4 *table;
  int n_blocks, group, kv_heads, tokens, sorted;
};
// With a window: `count` has the entries used (of at most `entries`), each with the query
// blocks that its items visit (first, number) in `range`, and how many of them come first
// whose items are their query heads, and then whose items are their key/value heads, each
// with all its query heads; the items of the rest are their query heads again.  The key
// blocks that begin below `split` are in several items, which add dK and dV to the
// accumulators.
struct BwdWindow : BwdPacked {
  const int2 *range;
  const int *count;
  int entries, split, window, sinks;
  int grouping;                 // there may be entries with all heads of a group
};
cudaError_t launch_bwd_packed_main_d128(const CUtensorMap &tq64, const CUtensorMap &tk,
                                        const CUtensorMap &tv, const CUtensorMap &tdo64,
                                        const CUtensorMap &tdq, const CUtensorMap &tdk,
                                        const CUtensorMap &tdv, const float *vecs, void *dk,
                                        void *dv, int H, const BwdPacked &pk, float scale,
                                        int causal, int *sched, int *dev_status, int fault_cta,
                                        cudaStream_t stream);
cudaError_t launch_bwd_packed_main_d64(const CUtensorMap &tq64, const CUtensorMap &tk,
                                       const CUtensorMap &tv, const CUtensorMap &tdo64,
                                       const CUtensorMap &tdq, const CUtensorMap &tdk,
                                       const CUtensorMap &tdv, const float *vecs, void *dk,
                                       void *dv, int H, const BwdPacked &pk, float scale,
                                       int causal, int *sched, int *dev_status, int fault_cta,
                                       cudaStream_t stream);

cudaError_t launch_bwd_window_main_d128(const CUtensorMap &tq64, const CUtensorMap &tk,
                                        const CUtensorMap &tv, const CUtensorMap &tdo64,
                                        const CUtensorMap &tdq, const CUtensorMap &tdk,
                                        const CUtensorMap &tdv, const float *vecs, void *dk,
                                        void *dv, int H, const BwdWindow &pk, float scale,
                                        int *sched, int *dev_status, int fault_cta,
                                        cudaStream_t stream);
cudaError_t launch_bwd_window_main_d64(const CUtensorMap &tq64, const CUtensorMap &tk,
                                       const CUtensorMap &tv, const CUtensorMap &tdo64,
                                       const CUtensorMap &tdq, const CUtensorMap &tdk,
                                       const CUtensorMap &tdv, const float *vecs, void *dk,
                                       void *dv, int H, const BwdWindow &pk, float scale,
                                       int *sched, int *dev_status, int fault_cta,
                                       cudaStream_t stream);

int decode_max_parts(int max_num_blocks_per_seq);
// Grouped key/value heads (decode_gqa.cu): group = num_heads / num_kv_heads
// must be 2 or a multiple of 4.  Same workspace and counters as the one-head
// decode (counters indexed per (sequence, query-head group of the CTA)).
bool decode_gqa_group_supported(int group);
cudaError_t launch_paged_decode_gqa(const void *q, const void *k_cache, const void *v_cache,
                                    const int *block_tables, const int *context_lens, void *out,
                                    int num_seqs, int num_heads, int num_kv_heads, int max_blocks,
                                    float scale, float *workspace, int *counters,
                                    int *dev_status, cudaStream_t stream);
// Grouped key/value heads on the tensor cores (decode_gqa_tc.cu): group =
// num_heads / num_kv_heads from 2 to 16, or a multiple of 16.  tm_k / tm_v are
// the TMA views of the caches (encode_paged_kv_maps in api.cu); sched is a
// pair of work counters kept at zero; the workspace is the split-K one below
// (a second kernel merges the partitions; no counters).
bool decode_gqa_tc_supported(int group);
// Below this many (sequence, partition, cached head) units the automatic
// choice keeps the CUDA-core kernel (fewer launches, less set-up).
constexpr long long kDecodeTcMinUnits = 152;
cudaError_t launch_paged_decode_gqa_tc(const CUtensorMap &tm_k, const CUtensorMap &tm_v,
                                       const void *q, const int *block_tables,
                                       const int *context_lens, void *out, int num_seqs,
                                       int num_heads, int num_kv_heads, int max_blocks,
                                       float scale, float *workspace, int *sched,
                                       int *dev_status, cudaStream_t stream);
// Split-K workspace: per (sequence, head, partition) an unnormalised output
// row and its (max, sum) pair, in fp32.  `counters` holds one int per
// (sequence, head); it must be all zero before the first launch and every
// launch leaves it all zero again.
size_t decode_workspace_bytes(int num_seqs, int num_heads, int max_parts);
cudaError_t launch_paged_decode(const void *q, const void *k_cache, const void *v_cache,
                                const int *block_tables, const int *context_lens, void *out,
                                int num_seqs, int num_heads, int max_blocks, float scale,
                                float *workspace, int *counters, cudaStream_t stream);

// Norm and rotation of queries and keys (qk_prep.cu).  d is 64, 128 or 256,
// rot a multiple of 16 up to d; strides in elements between tokens, heads
// dense; weights may be null (no norm on that side).
enum class ElemType { kBf16, kF16, kF32 };
struct QkPrep {
  const void *q, *k, *q_weight, *k_weight;
  const int *positions;
  const double *inv_freq;
  int T, H, Hk, d, rot, interleaved;
  int64_t q_stride, k_stride;
  float eps, mscale;
};
cudaError_t launch_qk_prep(ElemType type, const QkPrep &p, void *q_out, void *k_out,
                           cudaStream_t stream);
// bf16, d = kDecodeHeadSize: keys and values of token t go to slot slots[t]
// of the paged caches; slots outside [0, n_slots) are skipped.
cudaError_t launch_qk_prep_cache(const QkPrep &p, const void *v, int64_t v_stride,
                                 const long long *slots, int64_t n_slots, void *q_out,
                                 void *k_cache, void *v_cache, cudaStream_t stream);
size_t qk_prep_grad_workspace_bytes(int T, int d);
cudaError_t launch_qk_prep_grad(ElemType type, const QkPrep &p, const void *dq_out,
                                const void *dk_out, void *dq, void *dk, float *dqw, float *dkw,
                                float *workspace, cudaStream_t stream);

// Several queries per sequence, sequences of different lengths, grouped heads
// (fwd_packed.cu).  tq: 3-D map {d, H, T} of the queries, boxes of 64 x G x
// packed_tile_tokens(G); packed: tk, tv 3-D maps {d, T, Hk}, boxes of 64 x 128
// x 1; paged: the views of encode_paged_kv_maps with the cache's block count.
// 128-byte swizzle where not paged.  sched as for launch_fwd_bf16.
struct PackedProblem {
  void *o;
  float *lse;                                   // [H][T], packed only, or null
  const int *cu_seqlens, *context_lens, *block_tables;
  int S, T, H, Hk, max_blocks, num_blocks, causal;
  float scale;
  // A query at position p sees keys j <= p with j > p - window or j < sinks (both up to
  // 2^30); window 0: all keys up to its own (packed and not causal: all).
  int window, sinks;
  // Packed with a window: tk and tv with boxes of 64 x 16 x 1.
  const CUtensorMap *k_cells, *v_cells;
};
int packed_tile_tokens(int group);              // tokens of a 128-row query tile
int packed_blocks(int T, int S, int group);     // bound on the two-tile blocks of a call
cudaError_t launch_fwd_packed(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                              const PackedProblem &p, int d, bool f16, int *sched,
                              int *dev_status, int fault_cta, cudaStream_t stream);
// Paged: the most partitions that a context is cut into, and the fp32 workspace that
// they need (0 bytes when it is one).
int paged_max_parts(int T, int S, int H, int Hk, int max_blocks, int window = 0, int sinks = 0);
size_t paged_prefill_workspace_bytes(int T, int S, int H, int Hk, int max_blocks, int window = 0,
                                     int sinks = 0);
cudaError_t launch_paged_prefill(const CUtensorMap &tq, const CUtensorMap &tk,
                                 const CUtensorMap &tv, const PackedProblem &p, float *workspace,
                                 int *sched, int *dev_status, int fault_cta,
                                 cudaStream_t stream);

// Paged, with groups of sequences that share a prefix: P groups, cu_groups [P + 1] over
// the sequences, prefix_lens [P].  The workspace's parts are bytes from its start.
constexpr int kSharedMaxGroups = 1024, kSharedMaxCtas = 256;   // (an sm_103a GPU has 152 SMs)
struct SharedLayout {
  int split, pre_split;       // most partitions of a context, of a prefix
  size_t rows, sums, rec, seq, first, head, start, bytes;
};
SharedLayout shared_layout(int T, int S, int P, int H, int Hk, int max_blocks);
cudaError_t launch_paged_shared(const CUtensorMap &tq, const CUtensorMap &tk,
                                const CUtensorMap &tv, const PackedProblem &p,
                                const int *cu_groups, const int *prefix_lens, int P,
                                char *workspace, int *sched, int *dev_status, int fault_cta,
                                cudaStream_t stream);

// Gradients of the packed forward (bwd_packed.cu).  Workspace, in floats from
// its start: the dQ accumulator [H][n_blocks * 128][d], those of dK and dV
// [Hk][..][d] (where several items add to them), [-LSE2 | -D] per head and block,
// the block table (`entries` of 4; with a window, of 2 more, then the three counts, and for
// each block whether its dK and dV are stored, not added up).
struct PackedGradLayout {
  int n_blocks, split;        // split: see BwdWindow
  long long entries;
  bool shared;                // there are dK and dV accumulators
  size_t dk_acc, dv_acc, vecs, table, range, count, stored, bytes;
};
PackedGradLayout packed_grad_layout(int T, int S, int H, int Hk, int d, int window = 0,
                                    int sinks = 0);
// q, dout: maps {d, T, H} with boxes of 64 x bwd_qdo_box_rows(d) x 1; k, v
// {d, T, Hk}, 64 x 128 x 1; the accumulators' fp32 maps as for launch_bwd_bf16.
struct PackedGradMaps {
  CUtensorMap q, k, v, dout, dq_acc, dk_acc, dv_acc;
};
struct PackedGrad {
  const void *o, *dout;
  const float *lse;
  void *dq, *dk, *dv;
  const int *cu_seqlens;
  int S, T, H, Hk, d, causal;
  float scale;
  int window, sinks;          // as in PackedProblem
};
cudaError_t launch_bwd_packed(const PackedGradMaps &m, const PackedGrad &p, float *ws, int *sched,
                              int *dev_status, int fault_cta, cudaStream_t stream);

}  // namespace fattn
