// api.cu -- the C ABI of libfattn (declared in include/fattn.h): argument
// validation, TMA tensor-map encoding, the per-device state the library
// owns, and kernel launches.  Every public function returns a status code;
// nothing here aborts or asserts.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <atomic>
#include <cstring>
#include <mutex>

#include "fattn.h"
#include "kernels.h"

namespace {

using fattn::launch_fwd_bf16;

constexpr int kMaxDevices = 64;

struct DeviceState {
  int *status = nullptr;          // device-side latched status word
  float *decode_ws = nullptr;     // split-K partials
  size_t decode_ws_bytes = 0;
  int *decode_counters = nullptr; // one int per (sequence, head), kept at zero
  size_t decode_counter_bytes = 0;
  int *fwd_sched = nullptr;       // 2 * kFwdSchedSlots pairs of work counters, kept at zero
  unsigned fwd_sched_next = 0;    // slot for the next eager launch
  unsigned fwd_sched_next_captured = 0;  // slot for the next launch captured into a graph
  void *mask_ws = nullptr;        // tile summary of the last mask (fa_forward_masked)
  size_t mask_ws_bytes = 0;
  CUtensorMap kv_map_k, kv_map_v; // last TMA views of paged caches (grouped decode)
  const void *kv_maps_k = nullptr, *kv_maps_v = nullptr;
  int kv_maps_hk = 0;
  bool kv_maps_valid = false;
  int inject_fault = 0;           // fa_debug_inject_fault: 1 next forward, 2 next backward
  int checked = 0;                // 1: sm_103 verified, -1: unsupported
};

std::mutex g_mu;
DeviceState g_dev[kMaxDevices];
std::atomic<int> g_decode_gqa_impl{0};   // fa_decode_gqa_select: 0 auto, 1 CUDA cores, 2 tensor cores

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn g_encode = nullptr;

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// n zeroed ints that any stream may use at once: the first call on a device may be
// one that is being captured into a graph, or on a stream that does not wait for
// the legacy one, so they are cleared on a stream of their own, outside of any
// capture, before this returns.
int alloc_zeroed(int **p, size_t n) {
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  if (cudaThreadExchangeStreamCaptureMode(&mode) != cudaSuccess) return FA_ERR_CUDA;
  int rc = FA_ERR_CUDA;
  int *mem = nullptr;
  cudaStream_t s = nullptr;
  if (cudaMalloc(&mem, n * sizeof(int)) != cudaSuccess) {
    mem = nullptr;
    rc = FA_ERR_NO_MEMORY;
  } else if (cudaStreamCreateWithFlags(&s, cudaStreamNonBlocking) == cudaSuccess) {
    if (cudaMemsetAsync(mem, 0, n * sizeof(int), s) == cudaSuccess &&
        cudaStreamSynchronize(s) == cudaSuccess)
      rc = FA_OK;
    cudaStreamDestroy(s);
  }
  cudaThreadExchangeStreamCaptureMode(&mode);
  if (rc == FA_OK)
    *p = mem;
  else if (mem != nullptr)
    cudaFree(mem);
  return rc;
}

// Resolves the current device and makes sure its state exists.
int current_device(int *dev_out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FA_ERR_NO_DEVICE;
  if (dev < 0 || dev >= kMaxDevices) return FA_ERR_NO_DEVICE;
  DeviceState &st = g_dev[dev];
  if (st.checked == 0) {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
      return FA_ERR_NO_DEVICE;
    st.checked = (major == 10 && minor == 3) ? 1 : -1;
  }
  if (st.checked < 0) return FA_ERR_NO_DEVICE;
  int rc;
  if (st.status == nullptr && (rc = alloc_zeroed(&st.status, 1)) != FA_OK) return rc;
  if (st.fwd_sched == nullptr &&
      (rc = alloc_zeroed(&st.fwd_sched, 2 * 2 * fattn::kFwdSchedSlots)) != FA_OK)
    return rc;
  *dev_out = dev;
  return FA_OK;
}

int get_encoder() {
  if (g_encode) return FA_OK;
  void *fn = nullptr;
  cudaDriverEntryPointQueryResult q{};
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                       &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess || fn == nullptr)
    return FA_ERR_CUDA;
  g_encode = reinterpret_cast<EncodeTiledFn>(fn);
  return FA_OK;
}

// 3-D bf16 view {d, N, BH} of a [BH, N, d] tensor; boxes of 64 x box_rows x 1
// (one 128-byte row segment per box row) with the 128-byte swizzle.  Rows
// past N read as zero.
int encode_qkv_map(CUtensorMap *m, const void *base, int BH, int N, int d, int box_rows = 128,
                   CUtensorMapDataType dtype = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16) {
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)N, (cuuint64_t)BH};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)N * d * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = g_encode(m, dtype, 3, const_cast<void *>(base), dims,
                              strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FA_OK : FA_ERR_CUDA;
}

// 3-D E4M3 view {inner, rows, BH} of a [BH, rows, inner] byte tensor (inner
// = 128 codes of a row of Q or K, or Npad keys of a row of V^T), boxes of
// 128 x 128 x 1 with the 128-byte swizzle.  Reads past the extents give zero.
int encode_e4m3_map(CUtensorMap *m, const void *base, int BH, int rows, int inner) {
  const cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)rows, (cuuint64_t)BH};
  const cuuint64_t strides[2] = {(cuuint64_t)inner, (cuuint64_t)rows * inner};
  const cuuint32_t box[3] = {128, 128, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(base), dims,
                              strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FA_OK : FA_ERR_CUDA;
}

// TMA views of the paged caches for the tensor-core grouped decode.  K cache
// [blocks][Hk][16 d-groups][16 tokens][8]: 5-D dims (8 tokens x 8 values,
// token half, d-group, head, block), boxes of 64 x 1 x 16 (one token half's
// 16 d-groups: 2 KB of no-swizzle core matrices, in 128-byte rows).  V cache
// [blocks][Hk][128 d][16 tokens]: 4-D dims (token, d, head, block), boxes of
// 16 x 128 (a block's V^T, 4 KB) written with the 32-byte swizzle.  The block
// extent is the largest int block id: which blocks are read comes from the
// block tables, as in the plain decode.
// (fa_paged_prefill knows the cache's block count and passes it: ids outside
// the cache then read as zeros.  Its K view is one whole block a box, 4 KB:
// d-groups before token halves, so that the halves' matrices land 2 KB apart
// as two boxes of the decode's view do.)
int encode_paged_kv_maps(CUtensorMap *tk, CUtensorMap *tv, const void *k_cache,
                         const void *v_cache, int num_kv_heads, int num_blocks = 0x7fffffff,
                         bool whole_blocks = false) {
  const cuuint64_t nb = (cuuint64_t)num_blocks, hk = (cuuint64_t)num_kv_heads;
  const cuuint64_t half_first[5] = {64, 2, 16, hk, nb}, half_last[5] = {64, 16, 2, hk, nb};
  const cuuint64_t half_first_s[4] = {128, 256, 4096, 4096 * hk};
  const cuuint64_t half_last_s[4] = {256, 128, 4096, 4096 * hk};
  const cuuint32_t half_box[5] = {64, 1, 16, 1, 1}, block_box[5] = {64, 16, 2, 1, 1};
  const cuuint64_t *kd = whole_blocks ? half_last : half_first;
  const cuuint64_t *ks = whole_blocks ? half_last_s : half_first_s;
  const cuuint32_t *kb = whole_blocks ? block_box : half_box;
  const cuuint64_t vd[4] = {16, 128, hk, nb};
  const cuuint64_t vs[3] = {32, 4096, 4096 * hk};
  const cuuint32_t vb[4] = {16, 128, 1, 1};
  const cuuint32_t es[5] = {1, 1, 1, 1, 1};
  if (g_encode(tk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void *>(k_cache), kd, ks, kb,
               es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return FA_ERR_CUDA;
  if (g_encode(tv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(v_cache), vd, vs, vb,
               es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_32B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return FA_ERR_CUDA;
  return FA_OK;
}

// 3-D 16-bit view of a [T, heads, d] tensor with dense heads whose tokens are
// `stride` elements apart: {d, heads, T} (queries; boxes of 64 x box1 heads x
// box2 tokens) or, with tokens_first, {d, T, heads} (keys and values; boxes of
// 64 x box1 tokens x box2 heads).  128-byte swizzle; tokens past T read as
// zero.
int encode_rows_map(CUtensorMap *m, const void *base, int T, int heads, int d, long long stride,
                    bool tokens_first, int box1, int box2, CUtensorMapDataType dtype) {
  const cuuint64_t n_tok = (cuuint64_t)T, n_head = (cuuint64_t)heads;
  const cuuint64_t s_tok = (cuuint64_t)stride * 2, s_head = (cuuint64_t)d * 2;
  const cuuint64_t dims[3] = {(cuuint64_t)d, tokens_first ? n_tok : n_head,
                              tokens_first ? n_head : n_tok};
  const cuuint64_t strides[2] = {tokens_first ? s_tok : s_head, tokens_first ? s_head : s_tok};
  const cuuint32_t box[3] = {64, (cuuint32_t)box1, (cuuint32_t)box2};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = g_encode(m, dtype, 3, const_cast<void *>(base), dims, strides, box, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FA_OK : FA_ERR_CUDA;
}

// Keys per row of the transposed FP8 V: N rounded up to 16.
long long fp8_vt_stride(int N) { return ((long long)N + 15) / 16 * 16; }

// 3-D fp32 view {d, N, BH} of the backward's row-major dQ accumulator, boxes
// of 32 x 32 x 1 (128-byte rows, 128-byte swizzle) for the TMA reduce-add.
int encode_dq_acc_map(CUtensorMap *m, void *base, int BH, int N, int d) {
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)N, (cuuint64_t)BH};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 4, (cuuint64_t)N * d * 4};
  const cuuint32_t box[3] = {32, 32, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, base, dims, strides, box,
                              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FA_OK : FA_ERR_CUDA;
}

int check_forward_args(const void *q, const void *k, const void *v, const void *o,
                       const void *lse, int B, int H, int N, int d, float scale,
                       bool allow_d256 = false) {
  if (!q || !k || !v || !o) return FA_ERR_INVALID_ARG;
  if (B < 0 || H < 0 || N < 0) return FA_ERR_INVALID_ARG;
  if (!(std::isfinite(scale) && scale > 0.f)) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128 && !(allow_d256 && d == 256)) return FA_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
    return FA_ERR_ALIGNMENT;
  // Grid and tensor-map limits: B*H and the tile count index 32-bit grids.
  const long long BH = (long long)B * H;
  if (BH > 0x7fffffffLL / 2 || (long long)N > 0x7fffffffLL / 2) return FA_ERR_UNSUPPORTED;
  if (BH * ((N + 127) / 128) > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// Grows a library-owned buffer to at least `bytes`, in stream order on `s`:
// the old buffer is released with cudaFreeAsync and the new one taken with
// cudaMallocAsync, so growing never synchronises the device.  Earlier calls
// that used the old buffer are ordered before this one (the header's rule for
// calls that share library state), so the release cannot overtake them.
// During stream capture nothing may be allocated: a buffer that is too small
// then gives FA_ERR_UNSUPPORTED.  With `zero`, the new buffer is cleared on
// `s`.
int grow_on_stream(void **buf, size_t *have, size_t bytes, cudaStream_t s, bool zero) {
  if (*have >= bytes) return FA_OK;
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(s, &cs) != cudaSuccess) {
    cudaGetLastError();  // the legacy stream while another stream captures: consume the error
    return FA_ERR_UNSUPPORTED;
  }
  if (cs != cudaStreamCaptureStatusNone) return FA_ERR_UNSUPPORTED;
  if (*buf != nullptr && cudaFreeAsync(*buf, s) != cudaSuccess) return FA_ERR_CUDA;
  *buf = nullptr;
  *have = 0;
  void *p = nullptr;
  if (cudaMallocAsync(&p, bytes, s) != cudaSuccess) return FA_ERR_NO_MEMORY;
  if (zero && cudaMemsetAsync(p, 0, bytes, s) != cudaSuccess) {
    cudaFreeAsync(p, s);
    return FA_ERR_CUDA;
  }
  *buf = p;
  *have = bytes;
  return FA_OK;
}

// Checks shared by the decode entry points; grows the library-owned split-K
// workspace and counters for (num_seqs, num_heads, max_num_blocks_per_seq)
// on the call's stream.
int decode_prepare(const void *q, const void *k_cache, const void *v_cache,
                   const int *block_tables, const int *context_lens, const void *out,
                   int num_seqs, int num_heads, int head_size, int block_size,
                   int max_num_blocks_per_seq, float scale, cudaStream_t stream, float **ws,
                   int **counters, int **status) {
  if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !out)
    return FA_ERR_INVALID_ARG;
  if (num_seqs < 0 || num_heads <= 0 || max_num_blocks_per_seq <= 0) return FA_ERR_INVALID_ARG;
  if (!(std::isfinite(scale) && scale > 0.f)) return FA_ERR_INVALID_ARG;
  if (head_size != fattn::kDecodeHeadSize || block_size != fattn::kDecodeBlockSize)
    return FA_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out))
    return FA_ERR_ALIGNMENT;
  if (num_heads > 65535 || num_seqs > 65535) return FA_ERR_UNSUPPORTED;
  if (num_seqs == 0) return FA_OK;
  const int max_parts = fattn::decode_max_parts(max_num_blocks_per_seq);
  const size_t ws_bytes = fattn::decode_workspace_bytes(num_seqs, num_heads, max_parts);
  const size_t n_counters = (size_t)num_seqs * num_heads;
  std::lock_guard<std::mutex> lock(g_mu);
  int dev = 0, rc;
  if ((rc = current_device(&dev)) != FA_OK) return rc;
  DeviceState &st = g_dev[dev];
  if ((rc = grow_on_stream(reinterpret_cast<void **>(&st.decode_ws), &st.decode_ws_bytes,
                           ws_bytes, stream, false)) != FA_OK)
    return rc;
  if ((rc = grow_on_stream(reinterpret_cast<void **>(&st.decode_counters),
                           &st.decode_counter_bytes, n_counters * sizeof(int), stream, true)) !=
      FA_OK)
    return rc;
  *ws = st.decode_ws;
  *counters = st.decode_counters;
  *status = st.status;
  return FA_OK;
}

int cuda_status(cudaError_t e) { return e == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

// The work-counter pair of a persistent-kernel launch.  Eager launches take
// the first kFwdSchedSlots pairs round robin, so concurrent calls share one
// only with the kFwdSchedSlots-th call after them.  A launch captured into a CUDA graph
// keeps its pair for every replay: it takes one of the other kFwdSchedSlots
// pairs, never handed to an eager launch, shared only with the kFwdSchedSlots-th
// captured launch after it: graphs of whole networks, some hundred launches each,
// may be replayed at the same time.  (One graph must not run concurrently with
// itself.)
int *sched_slot(DeviceState &st, cudaStream_t s) {
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  bool captured = false;
  if (cudaStreamIsCapturing(s, &cs) != cudaSuccess)
    cudaGetLastError();  // the legacy stream while another stream captures: not captured
  else
    captured = cs != cudaStreamCaptureStatusNone;
  const unsigned slot = captured
                            ? fattn::kFwdSchedSlots + st.fwd_sched_next_captured++ % fattn::kFwdSchedSlots
                            : st.fwd_sched_next++ % fattn::kFwdSchedSlots;
  return st.fwd_sched + 2 * slot;
}

}  // namespace

extern "C" {

int fa_version(void) { return 10000; }

const char *fa_status_string(int status) {
  switch (status) {
    case FA_OK: return "ok";
    case FA_ERR_INVALID_ARG: return "invalid argument";
    case FA_ERR_UNSUPPORTED: return "unsupported size";
    case FA_ERR_ALIGNMENT: return "pointer not 16-byte aligned";
    case FA_ERR_CUDA: return "CUDA error";
    case FA_ERR_TIMEOUT: return "device-side wait timed out";
    case FA_ERR_NO_MEMORY: return "out of device memory";
    case FA_ERR_NO_DEVICE: return "no usable sm_103 device";
    default: return "unknown status";
  }
}

namespace {
// fa_forward, fa_forward_f16 and fa_forward_masked: the tensor-core forward
// for 16-bit inputs.
int forward16(const void *q, const void *k, const void *v, void *o, float *lse, int B, int H,
              int N, int d, float scale, int causal, fa_stream_t stream, bool f16,
              const uint8_t *mask = nullptr, long long mask_bh_stride = 0) {
  int rc = check_forward_args(q, k, v, o, lse, B, H, N, d, scale, mask == nullptr);
  if (rc != FA_OK) return rc;
  const int BH = B * H;
  if (BH == 0 || N == 0) return FA_OK;
  int dev = 0, fault_cta = -1;
  int *sched = nullptr;
  void *mask_ws = nullptr;
  const int mask_heads = mask_bh_stride != 0 ? BH : 1;
  if (mask != nullptr && (mask_heads > 65535 || (N + 127) / 128 > 65535)) return FA_ERR_UNSUPPORTED;
  CUtensorMap tq, tk, tv;
  {
    std::lock_guard<std::mutex> lock(g_mu);
    if ((rc = current_device(&dev)) != FA_OK) return rc;
    if ((rc = get_encoder()) != FA_OK) return rc;
    DeviceState &st = g_dev[dev];
    sched = sched_slot(st, reinterpret_cast<cudaStream_t>(stream));
    fault_cta = st.inject_fault == 1 ? 0 : -1;
    if (st.inject_fault == 1) st.inject_fault = 0;
    if (mask != nullptr) {
      const size_t need = fattn::mask_summary_bytes(mask_heads, N);
      if ((rc = grow_on_stream(&st.mask_ws, &st.mask_ws_bytes, need,
                               reinterpret_cast<cudaStream_t>(stream), false)) != FA_OK)
        return rc;
      mask_ws = st.mask_ws;
    }
  }
  const CUtensorMapDataType dt =
      f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  if ((rc = encode_qkv_map(&tq, q, BH, N, d, 128, dt)) != FA_OK) return rc;
  if ((rc = encode_qkv_map(&tk, k, BH, N, d, 128, dt)) != FA_OK) return rc;
  if (d == 256) {
    // One 128-row query tile per CTA; V arrives in 64-key halves.
    if ((rc = encode_qkv_map(&tv, v, BH, N, d, 64, dt)) != FA_OK) return rc;
    return cuda_status(fattn::launch_fwd_d256(tq, tk, tv, o, lse, BH, N, scale, causal ? 1 : 0,
                                              sched, g_dev[dev].status,
                                              reinterpret_cast<cudaStream_t>(stream), f16));
  }
  if ((rc = encode_qkv_map(&tv, v, BH, N, d, 128, dt)) != FA_OK) return rc;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint8_t *flags = nullptr;
  const int2 *ranges = nullptr;
  const uint4 *bits = nullptr;
  if (mask != nullptr &&
      (rc = cuda_status(fattn::launch_mask_summary(mask, static_cast<int64_t>(mask_bh_stride), N,
                                                   mask_heads, mask_ws, &flags, &ranges, &bits,
                                                   s))) != FA_OK)
    return rc;
  return cuda_status(launch_fwd_bf16(tq, tk, tv, o, lse, BH, N, d, scale, causal ? 1 : 0, sched,
                                     g_dev[dev].status, fault_cta, s, f16, mask,
                                     static_cast<int64_t>(mask_bh_stride), ranges, flags, bits));
}
}  // namespace

int fa_forward(const void *q, const void *k, const void *v, void *o, float *lse, int B, int H,
               int N, int d, float scale, int causal, fa_stream_t stream) {
  return forward16(q, k, v, o, lse, B, H, N, d, scale, causal, stream, false);
}

int fa_forward_f16(const void *q, const void *k, const void *v, void *o, float *lse, int B,
                   int H, int N, int d, float scale, int causal, fa_stream_t stream) {
  return forward16(q, k, v, o, lse, B, H, N, d, scale, causal, stream, true);
}

int fa_forward_masked(const void *q, const void *k, const void *v, void *o, float *lse,
                      const void *mask, long long mask_bh_stride, int B, int H, int N, int d,
                      float scale, fa_stream_t stream) {
  if (!mask || mask_bh_stride < 0) return FA_ERR_INVALID_ARG;
  if (!aligned16(mask) || mask_bh_stride % 16 != 0) return FA_ERR_ALIGNMENT;
  if (N % 16 != 0) return FA_ERR_UNSUPPORTED;
  return forward16(q, k, v, o, lse, B, H, N, d, scale, 0, stream, false,
                   static_cast<const uint8_t *>(mask), mask_bh_stride);
}

int fa_forward_fp32(const float *q, const float *k, const float *v, float *o, float *lse, int B,
                    int H, int N, int d, float scale, int causal, fa_stream_t stream) {
  int rc = check_forward_args(q, k, v, o, lse, B, H, N, d, scale);
  if (rc != FA_OK) return rc;
  const int BH = B * H;
  if (BH == 0 || N == 0) return FA_OK;
  if (BH > 0x7fffffff || (N + 31) / 32 > 65535) return FA_ERR_UNSUPPORTED;
  int dev = 0;
  {
    std::lock_guard<std::mutex> lock(g_mu);
    if ((rc = current_device(&dev)) != FA_OK) return rc;
  }
  return cuda_status(fattn::launch_fwd_f32(q, k, v, o, lse, BH, N, d, scale, causal ? 1 : 0,
                                           reinterpret_cast<cudaStream_t>(stream)));
}

unsigned long long fa_quantize_fp8_workspace_bytes(int B, int H, int N, int d) {
  if (B < 0 || H < 0 || N < 0 || d < 0) return 0;
  return static_cast<unsigned long long>(
      fattn::fp8_quant_workspace_bytes(static_cast<int>((long long)B * H), N));
}

long long fa_fp8_vt_stride(int N) { return N < 0 ? 0 : fp8_vt_stride(N); }

int fa_quantize_fp8(const void *q, const void *k, const void *v, const float *signs, void *q8,
                    void *k8, void *vt8, float *q_scale, float *k_scale, float *v_scale, int B,
                    int H, int N, int d, void *workspace, unsigned long long workspace_bytes,
                    fa_stream_t stream) {
  if (!q || !k || !v || !q8 || !k8 || !vt8 || !q_scale || !k_scale || !v_scale)
    return FA_ERR_INVALID_ARG;
  if (B < 0 || H < 0 || N < 0) return FA_ERR_INVALID_ARG;
  if (d != 128) return FA_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q8) || !aligned16(k8) ||
      !aligned16(vt8) || (signs && !aligned16(signs)))
    return FA_ERR_ALIGNMENT;
  const long long BH = (long long)B * H;
  if (BH > 65535 || N > (1 << 30)) return FA_ERR_UNSUPPORTED;
  if (BH == 0 || N == 0) return FA_OK;
  if (!workspace) return FA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(workspace) % 4 != 0) return FA_ERR_ALIGNMENT;
  if (workspace_bytes < fattn::fp8_quant_workspace_bytes((int)BH, N)) return FA_ERR_INVALID_ARG;
  int dev = 0, rc;
  {
    std::lock_guard<std::mutex> lock(g_mu);
    if ((rc = current_device(&dev)) != FA_OK) return rc;
  }
  // The transform's 1/sqrt(d), rounded once to fp32, multiplies the scales.
  const float rot_factor = static_cast<float>(1.0 / std::sqrt(static_cast<double>(d)));
  return cuda_status(fattn::launch_fp8_quantize(
      q, k, v, signs, q8, k8, vt8, q_scale, k_scale, v_scale, static_cast<float *>(workspace),
      (int)BH, N, (int)fp8_vt_stride(N), rot_factor, g_dev[dev].status,
      reinterpret_cast<cudaStream_t>(stream)));
}

int fa_forward_fp8(const void *q8, const void *k8, const void *vt8, const float *q_scale,
                   const float *k_scale, const float *v_scale, void *o, float *lse, int B, int H,
                   int N, int d, float scale, int causal, fa_stream_t stream) {
  if (!q_scale || !k_scale || !v_scale) return FA_ERR_INVALID_ARG;
  int rc = check_forward_args(q8, k8, vt8, o, lse, B, H, N, d, scale);
  if (rc != FA_OK) return rc;
  if (d != 128) return FA_ERR_UNSUPPORTED;
  const int BH = B * H;
  if (BH == 0 || N == 0) return FA_OK;
  int dev = 0, fault_cta = -1;
  int *sched = nullptr;
  CUtensorMap tq, tk, tvt;
  {
    std::lock_guard<std::mutex> lock(g_mu);
    if ((rc = current_device(&dev)) != FA_OK) return rc;
    if ((rc = get_encoder()) != FA_OK) return rc;
    DeviceState &st = g_dev[dev];
    sched = sched_slot(st, reinterpret_cast<cudaStream_t>(stream));
    fault_cta = st.inject_fault == 1 ? 0 : -1;
    if (st.inject_fault == 1) st.inject_fault = 0;
  }
  if ((rc = encode_e4m3_map(&tq, q8, BH, N, d)) != FA_OK) return rc;
  if ((rc = encode_e4m3_map(&tk, k8, BH, N, d)) != FA_OK) return rc;
  if ((rc = encode_e4m3_map(&tvt, vt8, BH, d, (int)fp8_vt_stride(N))) != FA_OK) return rc;
  return cuda_status(fattn::launch_fwd_fp8(tq, tk, tvt, q_scale, k_scale, v_scale, o, lse, BH, N,
                                           scale, causal ? 1 : 0, sched, g_dev[dev].status,
                                           fault_cta, reinterpret_cast<cudaStream_t>(stream)));
}

unsigned long long fa_backward_workspace_bytes(int B, int H, int N, int d) {
  if (B < 0 || H < 0 || N < 0 || d < 0) return 0;
  return static_cast<unsigned long long>(
      fattn::bwd_workspace_bytes(static_cast<int>((long long)B * H), N, d));
}

int fa_backward(const void *q, const void *k, const void *v, const void *o, const void *dout,
                const float *lse, void *dq, void *dk, void *dv, int B, int H, int N, int d,
                float scale, int causal, void *workspace, unsigned long long workspace_bytes,
                fa_stream_t stream) {
  if (!dout || !lse || !dq || !dk || !dv) return FA_ERR_INVALID_ARG;
  int rc = check_forward_args(q, k, v, o, lse, B, H, N, d, scale);
  if (rc != FA_OK) return rc;
  if (!aligned16(dout) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv))
    return FA_ERR_ALIGNMENT;
  const int BH = B * H;
  if (BH == 0 || N == 0) return FA_OK;
  if (!workspace) return FA_ERR_INVALID_ARG;
  if (!aligned16(workspace)) return FA_ERR_ALIGNMENT;
  if (workspace_bytes < fattn::bwd_workspace_bytes(BH, N, d)) return FA_ERR_INVALID_ARG;
  // The preparation kernel runs 16 padded rows per block of its 1-D grid.
  if ((long long)BH * ((N + 127) / 128) * 8 > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  int dev = 0, fault_cta = -1;
  int *sched = nullptr;
  CUtensorMap tq, tk, tv, tdo, tdq;
  {
    std::lock_guard<std::mutex> lock(g_mu);
    if ((rc = current_device(&dev)) != FA_OK) return rc;
    if ((rc = get_encoder()) != FA_OK) return rc;
    sched = sched_slot(g_dev[dev], reinterpret_cast<cudaStream_t>(stream));
    if (g_dev[dev].inject_fault == 2) {
      fault_cta = 0;
      g_dev[dev].inject_fault = 0;
    }
  }
  const int qdo_rows = fattn::bwd_qdo_box_rows(d);
  if ((rc = encode_qkv_map(&tq, q, BH, N, d, qdo_rows)) != FA_OK) return rc;
  if ((rc = encode_qkv_map(&tk, k, BH, N, d)) != FA_OK) return rc;
  if ((rc = encode_qkv_map(&tv, v, BH, N, d)) != FA_OK) return rc;
  if ((rc = encode_qkv_map(&tdo, dout, BH, N, d, qdo_rows)) != FA_OK) return rc;
  if ((rc = encode_dq_acc_map(&tdq, workspace, BH, N, d)) != FA_OK) return rc;
  return cuda_status(fattn::launch_bwd_bf16(tq, tk, tv, tdo, tdq, o, dout, lse, dq, dk, dv, BH,
                                            N, d,
                                            scale, causal ? 1 : 0,
                                            reinterpret_cast<float *>(workspace), sched,
                                            fault_cta, g_dev[dev].status,
                                            reinterpret_cast<cudaStream_t>(stream)));
}

int fa_paged_decode(const void *q, const void *k_cache, const void *v_cache,
                    const int *block_tables, const int *context_lens, void *out, int num_seqs,
                    int num_heads, int head_size, int block_size, int max_num_blocks_per_seq,
                    float scale, fa_stream_t stream) {
  float *ws = nullptr;
  int *counters = nullptr, *status = nullptr;
  const int rc = decode_prepare(q, k_cache, v_cache, block_tables, context_lens, out, num_seqs,
                                num_heads, head_size, block_size, max_num_blocks_per_seq, scale,
                                reinterpret_cast<cudaStream_t>(stream), &ws, &counters, &status);
  if (rc != FA_OK || num_seqs == 0) return rc;
  return cuda_status(fattn::launch_paged_decode(q, k_cache, v_cache, block_tables, context_lens,
                                                out, num_seqs, num_heads, max_num_blocks_per_seq,
                                                scale, ws, counters,
                                                reinterpret_cast<cudaStream_t>(stream)));
}

int fa_paged_decode_gqa(const void *q, const void *k_cache, const void *v_cache,
                        const int *block_tables, const int *context_lens, void *out,
                        int num_seqs, int num_heads, int num_kv_heads, int head_size,
                        int block_size, int max_num_blocks_per_seq, float scale,
                        fa_stream_t stream) {
  if (num_kv_heads <= 0 || num_heads <= 0 || num_heads % num_kv_heads != 0)
    return FA_ERR_INVALID_ARG;
  const int group = num_heads / num_kv_heads;
  const int impl = g_decode_gqa_impl.load();
  const bool cc_ok = fattn::decode_gqa_group_supported(group);
  const bool tc_ok = fattn::decode_gqa_tc_supported(group);
  // Automatic: the tensor-core kernel from group 3 up once there is at least
  // a unit (sequence, partition, cached head) per SM; measured faster there,
  // and slower for group 2 and for a handful of units.
  const long long units_bound = (long long)num_seqs * num_kv_heads *
                                fattn::decode_max_parts(max_num_blocks_per_seq);
  const bool tc_auto = tc_ok && (!cc_ok || (group >= 3 && units_bound >= fattn::kDecodeTcMinUnits));
  const bool tc = group > 1 && (impl == 2 ? tc_ok : impl == 0 ? tc_auto : false);
  if (group > 1 && !tc && (impl == 2 || !cc_ok)) return FA_ERR_UNSUPPORTED;
  float *ws = nullptr;
  int *counters = nullptr, *status = nullptr;
  const int rc = decode_prepare(q, k_cache, v_cache, block_tables, context_lens, out, num_seqs,
                                num_heads, head_size, block_size, max_num_blocks_per_seq, scale,
                                reinterpret_cast<cudaStream_t>(stream), &ws, &counters, &status);
  if (rc != FA_OK || num_seqs == 0) return rc;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (group == 1)
    return cuda_status(fattn::launch_paged_decode(q, k_cache, v_cache, block_tables,
                                                  context_lens, out, num_seqs, num_heads,
                                                  max_num_blocks_per_seq, scale, ws, counters, s));
  if (tc) {
    CUtensorMap tk, tv;
    int *sched = nullptr;
    {
      // The views depend only on the caches' addresses and head count: the
      // last pair encoded on the device is reused while those stay the same.
      std::lock_guard<std::mutex> lock(g_mu);
      int dev = 0, rc2;
      if ((rc2 = current_device(&dev)) != FA_OK) return rc2;
      if ((rc2 = get_encoder()) != FA_OK) return rc2;
      DeviceState &st = g_dev[dev];
      sched = sched_slot(st, reinterpret_cast<cudaStream_t>(stream));
      if (!(st.kv_maps_valid && st.kv_maps_k == k_cache && st.kv_maps_v == v_cache &&
            st.kv_maps_hk == num_kv_heads)) {
        st.kv_maps_valid = false;
        if ((rc2 = encode_paged_kv_maps(&st.kv_map_k, &st.kv_map_v, k_cache, v_cache,
                                        num_kv_heads)) != FA_OK)
          return rc2;
        st.kv_maps_k = k_cache;
        st.kv_maps_v = v_cache;
        st.kv_maps_hk = num_kv_heads;
        st.kv_maps_valid = true;
      }
      tk = st.kv_map_k;
      tv = st.kv_map_v;
    }
    return cuda_status(fattn::launch_paged_decode_gqa_tc(
        tk, tv, q, block_tables, context_lens, out, num_seqs, num_heads, num_kv_heads,
        max_num_blocks_per_seq, scale, ws, sched, status, s));
  }
  return cuda_status(fattn::launch_paged_decode_gqa(q, k_cache, v_cache, block_tables,
                                                    context_lens, out, num_seqs, num_heads,
                                                    num_kv_heads, max_num_blocks_per_seq, scale,
                                                    ws, counters, status, s));
}

namespace {
using fattn::ElemType;

size_t elem_bytes(ElemType t) { return t == ElemType::kF32 ? 4 : 2; }

bool aligned_to(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// A token stride (elements) of a [tokens, heads, d] tensor with dense heads:
// it covers the heads and keeps every row 16-byte aligned.
int check_token_stride(long long stride, int heads, int d, size_t es) {
  if (stride < (long long)heads * d) return FA_ERR_INVALID_ARG;
  return (unsigned long long)stride * es % 16 == 0 ? FA_OK : FA_ERR_ALIGNMENT;
}

// Checks shared by the norm-and-rotation calls.
int check_qk_prep(const fattn::QkPrep &p, ElemType type) {
  if (!p.q || !p.k || !p.positions) return FA_ERR_INVALID_ARG;
  if (p.T < 0 || p.H <= 0 || p.Hk <= 0) return FA_ERR_INVALID_ARG;
  if (!(std::isfinite(p.eps) && p.eps >= 0.f) || !std::isfinite(p.mscale)) return FA_ERR_INVALID_ARG;
  if (p.d != 64 && p.d != 128 && p.d != 256) return FA_ERR_UNSUPPORTED;
  if (p.rot < 0 || p.rot > p.d) return FA_ERR_INVALID_ARG;
  if (p.rot % 16 != 0) return FA_ERR_UNSUPPORTED;
  if (p.rot > 0 && !p.inv_freq) return FA_ERR_INVALID_ARG;
  if (p.H > 65535 || p.Hk > 65535) return FA_ERR_UNSUPPORTED;
  if (!aligned16(p.q) || !aligned16(p.k) || !aligned16(p.q_weight) || !aligned16(p.k_weight) ||
      !aligned_to(p.positions, 4) || !aligned_to(p.inv_freq, 8))
    return FA_ERR_ALIGNMENT;
  int rc;
  if ((rc = check_token_stride(p.q_stride, p.H, p.d, elem_bytes(type))) != FA_OK) return rc;
  if ((rc = check_token_stride(p.k_stride, p.Hk, p.d, elem_bytes(type))) != FA_OK) return rc;
  return FA_OK;
}

// Makes sure that the current device is one the kernels run on.
int require_device() {
  std::lock_guard<std::mutex> lock(g_mu);
  int dev = 0;
  return current_device(&dev);
}

int qk_norm_rope(ElemType type, const fattn::QkPrep &p, void *q_out, void *k_out,
                 fa_stream_t stream) {
  int rc = check_qk_prep(p, type);
  if (rc != FA_OK) return rc;
  if (!q_out || !k_out) return FA_ERR_INVALID_ARG;
  if (!aligned16(q_out) || !aligned16(k_out)) return FA_ERR_ALIGNMENT;
  if (p.T == 0) return FA_OK;
  if ((rc = require_device()) != FA_OK) return rc;
  return cuda_status(
      fattn::launch_qk_prep(type, p, q_out, k_out, reinterpret_cast<cudaStream_t>(stream)));
}

int qk_norm_rope_backward(ElemType type, const fattn::QkPrep &p, const void *dq_out,
                          const void *dk_out, void *dq, void *dk, float *dqw, float *dkw,
                          void *workspace, unsigned long long workspace_bytes,
                          fa_stream_t stream) {
  int rc = check_qk_prep(p, type);
  if (rc != FA_OK) return rc;
  if (!dq_out || !dk_out || !dq || !dk) return FA_ERR_INVALID_ARG;
  if ((dqw != nullptr) != (p.q_weight != nullptr) || (dkw != nullptr) != (p.k_weight != nullptr))
    return FA_ERR_INVALID_ARG;
  if (!aligned16(dq_out) || !aligned16(dk_out) || !aligned16(dq) || !aligned16(dk) ||
      !aligned_to(dqw, 4) || !aligned_to(dkw, 4))
    return FA_ERR_ALIGNMENT;
  const bool weights = dqw != nullptr || dkw != nullptr;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (p.T == 0 && !weights) return FA_OK;
  if (p.T > 0 && weights) {
    if (!workspace) return FA_ERR_INVALID_ARG;
    if (!aligned16(workspace)) return FA_ERR_ALIGNMENT;
    if (workspace_bytes < fattn::qk_prep_grad_workspace_bytes(p.T, p.d)) return FA_ERR_INVALID_ARG;
  }
  if ((rc = require_device()) != FA_OK) return rc;
  if (p.T == 0) {
    if (dqw && cudaMemsetAsync(dqw, 0, sizeof(float) * p.d, s) != cudaSuccess) return FA_ERR_CUDA;
    if (dkw && cudaMemsetAsync(dkw, 0, sizeof(float) * p.d, s) != cudaSuccess) return FA_ERR_CUDA;
    return FA_OK;
  }
  return cuda_status(fattn::launch_qk_prep_grad(type, p, dq_out, dk_out, dq, dk, dqw, dkw,
                                                static_cast<float *>(workspace), s));
}
}  // namespace

#define FATTN_QK_PREP                                                                            \
  fattn::QkPrep {                                                                                \
    q, k, q_weight, k_weight, positions, inv_freq, num_tokens, num_heads, num_kv_heads, d,       \
        rot_dim, interleaved ? 1 : 0, static_cast<int64_t>(q_stride),                            \
        static_cast<int64_t>(k_stride), eps, mscale                                              \
  }

int fa_qk_norm_rope(const void *q, const void *k, const void *q_weight, const void *k_weight,
                    const int *positions, const double *inv_freq, void *q_out, void *k_out,
                    int num_tokens, int num_heads, int num_kv_heads, int d, int rot_dim,
                    int interleaved, long long q_stride, long long k_stride, float eps,
                    float mscale, fa_stream_t stream) {
  return qk_norm_rope(ElemType::kBf16, FATTN_QK_PREP, q_out, k_out, stream);
}

int fa_qk_norm_rope_f16(const void *q, const void *k, const void *q_weight, const void *k_weight,
                        const int *positions, const double *inv_freq, void *q_out, void *k_out,
                        int num_tokens, int num_heads, int num_kv_heads, int d, int rot_dim,
                        int interleaved, long long q_stride, long long k_stride, float eps,
                        float mscale, fa_stream_t stream) {
  return qk_norm_rope(ElemType::kF16, FATTN_QK_PREP, q_out, k_out, stream);
}

int fa_qk_norm_rope_fp32(const void *q, const void *k, const void *q_weight, const void *k_weight,
                         const int *positions, const double *inv_freq, void *q_out, void *k_out,
                         int num_tokens, int num_heads, int num_kv_heads, int d, int rot_dim,
                         int interleaved, long long q_stride, long long k_stride, float eps,
                         float mscale, fa_stream_t stream) {
  return qk_norm_rope(ElemType::kF32, FATTN_QK_PREP, q_out, k_out, stream);
}

int fa_qk_norm_rope_cache(const void *q, const void *k, const void *v, const void *q_weight,
                          const void *k_weight, const int *positions, const double *inv_freq,
                          const long long *slots, void *q_out, void *k_cache, void *v_cache,
                          int num_tokens, int num_heads, int num_kv_heads, int head_size,
                          int block_size, int num_blocks, int rot_dim, int interleaved,
                          long long q_stride, long long k_stride, long long v_stride, float eps,
                          float mscale, fa_stream_t stream) {
  const int d = head_size;
  const fattn::QkPrep p = FATTN_QK_PREP;
  int rc = check_qk_prep(p, ElemType::kBf16);
  if (rc != FA_OK) return rc;
  if (!v || !slots || !q_out || !k_cache || !v_cache || num_blocks < 0) return FA_ERR_INVALID_ARG;
  if (head_size != fattn::kDecodeHeadSize || block_size != fattn::kDecodeBlockSize)
    return FA_ERR_UNSUPPORTED;
  if (!aligned16(v) || !aligned16(q_out) || !aligned16(k_cache) || !aligned16(v_cache) ||
      !aligned_to(slots, 8))
    return FA_ERR_ALIGNMENT;
  if ((rc = check_token_stride(v_stride, num_kv_heads, d, 2)) != FA_OK) return rc;
  // One block per 16 tokens and cached head, beside those of the queries and keys.
  if (((long long)num_tokens + 15) / 16 * num_kv_heads > 0x3fffffffLL) return FA_ERR_UNSUPPORTED;
  if (num_tokens == 0) return FA_OK;
  if ((rc = require_device()) != FA_OK) return rc;
  return cuda_status(fattn::launch_qk_prep_cache(
      p, v, static_cast<int64_t>(v_stride), slots, (int64_t)num_blocks * block_size, q_out,
      k_cache, v_cache, reinterpret_cast<cudaStream_t>(stream)));
}

unsigned long long fa_qk_norm_rope_backward_workspace_bytes(int num_tokens, int d) {
  if (num_tokens < 0 || d < 0) return 0;
  return static_cast<unsigned long long>(fattn::qk_prep_grad_workspace_bytes(num_tokens, d));
}

#define FATTN_QK_PREP_BACKWARD(NAME, TYPE)                                                       \
  int NAME(const void *dq_out, const void *dk_out, const void *q, const void *k,                 \
           const void *q_weight, const void *k_weight, const int *positions,                     \
           const double *inv_freq, void *dq, void *dk, float *dq_weight, float *dk_weight,       \
           int num_tokens, int num_heads, int num_kv_heads, int d, int rot_dim, int interleaved, \
           long long q_stride, long long k_stride, float eps, float mscale, void *workspace,     \
           unsigned long long workspace_bytes, fa_stream_t stream) {                             \
    return qk_norm_rope_backward(TYPE, FATTN_QK_PREP, dq_out, dk_out, dq, dk, dq_weight,         \
                                 dk_weight, workspace, workspace_bytes, stream);                 \
  }
FATTN_QK_PREP_BACKWARD(fa_qk_norm_rope_backward, ElemType::kBf16)
FATTN_QK_PREP_BACKWARD(fa_qk_norm_rope_backward_f16, ElemType::kF16)
FATTN_QK_PREP_BACKWARD(fa_qk_norm_rope_backward_fp32, ElemType::kF32)
#undef FATTN_QK_PREP_BACKWARD
#undef FATTN_QK_PREP

namespace {
// Sizes that the packed calls share: T tokens of S sequences, H query heads on
// Hk key/value heads.
int check_packed_sizes(int S, int T, int H, int Hk) {
  if (S < 0 || T < 0 || H <= 0 || Hk <= 0 || H % Hk != 0) return FA_ERR_INVALID_ARG;
  // A query tile holds 128 / group tokens; indices of rows and items are 32-bit.
  const int group = H / Hk;
  if (group > 128 || H > 65535 || S > (1 << 26) || T > (1 << 29)) return FA_ERR_UNSUPPORTED;
  if ((long long)T * H > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  if ((long long)fattn::packed_blocks(T, S, group) * Hk > 0x3fffffffLL) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// Checks shared by the packed forward and backward.
int check_packed(const void *q, const void *k, const void *v, const void *o, const void *lse,
                 const int *cu_seqlens, int S, int T, int H, int Hk, int d, long long q_stride,
                 long long k_stride, long long v_stride, float scale) {
  if (!q || !k || !v || !o || !cu_seqlens) return FA_ERR_INVALID_ARG;
  if (!(std::isfinite(scale) && scale > 0.f)) return FA_ERR_INVALID_ARG;
  int rc = check_packed_sizes(S, T, H, Hk);
  if (rc != FA_OK) return rc;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned_to(lse, 4) ||
      !aligned_to(cu_seqlens, 4))
    return FA_ERR_ALIGNMENT;
  if ((rc = check_token_stride(q_stride, H, d, 2)) != FA_OK) return rc;
  if ((rc = check_token_stride(k_stride, Hk, d, 2)) != FA_OK) return rc;
  return check_token_stride(v_stride, Hk, d, 2);
}

// The current device's work counters for one launch, its status word, and the CTA
// that is to lose its copies (0 if fa_debug_inject_fault armed `mode`, else -1).
int acquire_sched(cudaStream_t s, int mode, int **sched, int **status, int *fault_cta) {
  std::lock_guard<std::mutex> lock(g_mu);
  int dev = 0, rc;
  if ((rc = current_device(&dev)) != FA_OK) return rc;
  if ((rc = get_encoder()) != FA_OK) return rc;
  DeviceState &st = g_dev[dev];
  *sched = sched_slot(st, s);
  *status = st.status;
  *fault_cta = st.inject_fault == mode ? 0 : -1;
  if (st.inject_fault == mode) st.inject_fault = 0;
  return FA_OK;
}

// What a query sees: all keys up to its own (`causal`; else all), or of those the last
// `window` and the first `sinks` (window > 0).
struct Visible {
  int causal, window, sinks;
};
constexpr Visible all_keys(int causal) { return {causal ? 1 : 0, 0, 0}; }
// A window and first tokens; lengths past 2^30 see what 2^30 sees (sequences are shorter).
int window_keys(int window, int sinks, Visible *out) {
  if (window <= 0 || sinks < 0) return FA_ERR_INVALID_ARG;
  *out = {1, std::min(window, 1 << 30), std::min(sinks, 1 << 30)};
  return FA_OK;
}

int forward_packed(const void *q, const void *k, const void *v, void *o, float *lse,
                   const int *cu_seqlens, int S, int T, int H, int Hk, int d, long long q_stride,
                   long long k_stride, long long v_stride, float scale, const Visible &see,
                   fa_stream_t stream, bool f16) {
  int rc = check_packed(q, k, v, o, lse, cu_seqlens, S, T, H, Hk, d, q_stride, k_stride, v_stride,
                        scale);
  if (rc != FA_OK) return rc;
  if (S == 0 || T == 0) return FA_OK;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int *sched = nullptr, *status = nullptr, fault_cta = -1;
  if ((rc = acquire_sched(s, 1, &sched, &status, &fault_cta)) != FA_OK) return rc;
  const CUtensorMapDataType dt =
      f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const int group = H / Hk;
  CUtensorMap tq, tk, tv;
  if ((rc = encode_rows_map(&tq, q, T, H, d, q_stride, false, group,
                            fattn::packed_tile_tokens(group), dt)) != FA_OK)
    return rc;
  if ((rc = encode_rows_map(&tk, k, T, Hk, d, k_stride, true, 128, 1, dt)) != FA_OK) return rc;
  if ((rc = encode_rows_map(&tv, v, T, Hk, d, v_stride, true, 128, 1, dt)) != FA_OK) return rc;
  fattn::PackedProblem p{};
  p.o = o, p.lse = lse, p.cu_seqlens = cu_seqlens;
  p.S = S, p.T = T, p.H = H, p.Hk = Hk, p.scale = scale;
  p.causal = see.causal, p.window = see.window, p.sinks = see.sinks;
  CUtensorMap k_cells = tk, v_cells = tv;
  if (see.sinks > 0) {   // (without first tokens a tile has no gap)
    rc = encode_rows_map(&k_cells, k, T, Hk, d, k_stride, true, 16, 1, dt);
    if (rc == FA_OK) rc = encode_rows_map(&v_cells, v, T, Hk, d, v_stride, true, 16, 1, dt);
    if (rc != FA_OK) return rc;
  }
  p.k_cells = &k_cells, p.v_cells = &v_cells;
  return cuda_status(
      fattn::launch_fwd_packed(tq, tk, tv, p, d, f16, sched, status, fault_cta, s));
}
}  // namespace

int fa_forward_packed(const void *q, const void *k, const void *v, void *o, float *lse,
                      const int *cu_seqlens, int num_seqs, int total_tokens, int num_heads,
                      int num_kv_heads, int d, long long q_stride, long long k_stride,
                      long long v_stride, float scale, int causal, fa_stream_t stream) {
  return forward_packed(q, k, v, o, lse, cu_seqlens, num_seqs, total_tokens, num_heads,
                        num_kv_heads, d, q_stride, k_stride, v_stride, scale, all_keys(causal),
                        stream, false);
}

int fa_forward_packed_f16(const void *q, const void *k, const void *v, void *o, float *lse,
                          const int *cu_seqlens, int num_seqs, int total_tokens, int num_heads,
                          int num_kv_heads, int d, long long q_stride, long long k_stride,
                          long long v_stride, float scale, int causal, fa_stream_t stream) {
  return forward_packed(q, k, v, o, lse, cu_seqlens, num_seqs, total_tokens, num_heads,
                        num_kv_heads, d, q_stride, k_stride, v_stride, scale, all_keys(causal),
                        stream, true);
}

int fa_forward_packed_window(const void *q, const void *k, const void *v, void *o, float *lse,
                             const int *cu_seqlens, int num_seqs, int total_tokens,
                             int num_heads, int num_kv_heads, int d, long long q_stride,
                             long long k_stride, long long v_stride, float scale, int window,
                             int sinks, fa_stream_t stream) {
  Visible see;
  const int rc = window_keys(window, sinks, &see);
  if (rc != FA_OK) return rc;
  return forward_packed(q, k, v, o, lse, cu_seqlens, num_seqs, total_tokens, num_heads,
                        num_kv_heads, d, q_stride, k_stride, v_stride, scale, see, stream, false);
}

int fa_forward_packed_window_f16(const void *q, const void *k, const void *v, void *o, float *lse,
                                 const int *cu_seqlens, int num_seqs, int total_tokens,
                                 int num_heads, int num_kv_heads, int d, long long q_stride,
                                 long long k_stride, long long v_stride, float scale, int window,
                                 int sinks, fa_stream_t stream) {
  Visible see;
  const int rc = window_keys(window, sinks, &see);
  if (rc != FA_OK) return rc;
  return forward_packed(q, k, v, o, lse, cu_seqlens, num_seqs, total_tokens, num_heads,
                        num_kv_heads, d, q_stride, k_stride, v_stride, scale, see, stream, true);
}

unsigned long long fa_backward_packed_workspace_bytes(int num_seqs, int total_tokens,
                                                      int num_heads, int num_kv_heads, int d) {
  if (num_seqs <= 0 || total_tokens <= 0 || d <= 0) return 0;
  if (check_packed_sizes(num_seqs, total_tokens, num_heads, num_kv_heads) != FA_OK) return 0;
  return static_cast<unsigned long long>(
      fattn::packed_grad_layout(total_tokens, num_seqs, num_heads, num_kv_heads, d).bytes);
}

namespace {
int backward_packed(const void *q, const void *k, const void *v, const void *o, const void *dout,
                    const float *lse, void *dq, void *dk, void *dv, const int *cu_seqlens,
                    int num_seqs, int total_tokens, int num_heads, int num_kv_heads, int d,
                    long long q_stride, long long k_stride, long long v_stride, float scale,
                    const Visible &see, void *workspace, unsigned long long workspace_bytes,
                    fa_stream_t stream) {
  if (!dout || !lse || !dq || !dk || !dv) return FA_ERR_INVALID_ARG;
  const int S = num_seqs, T = total_tokens, H = num_heads, Hk = num_kv_heads;
  int rc = check_packed(q, k, v, o, lse, cu_seqlens, S, T, H, Hk, d, q_stride, k_stride, v_stride,
                        scale);
  if (rc != FA_OK) return rc;
  if (!aligned16(dout) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv))
    return FA_ERR_ALIGNMENT;
  if (S == 0 || T == 0) return FA_OK;
  // Padded rows and the items (block, head) are 32-bit.
  const fattn::PackedGradLayout l =
      fattn::packed_grad_layout(T, S, H, Hk, d, see.window, see.sinks);
  if (((long long)T / 128 + S) * 128 > (1 << 30) ||
      ((long long)T / 128 + S) * (H + Hk) > 0x3fffffffLL || l.entries * H > 0x3fffffffLL)
    return FA_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < l.bytes) return FA_ERR_INVALID_ARG;
  if (!aligned16(workspace)) return FA_ERR_ALIGNMENT;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int *sched = nullptr, *status = nullptr, fault_cta = -1;
  if ((rc = acquire_sched(s, 2, &sched, &status, &fault_cta)) != FA_OK) return rc;
  const CUtensorMapDataType dt = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const int box = fattn::bwd_qdo_box_rows(d), rows = l.n_blocks * 128;
  float *ws = static_cast<float *>(workspace);
  fattn::PackedGradMaps m;
  if ((rc = encode_rows_map(&m.q, q, T, H, d, q_stride, true, box, 1, dt)) != FA_OK) return rc;
  if ((rc = encode_rows_map(&m.dout, dout, T, H, d, (long long)H * d, true, box, 1, dt)) != FA_OK)
    return rc;
  if ((rc = encode_rows_map(&m.k, k, T, Hk, d, k_stride, true, 128, 1, dt)) != FA_OK) return rc;
  if ((rc = encode_rows_map(&m.v, v, T, Hk, d, v_stride, true, 128, 1, dt)) != FA_OK) return rc;
  if ((rc = encode_dq_acc_map(&m.dq_acc, ws, H, rows, d)) != FA_OK) return rc;
  m.dk_acc = m.dv_acc = m.dq_acc;
  if (l.shared) {
    if ((rc = encode_dq_acc_map(&m.dk_acc, ws + l.dk_acc, Hk, rows, d)) != FA_OK) return rc;
    if ((rc = encode_dq_acc_map(&m.dv_acc, ws + l.dv_acc, Hk, rows, d)) != FA_OK) return rc;
  }
  fattn::PackedGrad p{};
  p.o = o, p.dout = dout, p.lse = lse, p.dq = dq, p.dk = dk, p.dv = dv, p.cu_seqlens = cu_seqlens;
  p.S = S, p.T = T, p.H = H, p.Hk = Hk, p.d = d, p.scale = scale;
  p.causal = see.causal, p.window = see.window, p.sinks = see.sinks;
  return cuda_status(fattn::launch_bwd_packed(m, p, ws, sched, status, fault_cta, s));
}
}  // namespace

int fa_backward_packed(const void *q, const void *k, const void *v, const void *o,
                       const void *dout, const float *lse, void *dq, void *dk, void *dv,
                       const int *cu_seqlens, int num_seqs, int total_tokens, int num_heads,
                       int num_kv_heads, int d, long long q_stride, long long k_stride,
                       long long v_stride, float scale, int causal, void *workspace,
                       unsigned long long workspace_bytes, fa_stream_t stream) {
  return backward_packed(q, k, v, o, dout, lse, dq, dk, dv, cu_seqlens, num_seqs, total_tokens,
                         num_heads, num_kv_heads, d, q_stride, k_stride, v_stride, scale,
                         all_keys(causal), workspace, workspace_bytes, stream);
}

unsigned long long fa_backward_packed_window_workspace_bytes(int num_seqs, int total_tokens,
                                                             int num_heads, int num_kv_heads,
                                                             int d, int window, int sinks) {
  Visible see;
  if (num_seqs <= 0 || total_tokens <= 0 || d <= 0) return 0;
  if (check_packed_sizes(num_seqs, total_tokens, num_heads, num_kv_heads) != FA_OK) return 0;
  if (window_keys(window, sinks, &see) != FA_OK) return 0;
  return static_cast<unsigned long long>(fattn::packed_grad_layout(total_tokens, num_seqs,
                                                                   num_heads, num_kv_heads, d,
                                                                   see.window, see.sinks)
                                             .bytes);
}

int fa_backward_packed_window(const void *q, const void *k, const void *v, const void *o,
                              const void *dout, const float *lse, void *dq, void *dk, void *dv,
                              const int *cu_seqlens, int num_seqs, int total_tokens,
                              int num_heads, int num_kv_heads, int d, long long q_stride,
                              long long k_stride, long long v_stride, float scale, int window,
                              int sinks, void *workspace, unsigned long long workspace_bytes,
                              fa_stream_t stream) {
  Visible see;
  const int rc = window_keys(window, sinks, &see);
  if (rc != FA_OK) return rc;
  return backward_packed(q, k, v, o, dout, lse, dq, dk, dv, cu_seqlens, num_seqs, total_tokens,
                         num_heads, num_kv_heads, d, q_stride, k_stride, v_stride, scale, see,
                         workspace, workspace_bytes, stream);
}

unsigned long long fa_paged_prefill_workspace_bytes(int num_seqs, int total_tokens, int num_heads,
                                                    int num_kv_heads,
                                                    int max_num_blocks_per_seq) {
  if (num_seqs <= 0 || total_tokens <= 0 || max_num_blocks_per_seq <= 0) return 0;
  if (check_packed_sizes(num_seqs, total_tokens, num_heads, num_kv_heads) != FA_OK) return 0;
  return static_cast<unsigned long long>(fattn::paged_prefill_workspace_bytes(
      total_tokens, num_seqs, num_heads, num_kv_heads, max_num_blocks_per_seq));
}

namespace {
// Checks shared by the chunk calls over the paged cache.
int check_chunks(const void *q, const void *k_cache, const void *v_cache, const int *block_tables,
                 const int *context_lens, const int *cu_seqlens, const void *out, int num_seqs,
                 int total_tokens, int num_heads, int num_kv_heads, int head_size, int block_size,
                 int num_blocks, int max_num_blocks_per_seq, long long q_stride, float scale) {
  if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !cu_seqlens || !out)
    return FA_ERR_INVALID_ARG;
  if (num_blocks <= 0 || max_num_blocks_per_seq <= 0) return FA_ERR_INVALID_ARG;
  if (!(std::isfinite(scale) && scale > 0.f)) return FA_ERR_INVALID_ARG;
  const int rc = check_packed_sizes(num_seqs, total_tokens, num_heads, num_kv_heads);
  if (rc != FA_OK) return rc;
  if (head_size != fattn::kDecodeHeadSize || block_size != fattn::kDecodeBlockSize)
    return FA_ERR_UNSUPPORTED;
  if (max_num_blocks_per_seq > (1 << 25)) return FA_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
      !aligned_to(block_tables, 4) || !aligned_to(context_lens, 4) || !aligned_to(cu_seqlens, 4))
    return FA_ERR_ALIGNMENT;
  return check_token_stride(q_stride, num_heads, head_size, 2);
}

int check_workspace(const void *workspace, unsigned long long bytes, size_t need) {
  if (need == 0) return FA_OK;
  if (!workspace || bytes < need) return FA_ERR_INVALID_ARG;
  return aligned16(workspace) ? FA_OK : FA_ERR_ALIGNMENT;
}

// The tensor maps of a chunk call.
int encode_chunk_maps(CUtensorMap *tq, CUtensorMap *tk, CUtensorMap *tv, const void *q,
                      const void *k_cache, const void *v_cache, int T, int H, int Hk,
                      int num_blocks, long long q_stride) {
  const int group = H / Hk;
  const int rc = encode_rows_map(tq, q, T, H, fattn::kDecodeHeadSize, q_stride, false, group,
                                 fattn::packed_tile_tokens(group),
                                 CU_TENSOR_MAP_DATA_TYPE_BFLOAT16);
  return rc != FA_OK ? rc : encode_paged_kv_maps(tk, tv, k_cache, v_cache, Hk, num_blocks, true);
}

int paged_prefill(const void *q, const void *k_cache, const void *v_cache,
                  const int *block_tables, const int *context_lens, const int *cu_seqlens,
                  void *out, int num_seqs, int total_tokens, int num_heads, int num_kv_heads,
                  int head_size, int block_size, int num_blocks, int max_num_blocks_per_seq,
                  long long q_stride, float scale, const Visible &see, void *workspace,
                  unsigned long long workspace_bytes, fa_stream_t stream) {
  int rc = check_chunks(q, k_cache, v_cache, block_tables, context_lens, cu_seqlens, out, num_seqs,
                        total_tokens, num_heads, num_kv_heads, head_size, block_size, num_blocks,
                        max_num_blocks_per_seq, q_stride, scale);
  if (rc != FA_OK) return rc;
  if (num_seqs == 0 || total_tokens == 0) return FA_OK;
  rc = check_workspace(workspace, workspace_bytes,
                       fattn::paged_prefill_workspace_bytes(total_tokens, num_seqs, num_heads,
                                                            num_kv_heads, max_num_blocks_per_seq,
                                                            see.window, see.sinks));
  if (rc != FA_OK) return rc;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int *sched = nullptr, *status = nullptr, fault_cta = -1;
  if ((rc = acquire_sched(s, 1, &sched, &status, &fault_cta)) != FA_OK) return rc;
  CUtensorMap tq, tk, tv;
  if ((rc = encode_chunk_maps(&tq, &tk, &tv, q, k_cache, v_cache, total_tokens, num_heads,
                              num_kv_heads, num_blocks, q_stride)) != FA_OK)
    return rc;
  fattn::PackedProblem p{};
  p.o = out, p.cu_seqlens = cu_seqlens, p.context_lens = context_lens;
  p.block_tables = block_tables;
  p.S = num_seqs, p.T = total_tokens, p.H = num_heads, p.Hk = num_kv_heads;
  p.max_blocks = max_num_blocks_per_seq, p.num_blocks = num_blocks, p.scale = scale;
  p.causal = see.causal, p.window = see.window, p.sinks = see.sinks;
  return cuda_status(fattn::launch_paged_prefill(tq, tk, tv, p, static_cast<float *>(workspace),
                                                 sched, status, fault_cta, s));
}
}  // namespace

int fa_paged_prefill(const void *q, const void *k_cache, const void *v_cache,
                     const int *block_tables, const int *context_lens, const int *cu_seqlens,
                     void *out, int num_seqs, int total_tokens, int num_heads, int num_kv_heads,
                     int head_size, int block_size, int num_blocks, int max_num_blocks_per_seq,
                     long long q_stride, float scale, void *workspace,
                     unsigned long long workspace_bytes, fa_stream_t stream) {
  return paged_prefill(q, k_cache, v_cache, block_tables, context_lens, cu_seqlens, out, num_seqs,
                       total_tokens, num_heads, num_kv_heads, head_size, block_size, num_blocks,
                       max_num_blocks_per_seq, q_stride, scale, all_keys(1), workspace,
                       workspace_bytes, stream);
}

unsigned long long fa_paged_prefill_window_workspace_bytes(int num_seqs, int total_tokens,
                                                           int num_heads, int num_kv_heads,
                                                           int max_num_blocks_per_seq, int window,
                                                           int sinks) {
  Visible see;
  if (num_seqs <= 0 || total_tokens <= 0 || max_num_blocks_per_seq <= 0) return 0;
  if (check_packed_sizes(num_seqs, total_tokens, num_heads, num_kv_heads) != FA_OK) return 0;
  if (window_keys(window, sinks, &see) != FA_OK) return 0;
  return static_cast<unsigned long long>(fattn::paged_prefill_workspace_bytes(
      total_tokens, num_seqs, num_heads, num_kv_heads, max_num_blocks_per_seq, see.window,
      see.sinks));
}

int fa_paged_prefill_window(const void *q, const void *k_cache, const void *v_cache,
                            const int *block_tables, const int *context_lens,
                            const int *cu_seqlens, void *out, int num_seqs, int total_tokens,
                            int num_heads, int num_kv_heads, int head_size, int block_size,
                            int num_blocks, int max_num_blocks_per_seq, long long q_stride,
                            float scale, int window, int sinks, void *workspace,
                            unsigned long long workspace_bytes, fa_stream_t stream) {
  Visible see;
  const int rc = window_keys(window, sinks, &see);
  if (rc != FA_OK) return rc;
  return paged_prefill(q, k_cache, v_cache, block_tables, context_lens, cu_seqlens, out, num_seqs,
                       total_tokens, num_heads, num_kv_heads, head_size, block_size, num_blocks,
                       max_num_blocks_per_seq, q_stride, scale, see, workspace, workspace_bytes,
                       stream);
}

unsigned long long fa_paged_prefill_shared_workspace_bytes(int num_seqs, int total_tokens,
                                                           int num_groups, int num_heads,
                                                           int num_kv_heads,
                                                           int max_num_blocks_per_seq) {
  if (num_seqs <= 0 || total_tokens <= 0 || max_num_blocks_per_seq <= 0) return 0;
  if (num_groups < 0 || num_groups > fattn::kSharedMaxGroups) return 0;
  if (check_packed_sizes(num_seqs, total_tokens, num_heads, num_kv_heads) != FA_OK) return 0;
  return static_cast<unsigned long long>(fattn::shared_layout(total_tokens, num_seqs, num_groups,
                                                              num_heads, num_kv_heads,
                                                              max_num_blocks_per_seq)
                                             .bytes);
}

int fa_paged_prefill_shared(const void *q, const void *k_cache, const void *v_cache,
                            const int *block_tables, const int *context_lens,
                            const int *cu_seqlens, const int *cu_groups, const int *prefix_lens,
                            void *out, int num_seqs, int total_tokens, int num_groups,
                            int num_heads, int num_kv_heads, int head_size, int block_size,
                            int num_blocks, int max_num_blocks_per_seq, long long q_stride,
                            float scale, void *workspace, unsigned long long workspace_bytes,
                            fa_stream_t stream) {
  if (num_groups < 0 || (num_groups > 0 && (!cu_groups || !prefix_lens))) return FA_ERR_INVALID_ARG;
  int rc = check_chunks(q, k_cache, v_cache, block_tables, context_lens, cu_seqlens, out, num_seqs,
                        total_tokens, num_heads, num_kv_heads, head_size, block_size, num_blocks,
                        max_num_blocks_per_seq, q_stride, scale);
  if (rc != FA_OK) return rc;
  if (num_groups > fattn::kSharedMaxGroups) return FA_ERR_UNSUPPORTED;
  if (!aligned_to(cu_groups, 4) || !aligned_to(prefix_lens, 4)) return FA_ERR_ALIGNMENT;
  if (num_seqs == 0 || total_tokens == 0) return FA_OK;
  rc = check_workspace(workspace, workspace_bytes,
                       fattn::shared_layout(total_tokens, num_seqs, num_groups, num_heads,
                                            num_kv_heads, max_num_blocks_per_seq)
                           .bytes);
  if (rc != FA_OK) return rc;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int *sched = nullptr, *status = nullptr, fault_cta = -1;
  if ((rc = acquire_sched(s, 1, &sched, &status, &fault_cta)) != FA_OK) return rc;
  CUtensorMap tq, tk, tv;
  if ((rc = encode_chunk_maps(&tq, &tk, &tv, q, k_cache, v_cache, total_tokens, num_heads,
                              num_kv_heads, num_blocks, q_stride)) != FA_OK)
    return rc;
  fattn::PackedProblem p{};
  p.o = out, p.cu_seqlens = cu_seqlens, p.context_lens = context_lens;
  p.block_tables = block_tables;
  p.S = num_seqs, p.T = total_tokens, p.H = num_heads, p.Hk = num_kv_heads;
  p.max_blocks = max_num_blocks_per_seq, p.num_blocks = num_blocks, p.scale = scale;
  p.causal = 1;
  return cuda_status(fattn::launch_paged_shared(tq, tk, tv, p, cu_groups, prefix_lens, num_groups,
                                                static_cast<char *>(workspace), sched, status,
                                                fault_cta, s));
}

int fa_device_status(void) {
  std::lock_guard<std::mutex> lock(g_mu);
  int dev = 0, rc;
  if ((rc = current_device(&dev)) != FA_OK) return rc;
  if (cudaDeviceSynchronize() != cudaSuccess) return FA_ERR_CUDA;
  int h = 0;
  if (cudaMemcpy(&h, g_dev[dev].status, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess)
    return FA_ERR_CUDA;
  if (h != 0 && cudaMemset(g_dev[dev].status, 0, sizeof(int)) != cudaSuccess) return FA_ERR_CUDA;
  return h;
}

int fa_decode_gqa_select(int impl) {
  if (impl < 0 || impl > 2) return FA_ERR_INVALID_ARG;
  g_decode_gqa_impl.store(impl);
  return FA_OK;
}

int fa_debug_inject_fault(int mode) {
  if (mode != 0 && mode != 1 && mode != 2) return FA_ERR_INVALID_ARG;
  std::lock_guard<std::mutex> lock(g_mu);
  int dev = 0, rc;
  if ((rc = current_device(&dev)) != FA_OK) return rc;
  g_dev[dev].inject_fault = mode;
  return FA_OK;
}

void fa_release(void) {
  std::lock_guard<std::mutex> lock(g_mu);
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return;
  DeviceState &st = g_dev[dev];
  // The buffers grown in stream order may still be in use by work the caller
  // has not waited for; cudaFree does not order itself after it.
  cudaDeviceSynchronize();
  if (st.decode_ws) cudaFree(st.decode_ws);
  if (st.decode_counters) cudaFree(st.decode_counters);
  if (st.status) cudaFree(st.status);
  if (st.fwd_sched) cudaFree(st.fwd_sched);
  if (st.mask_ws) cudaFree(st.mask_ws);
  st = DeviceState{};
}

}  // extern "C"
