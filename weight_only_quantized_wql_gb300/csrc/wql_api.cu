// wql_api.cu -- the extern "C" entry points declared in include/wql.h.
//
// Every entry point validates its arguments on the host before it touches
// the CUDA runtime, so bad arguments never launch anything and never need a
// GPU to be diagnosed.  Kernel choice by token count lives here.
#include <atomic>
#include <cstdint>
#include <cstring>
#include <string>

#include <cudaTypedefs.h>

#include <mutex>

#include "sm100.cuh"
#include "wql_common.cuh"
#include "embed.cuh"
#include "mx.cuh"
#include "requests.cuh"

namespace wql {

namespace {
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

void resolve_encoder() {
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                       &q) == cudaSuccess &&
      q == cudaDriverEntryPointSuccess)
    g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
}
}  // namespace

cudaError_t make_tmap_2d(CUtensorMap* map, const void* base, int elem_bytes, uint64_t cols,
                         uint64_t rows, uint64_t row_stride_bytes, uint32_t box_cols,
                         uint32_t box_rows, Swizzle swz) {
  std::call_once(g_encode_once, resolve_encoder);
  if (!g_encode) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {row_stride_bytes};
  const cuuint32_t box[2] = {box_cols, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  const CUtensorMapDataType dt =
      elem_bytes == 4 ? CU_TENSOR_MAP_DATA_TYPE_UINT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16;
  const CUresult r = g_encode(
      map, dt, 2, const_cast<void*>(base), dims, strides, box, estr,
      CU_TENSOR_MAP_INTERLEAVE_NONE,
      swz == Swizzle::k128B ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
      CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t make_tmap_blocks(CUtensorMap* map, bool spread, const void* base, uint64_t row_bytes,
                             uint64_t rows, uint32_t box_rows, uint32_t box_blocks) {
  std::call_once(g_encode_once, resolve_encoder);
  if (!g_encode) return cudaErrorNotSupported;
  const uint64_t block = spread ? 64 : 128;
  const cuuint64_t dims[3] = {spread ? 128u : 32u, rows, row_bytes / block};
  const cuuint64_t strides[2] = {row_bytes, block};
  const cuuint32_t box[3] = {spread ? 128u : 32u, box_rows, box_blocks};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = g_encode(
      map, spread ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B : CU_TENSOR_MAP_DATA_TYPE_UINT32, 3,
      const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

namespace {
std::atomic<uint64_t> g_launches{0};
thread_local std::string g_last_error;
constexpr int kDecodeMaxTokens = 16;
constexpr int64_t kLoraMaxTokens = int64_t(1) << 23;   // 2^15 slices of 256
constexpr int64_t kBeamMaxRows = int64_t(1) << 20;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
// Whether two pieces of memory share a byte (0 bytes: none).
bool share(const void* p, int64_t p_bytes, const void* q, int64_t q_bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return p_bytes > 0 && q_bytes > 0 && a < b + (uintptr_t)q_bytes && b < a + (uintptr_t)p_bytes;
}
bool half_dtype(int d) { return d == WQL_F16 || d == WQL_BF16; }

wql_status cuda_fail(cudaError_t e) {
  g_last_error = cudaGetErrorString(e);
  return WQL_ECUDA;
}

size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
}  // namespace

void note_launch() { g_launches.fetch_add(1, std::memory_order_relaxed); }

wql_status record_cuda_error(cudaError_t e) { return cuda_fail(e); }

int device_sm_count() {
  static thread_local int cached_dev = -1;
  static thread_local int cached_sms = 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  if (dev != cached_dev) {
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
      sms = 1;
    cached_dev = dev;
    cached_sms = sms;
  }
  return cached_sms;
}

WorkspaceLayout workspace_layout(int64_t m, int64_t n, int32_t topk) {
  WorkspaceLayout l{};
  l.counter_off = 0;
  size_t off = 256;
  // fixed place (any m): per-token tickets of the top-K selection
  l.tickets_off = off;
  if (topk > 0) off += 256 * sizeof(unsigned int);
  l.cand_off = off;
  if (topk > 0) off += round_up((size_t)m * WQL_MAX_CTAS * (size_t)topk * 8, 256);
  (void)n;
  l.total = off;
  return l;
}

namespace {
std::atomic<long long> g_wait_budget{0};
std::atomic<int> g_stall_mma{0};
}  // namespace

long long diag_wait_budget() {
  const long long b = g_wait_budget.load(std::memory_order_relaxed);
  return b > 0 ? b : kWaitBudgetCycles;
}
int diag_stall_mma() { return g_stall_mma.load(std::memory_order_relaxed); }

wql_status check_logits_args(const void* x, int32_t x_dtype, int64_t m, const wql_weight* w,
                             const void* bias, const void* logits_out, int32_t topk,
                             const void* topk_idx, const void* topk_val, int64_t* g_out) {
  if (!w || m < 0 || w->n < 0 || w->k <= 0 || w->group < 0) return WQL_EINVAL;
  const int fmt = weight_format(w);
  if ((w->format & ~(WQL_FMT_MASK | WQL_WEIGHT_STATIC)) != 0 ||
      (fmt != WQL_FMT_SYM && fmt != WQL_FMT_E4M3 && fmt != WQL_FMT_ASYM))
    return WQL_EINVAL;
  if (topk < 0 || topk > WQL_MAX_TOPK) return WQL_EINVAL;
  const int64_t n = w->n, k = w->k;
  if (m > 0 && n > 0) {
    if (!x || !w->qweight || !w->scales) return WQL_EINVAL;
    // logits_out may be NULL only for candidates alone (top-K on)
    if (!logits_out && topk == 0) return WQL_EINVAL;
    if (topk > 0 && (!topk_idx || !topk_val)) return WQL_EINVAL;
    if (topk > n) return WQL_EINVAL;
    if (fmt == WQL_FMT_ASYM && !w->zeros) return WQL_EINVAL;
  }
  if (w->bits != 4 && w->bits != 8) return WQL_EUNSUPPORTED;
  if (fmt == WQL_FMT_E4M3 && (w->bits != 8 || w->group != 0)) return WQL_EUNSUPPORTED;
  if (fmt == WQL_FMT_ASYM && (w->bits != 4 || w->group == 0 || w->group % 128 != 0))
    return WQL_EUNSUPPORTED;
  if (!half_dtype(x_dtype) || !half_dtype(w->scale_dtype)) return WQL_EUNSUPPORTED;
  const int64_t g = w->group == 0 ? k : w->group;
  if (k % 64 != 0 || g % 64 != 0 || k % g != 0) return WQL_EUNSUPPORTED;
  if (n >= (int64_t(1) << 31) || m >= (int64_t(1) << 31) || k >= (int64_t(1) << 30))
    return WQL_EUNSUPPORTED;
  if (!aligned(x, 16) || !aligned(w->qweight, 16) || !aligned(w->scales, 2) ||
      !aligned(logits_out, 2) || !aligned(bias, 2))
    return WQL_EUNSUPPORTED;
  *g_out = g;
  return WQL_OK;
}

// A microscaled operand: format, sizes, pointers, alignment.
wql_status check_mx(const wql_mx* a) {
  if (!a || a->rows < 0 || a->k <= 0 || a->reserved != 0) return WQL_EINVAL;
  if (a->format != WQL_MX_FP4 && a->format != WQL_MX_FP8) return WQL_EINVAL;
  if (a->rows > 0 && (!a->codes || !a->scales)) return WQL_EINVAL;
  if (a->k % kMxBlock != 0 || a->k > kMxMaxK ||
      a->rows >= (int64_t(1) << 31) - kMxTileRows)
    return WQL_EUNSUPPORTED;
  if (!aligned(a->codes, 16) || !aligned(a->scales, 16)) return WQL_EUNSUPPORTED;
  return WQL_OK;
}

}  // namespace wql

using namespace wql;

extern "C" {

const char* wql_status_string(wql_status status) {
  switch (status) {
    case WQL_OK: return "WQL_OK: success";
    case WQL_EINVAL: return "WQL_EINVAL: invalid argument";
    case WQL_EUNSUPPORTED: return "WQL_EUNSUPPORTED: unsupported configuration";
    case WQL_ECUDA: return "WQL_ECUDA: CUDA error";
    case WQL_EWORKSPACE: return "WQL_EWORKSPACE: workspace missing or too small";
  }
  return "unknown wql_status";
}

const char* wql_last_error(void) { return g_last_error.c_str(); }

uint64_t wql_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

size_t wql_workspace_size(int64_t m, int64_t n, int32_t topk) {
  if (m < 0 || n < 0 || topk < 0 || topk > WQL_MAX_TOPK) return 0;
  return workspace_layout(m, n, topk).total;
}

wql_status wql_quantize(const void* w, int32_t w_dtype, int64_t n, int64_t k, int32_t bits,
                        int32_t group, int32_t scale_dtype, int32_t clip, void* qweight_out,
                        void* scales_out, cudaStream_t stream) {
  return wql_quantize_ex(w, w_dtype, n, k, WQL_FMT_SYM, bits, group, scale_dtype, clip,
                         qweight_out, scales_out, nullptr, stream);
}

wql_status wql_quantize_ex(const void* w, int32_t w_dtype, int64_t n, int64_t k, int32_t format,
                           int32_t bits, int32_t group, int32_t scale_dtype, int32_t clip,
                           void* qweight_out, void* scales_out, void* zeros_out,
                           cudaStream_t stream) {
  if (n < 0 || k <= 0 || group < 0) return WQL_EINVAL;
  if (n > 0 && (!w || !qweight_out || !scales_out)) return WQL_EINVAL;
  if (clip != WQL_CLIP_RTN && clip != WQL_CLIP_MSE) return WQL_EINVAL;
  if (format != WQL_FMT_SYM && format != WQL_FMT_E4M3 && format != WQL_FMT_ASYM)
    return WQL_EINVAL;
  if (format == WQL_FMT_ASYM && n > 0 && !zeros_out) return WQL_EINVAL;
  if (format == WQL_FMT_E4M3 && (bits != 8 || group != 0 || clip != WQL_CLIP_RTN))
    return WQL_EUNSUPPORTED;
  if (format == WQL_FMT_ASYM && (bits != 4 || group == 0 || group % 128 != 0 ||
                                 clip != WQL_CLIP_RTN))
    return WQL_EUNSUPPORTED;
  if (bits != 4 && bits != 8) return WQL_EUNSUPPORTED;
  if (w_dtype != WQL_F32 && !half_dtype(w_dtype)) return WQL_EUNSUPPORTED;
  if (!half_dtype(scale_dtype)) return WQL_EUNSUPPORTED;
  const int64_t g = group == 0 ? k : group;
  if (k % 8 != 0 || k % g != 0 || g % 8 != 0) return WQL_EUNSUPPORTED;
  if (!aligned(w, 16) || !aligned(qweight_out, 16) || !aligned(scales_out, 2))
    return WQL_EUNSUPPORTED;
  if (n == 0) return WQL_OK;
  if (g > (1 << 30)) return WQL_EUNSUPPORTED;
  QuantizeArgs a{};
  a.w = w;
  a.w_dtype = w_dtype;
  a.n = n;
  a.k = k;
  a.bits = bits;
  a.group_eff = (int)g;
  a.scale_dtype = scale_dtype;
  a.nratios = clip == WQL_CLIP_MSE ? 5 : 1;
  static const double kRatios[5] = {1.0, 0.95, 0.9, 0.85, 0.8};
  // the largest code magnitude the scale maps amax (or, asymmetric, the
  // group's range) to
  const double qmax = format == WQL_FMT_E4M3 ? 448.0 : format == WQL_FMT_ASYM ? 15.0
                      : bits == 4 ? 7.0 : 127.0;
  for (int i = 0; i < 5; ++i) a.ratio_c[i] = (float)(kRatios[i] / qmax);
  a.qweight = qweight_out;
  a.scales = static_cast<uint16_t*>(scales_out);
  a.format = format;
  a.zeros = static_cast<uint8_t*>(zeros_out);
  cudaError_t e = launch_quantize(a, stream);
  return e == cudaSuccess ? WQL_OK : cuda_fail(e);
}

wql_status wql_pack(const uint8_t* nibbles, int64_t n, int64_t k, int32_t* packed_out,
                    cudaStream_t stream) {
  if (n < 0 || k < 0) return WQL_EINVAL;
  if (n > 0 && k > 0 && (!nibbles || !packed_out)) return WQL_EINVAL;
  if (k % 8 != 0) return WQL_EUNSUPPORTED;
  if (!aligned(nibbles, 8) || !aligned(packed_out, 4)) return WQL_EUNSUPPORTED;
  if (n == 0 || k == 0) return WQL_OK;
  cudaError_t e = launch_pack(nibbles, n, k, reinterpret_cast<uint32_t*>(packed_out), stream);
  return e == cudaSuccess ? WQL_OK : cuda_fail(e);
}

wql_status wql_unpack(const int32_t* packed, int64_t n, int64_t k, uint8_t* nibbles_out,
                      cudaStream_t stream) {
  if (n < 0 || k < 0) return WQL_EINVAL;
  if (n > 0 && k > 0 && (!packed || !nibbles_out)) return WQL_EINVAL;
  if (k % 8 != 0) return WQL_EUNSUPPORTED;
  if (!aligned(packed, 4) || !aligned(nibbles_out, 8)) return WQL_EUNSUPPORTED;
  if (n == 0 || k == 0) return WQL_OK;
  cudaError_t e = launch_unpack(reinterpret_cast<const uint32_t*>(packed), n, k, nibbles_out,
                                stream);
  return e == cudaSuccess ? WQL_OK : cuda_fail(e);
}

wql_status wql_logits(const void* x, int32_t x_dtype, int64_t m, const wql_weight* w,
                      const void* bias, void* logits_out, int32_t topk, int32_t* topk_idx,
                      float* topk_val, void* workspace, size_t ws_bytes, cudaStream_t stream) {
  int64_t g = 0;
  const wql_status st = check_logits_args(x, x_dtype, m, w, bias, logits_out, topk, topk_idx,
                                          topk_val, &g);
  if (st != WQL_OK) return st;
  const int64_t n = w->n, k = w->k;
  if (m == 0 || n == 0) return WQL_OK;
  const WorkspaceLayout lay = workspace_layout(m, n, topk);
  // top-K needs a workspace; any workspace given (top-K or not) holds the
  // kernels' counter block, so it must be large enough and aligned
  if (topk > 0 && !workspace) return WQL_EWORKSPACE;
  if (workspace && (ws_bytes < lay.total || !aligned(workspace, 256))) return WQL_EWORKSPACE;
  const int esz = 2;
  // tokens per decode launch: 16, fewer when x for 16 rows does not fit in
  // shared memory next to the rest
  const int dchunk = decode_max_tokens((int)k, w->bits, (int)g, topk, weight_format(w));
  if (dchunk < 1) return WQL_EUNSUPPORTED;

  unsigned char* ws = static_cast<unsigned char*>(workspace);
  // No workspace (allowed when topk == 0): the kernels skip the error word.
  unsigned int* err_word =
      ws ? reinterpret_cast<unsigned int*>(ws + lay.counter_off) + 1 : nullptr;
  LogitsArgs base{};
  base.x_dtype = x_dtype;
  base.qweight = w->qweight;
  base.scales = static_cast<const uint16_t*>(w->scales);
  base.bits = w->bits;
  base.group_eff = (int)g;
  base.scale_dtype = w->scale_dtype;
  base.n = (int)n;
  base.k = (int)k;
  base.bias = bias;
  base.topk = topk;
  base.format = weight_format(w);
  base.weights_static = (w->format & WQL_WEIGHT_STATIC) ? 1 : 0;
  base.zeros = static_cast<const uint8_t*>(w->zeros);
  // the counter block also schedules the decode kernel's work units
  if (ws) base.counter = reinterpret_cast<unsigned int*>(ws + lay.counter_off);
  if (topk > 0) {
    base.cand = reinterpret_cast<unsigned long long*>(ws + lay.cand_off);
    base.tickets = reinterpret_cast<unsigned int*>(ws + lay.tickets_off);
  }
  // Token counts above 16 go to the tensor-core kernel (up to 256 tokens per
  // launch) when it supports the dtype combination; otherwise the decode
  // kernel runs on 16-token slices.
  LogitsArgs probe = base;
  probe.m = (int)(m < 256 ? m : 256);
  // (fp8 and zero-point weights, and candidates alone, take the decode
  // kernel's 16-token slices at every m)
  const bool use_tc = m > kDecodeMaxTokens && weight_format(w) == WQL_FMT_SYM && logits_out &&
                      tc_supported(probe);
  // decode slices of balanced size (16 tokens that do not fit one launch run
  // as 8 + 8, not 15 + 1: the weight is streamed once per slice either way)
  const int64_t nslices = (m + dchunk - 1) / dchunk;
  const int64_t chunk = use_tc ? 256 : (m + nslices - 1) / nslices;
  for (int64_t m0 = 0; m0 < m; m0 += chunk) {
    const int64_t mc = (m - m0) < chunk ? (m - m0) : chunk;
    LogitsArgs a = base;
    a.x = static_cast<const unsigned char*>(x) + (size_t)m0 * k * esz;
    a.m = (int)mc;
    a.logits = logits_out ? static_cast<unsigned char*>(logits_out) + (size_t)m0 * n * esz
                          : nullptr;
    if (topk > 0) {
      a.topk_idx = topk_idx + (size_t)m0 * topk;
      a.topk_val = topk_val + (size_t)m0 * topk;
    }
    cudaError_t e;
    if (use_tc && mc > kDecodeMaxTokens) {
      // logits on the tensor cores, then the top-K from the rounded logits
      LogitsArgs g = a;
      g.topk = 0;
      e = launch_tc(g, err_word, stream);
      if (e == cudaSuccess && a.topk > 0) e = launch_topk_select(a, stream);
    } else
      e = launch_decode(a, err_word, stream);
    if (e != cudaSuccess) return cuda_fail(e);
  }
  return WQL_OK;
}

wql_status wql_embed_gather(const int32_t* ids, int64_t t, const wql_weight* w,
                            int32_t out_dtype, void* out, cudaStream_t stream) {
  if (!w || t < 0 || w->n < 0 || w->k <= 0 || w->group < 0) return WQL_EINVAL;
  const int fmt = weight_format(w);
  if ((w->format & ~(WQL_FMT_MASK | WQL_WEIGHT_STATIC)) != 0 ||
      (fmt != WQL_FMT_SYM && fmt != WQL_FMT_E4M3 && fmt != WQL_FMT_ASYM))
    return WQL_EINVAL;
  if (fmt != WQL_FMT_SYM) return WQL_EUNSUPPORTED;
  const int64_t n = w->n, k = w->k;
  if (t > 0 && (!ids || !out)) return WQL_EINVAL;
  if (t > 0 && n > 0 && (!w->qweight || !w->scales)) return WQL_EINVAL;
  if (w->bits != 4 && w->bits != 8) return WQL_EUNSUPPORTED;
  if (!half_dtype(out_dtype) || !half_dtype(w->scale_dtype)) return WQL_EUNSUPPORTED;
  const int64_t g = w->group == 0 ? k : w->group;
  if (k % 8 != 0 || g % 8 != 0 || k % g != 0) return WQL_EUNSUPPORTED;
  if (n >= (int64_t(1) << 31) || t >= (int64_t(1) << 31) || k >= (int64_t(1) << 30))
    return WQL_EUNSUPPORTED;
  if (!aligned(ids, 4) || !aligned(w->qweight, 8) || !aligned(w->scales, 2) || !aligned(out, 16))
    return WQL_EUNSUPPORTED;
  if (t == 0) return WQL_OK;
  EmbedArgs a{};
  a.ids = ids;
  a.t = (int)t;
  a.qweight = w->qweight;
  a.scales = static_cast<const uint16_t*>(w->scales);
  a.bits = w->bits;
  a.group_eff = (int)g;
  a.scale_dtype = w->scale_dtype;
  a.n = (int)n;
  a.k = (int)k;
  a.out_dtype = out_dtype;
  a.out = out;
  cudaError_t e = launch_embed_gather(a, stream);
  return e == cudaSuccess ? WQL_OK : cuda_fail(e);
}

wql_status wql_topk_rescore(const void* x, int32_t x_dtype, int64_t m, const void* w_ref,
                            int32_t wref_dtype, int64_t n, int64_t k, const void* bias,
                            int32_t topk, int32_t* topk_idx, float* topk_val,
                            void* logits_inout, cudaStream_t stream) {
  if (m < 0 || n < 0 || k <= 0) return WQL_EINVAL;
  if (topk < 0 || topk > WQL_MAX_TOPK || topk > n) return WQL_EINVAL;
  if (m > 0 && topk > 0 && (!x || !w_ref || !topk_idx || !topk_val || !logits_inout))
    return WQL_EINVAL;
  if (!half_dtype(x_dtype) || wref_dtype != x_dtype) return WQL_EUNSUPPORTED;
  if (k % 8 != 0) return WQL_EUNSUPPORTED;
  if (n >= (int64_t(1) << 31) || m >= (int64_t(1) << 31)) return WQL_EUNSUPPORTED;
  if (!aligned(x, 16) || !aligned(w_ref, 16) || !aligned(logits_inout, 2) || !aligned(bias, 2))
    return WQL_EUNSUPPORTED;
  if (m == 0 || n == 0 || topk == 0) return WQL_OK;
  RescoreArgs a{};
  a.x = x;
  a.x_dtype = x_dtype;
  a.m = (int)m;
  a.n = (int)n;
  a.k = (int)k;
  a.w_ref = w_ref;
  a.bias = bias;
  a.topk = topk;
  a.topk_idx = topk_idx;
  a.topk_val = topk_val;
  a.logits = logits_inout;
  cudaError_t e = launch_rescore(a, stream);
  return e == cudaSuccess ? WQL_OK : cuda_fail(e);
}

size_t wql_mx_scale_bytes(int64_t rows, int64_t k) {
  if (rows < 0 || k <= 0) return 0;
  return (size_t)((rows + kMxTileRows - 1) / kMxTileRows) * (size_t)mx_tile_cols(k) * kMxTileBytes;
}

wql_status wql_mx_quantize(const void* x, int32_t x_dtype, int64_t rows, int64_t k,
                           int32_t format, void* codes_out, void* scales_out,
                           cudaStream_t stream) {
  if (rows < 0 || k <= 0) return WQL_EINVAL;
  if (format != WQL_MX_FP4 && format != WQL_MX_FP8) return WQL_EINVAL;
  if (rows > 0 && (!x || !codes_out || !scales_out)) return WQL_EINVAL;
  if (x_dtype != WQL_F32 && !half_dtype(x_dtype)) return WQL_EUNSUPPORTED;
  if (k % kMxBlock != 0 || k > kMxMaxK || rows >= (int64_t(1) << 31) - kMxTileRows)
    return WQL_EUNSUPPORTED;
  if (!aligned(x, 16) || !aligned(codes_out, 16) || !aligned(scales_out, 16))
    return WQL_EUNSUPPORTED;
  if (rows == 0) return WQL_OK;
  MxQuantizeArgs a{};
  a.x = x;
  a.x_dtype = x_dtype;
  a.rows = (int)rows;
  a.k = (int)k;
  a.format = format;
  a.codes = codes_out;
  a.scales = scales_out;
  const cudaError_t e = launch_mx_quantize(a, stream);
  return e == cudaSuccess ? WQL_OK : cuda_fail(e);
}

wql_status wql_mx_dequantize(const wql_mx* a, int32_t out_dtype, void* out, cudaStream_t stream) {
  const wql_status st = check_mx(a);
  if (st != WQL_OK) return st;
  if (a->rows > 0 && !out) return WQL_EINVAL;
  if (out_dtype != WQL_F32 && !half_dtype(out_dtype)) return WQL_EUNSUPPORTED;
  if (!aligned(out, 16)) return WQL_EUNSUPPORTED;
  if (a->rows == 0) return WQL_OK;
  MxDequantizeArgs d{};
  d.codes = a->codes;
  d.scales = a->scales;
  d.format = a->format;
  d.rows = (int)a->rows;
  d.k = (int)a->k;
  d.out_dtype = out_dtype;
  d.out = out;
  const cudaError_t e = launch_mx_dequantize(d, stream);
  return e == cudaSuccess ? WQL_OK : cuda_fail(e);
}

wql_status wql_mx_logits(const wql_mx* x, const wql_mx* w, const void* bias, int32_t out_dtype,
                         void* logits_out, void* workspace, size_t ws_bytes,
                         cudaStream_t stream) {
  wql_status st = check_mx(x);
  if (st == WQL_OK) st = check_mx(w);
  if (st != WQL_OK) return st;
  if (x->k != w->k) return WQL_EINVAL;
  const bool work = x->rows > 0 && w->rows > 0;
  if (work && !logits_out) return WQL_EINVAL;
  if (w->format != WQL_MX_FP4) return WQL_EUNSUPPORTED;
  if (!half_dtype(out_dtype)) return WQL_EUNSUPPORTED;
  if (!aligned(logits_out, 2) || !aligned(bias, 2)) return WQL_EUNSUPPORTED;
  if (!work) return WQL_OK;
  const WorkspaceLayout lay = workspace_layout(x->rows, w->rows, 0);
  if (workspace && (ws_bytes < lay.total || !aligned(workspace, 256))) return WQL_EWORKSPACE;
  MxLogitsArgs a{};
  a.x_codes = x->codes;
  a.x_scales = x->scales;
  a.x_format = x->format;
  a.w_codes = w->codes;
  a.w_scales = w->scales;
  a.m = (int)x->rows;
  a.n = (int)w->rows;
  a.k = (int)x->k;
  a.bias = bias;
  a.out_dtype = out_dtype;
  a.out = logits_out;
  if (workspace)
    a.err = reinterpret_cast<unsigned int*>(static_cast<unsigned char*>(workspace) +
                                            lay.counter_off) + 1;
  const cudaError_t e = launch_mx_logits(a, stream);
  return e == cudaSuccess ? WQL_OK : cuda_fail(e);
}

wql_status wql_add_rmsnorm(const void* x, const void* residual, const void* gamma, int32_t dtype,
                           int64_t m, int64_t k, float eps, int32_t out_format, void* out,
                           void* scales_out, void* residual_out, cudaStream_t stream) {
  if (m < 0 || k <= 0 || !(eps >= 0.f)) return WQL_EINVAL;
  if (out_format < WQL_NORM_SAME || out_format > WQL_NORM_MX_FP4) return WQL_EINVAL;
  if (m > 0 && (!x || !gamma || !out)) return WQL_EINVAL;
  if (m > 0 && out_format != WQL_NORM_SAME && !scales_out) return WQL_EINVAL;
  if (!half_dtype(dtype)) return WQL_EUNSUPPORTED;
  if (k > 65536 || m >= (int64_t(1) << 31) - kMxTileRows) return WQL_EUNSUPPORTED;
  const bool mx = out_format == WQL_NORM_MX_FP8 || out_format == WQL_NORM_MX_FP4;
  if (mx && k % kMxBlock != 0) return WQL_EUNSUPPORTED;
  const size_t al = mx ? 16 : 2;
  if (!aligned(x, al) || !aligned(residual, al) || !aligned(gamma, al) ||
      !aligned(residual_out, al) ||
      !aligned(out, mx ? 16 : out_format == WQL_NORM_SAME ? 2 : 1) ||
      !aligned(scales_out, mx ? 16 : 4))
    return WQL_EUNSUPPORTED;
  if (m == 0) return WQL_OK;
  NormArgs a{};
  a.x = x;
  a.residual = residual;
  a.gamma = gamma;
  a.dtype = dtype;
  a.m = (int)m;
  a.k = (int)k;
  a.eps = eps;
  a.out_format = out_format;
  a.out = out;
  a.scales = scales_out;
  a.residual_out = residual_out;
  const cudaError_t e = launch_add_rmsnorm(a, stream);
  return e == cudaSuccess ? WQL_OK : cuda_fail(e);
}

wql_status wql_sample(const void* logits, int32_t dtype, int64_t m, int64_t n, const float* u,
                      const float* temperature, const int32_t* top_k, const float* top_p,
                      const float* min_p, int32_t* ids_out, float* logp_out,
                      cudaStream_t stream) {
  if (m < 0 || n <= 0) return WQL_EINVAL;
  if (m > 0 && (!logits || !u || !ids_out)) return WQL_EINVAL;
  if (dtype != WQL_F32 && !half_dtype(dtype)) return WQL_EUNSUPPORTED;
  if (n > WQL_SAMPLE_MAX_N || m >= (int64_t(1) << 27)) return WQL_EUNSUPPORTED;
  if (!aligned(logits, dtype == WQL_F32 ? 4 : 2) || !aligned(u, 4) || !aligned(temperature, 4) || !aligned(top_k, 4) ||
      !aligned(top_p, 4) || !aligned(min_p, 4) || !aligned(ids_out, 4) || !aligned(logp_out, 4))
    return WQL_EUNSUPPORTED;
  if (m == 0) return WQL_OK;
  SampleArgs a{};
  a.logits = logits;
  a.dtype = dtype;
  a.m = (int)m;
  a.n = (int)n;
  a.u = u;
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.ids = ids_out;
  a.logp = logp_out;
  a.wait_budget = diag_wait_budget();
  a.diag_stall = diag_stall_mma();
  const cudaError_t e = launch_sample(a, stream);
  return e == cudaSuccess ? WQL_OK : cuda_fail(e);
}

size_t wql_lora_workspace_size(int64_t m, int32_t rank) {
  if (m <= 0 || m > kLoraMaxTokens || rank <= 0 || rank > WQL_LORA_MAX_RANK) return 0;
  return round_up((size_t)m * lora_chunks(rank) * 64, 256) + round_up((size_t)m * 4, 256);
}

wql_status wql_lora_add(const wql_lora* w, const void* x, int64_t m, const int32_t* ids,
                        const void* y, void* out, void* workspace, size_t ws_bytes,
                        cudaStream_t stream) {
  if (!w || m < 0 || w->count < 0 || w->n < 0 || w->k <= 0 || w->rank <= 0) return WQL_EINVAL;
  const bool work = m > 0 && w->n > 0;
  if (work && (!x || !ids || !y || !out)) return WQL_EINVAL;
  if (work && w->count > 0 && (!w->a || !w->b)) return WQL_EINVAL;
  if (!half_dtype(w->dtype) || w->rank % 8 != 0 || w->rank > WQL_LORA_MAX_RANK) return WQL_EUNSUPPORTED;
  if (w->k % 8 != 0 || w->k > kMxMaxK || w->n >= (int64_t(1) << 31) ||
      w->count >= WQL_LORA_MAX_COUNT || m > kLoraMaxTokens)
    return WQL_EUNSUPPORTED;
  if (!aligned(w->a, 16) || !aligned(w->b, 16) || !aligned(w->scale, 4) || !aligned(x, 16) ||
      !aligned(ids, 4) || !aligned(y, 2) || !aligned(out, 2))
    return WQL_EUNSUPPORTED;
  if (!work) return WQL_OK;
  const size_t u_bytes = round_up((size_t)m * lora_chunks(w->rank) * 64, 256);
  if (!workspace || ws_bytes < wql_lora_workspace_size(m, w->rank) || !aligned(workspace, 256))
    return WQL_EWORKSPACE;
  const int64_t out_bytes = m * w->n * 2;              // below 2^55
  if ((out != y && share(out, out_bytes, y, out_bytes)) || share(out, out_bytes, x, m * w->k * 2) ||
      share(out, out_bytes, ids, m * 4) || share(out, out_bytes, w->a, w->count * w->rank * w->k * 2) ||
      share(out, out_bytes, w->b, w->count * w->rank * w->n * 2) ||
      (w->scale && share(out, out_bytes, w->scale, w->count * 4)) ||
      share(out, out_bytes, workspace, (int64_t)wql_lora_workspace_size(m, w->rank)))
    return WQL_EINVAL;
  LoraArgs a{};
  a.a = w->a;
  a.b = w->b;
  a.scale = w->scale;
  a.x = x;
  a.ids = ids;
  a.y = y;
  a.out = out;
  a.u = static_cast<uint4*>(workspace);
  a.factor = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + u_bytes);
  a.dtype = w->dtype;
  a.rank = w->rank;
  a.chunks = lora_chunks(w->rank);
  a.count = (int)w->count;
  a.n = (int)w->n;
  a.k = (int)w->k;
  a.m = (int)m;
  const cudaError_t e = launch_lora_add(a, stream);
  return e == cudaSuccess ? WQL_OK : cuda_fail(e);
}

size_t wql_beam_workspace_size(int64_t batch, int64_t beams, int64_t n) {
  if (batch <= 0 || beams <= 0 || beams > WQL_MAX_BEAMS || n <= 0 || n > WQL_BEAM_MAX_N ||
      batch > kBeamMaxRows / beams)
    return 0;
  const int wide = beam_parts(batch * beams, n, WQL_F32).parts;
  const int half = beam_parts(batch * beams, n, WQL_F16).parts;
  const size_t parts = (size_t)batch * beams * (wide > half ? wide : half);
  return round_up(parts * sizeof(float2), 256) + round_up(parts * beams * 8, 256);
}

wql_status wql_beam_select(const void* logits, int32_t dtype, int64_t batch, int64_t beams,
                           int64_t n, const float* scores, int32_t eos, int32_t order,
                           int32_t* tokens_out, int32_t* parents_out, float* scores_out,
                           float* ended_out, void* workspace, size_t ws_bytes,
                           cudaStream_t stream) {
  if (batch < 0 || beams <= 0 || n <= 0 || eos < -1 || eos >= n) return WQL_EINVAL;
  if (order != WQL_BEAM_RANKED && order != WQL_BEAM_ANCHORED) return WQL_EINVAL;
  if (batch > 0 && (!logits || !scores || !tokens_out || !parents_out || !scores_out))
    return WQL_EINVAL;
  if (dtype != WQL_F32 && !half_dtype(dtype)) return WQL_EUNSUPPORTED;
  if (beams > WQL_MAX_BEAMS || n > WQL_BEAM_MAX_N || batch > kBeamMaxRows / beams)
    return WQL_EUNSUPPORTED;
  if (!aligned(logits, dtype == WQL_F32 ? 4 : 2) || !aligned(scores, 4) || !aligned(tokens_out, 4) ||
      !aligned(parents_out, 4) || !aligned(scores_out, 4) || !aligned(ended_out, 4))
    return WQL_EUNSUPPORTED;
  if (batch == 0) return WQL_OK;
  if (!workspace || ws_bytes < wql_beam_workspace_size(batch, beams, n) || !aligned(workspace, 256))
    return WQL_EWORKSPACE;
  BeamSelectArgs a{};
  a.logits = logits;
  a.dtype = dtype;
  a.batch = (int)batch;
  a.beams = (int)beams;
  a.n = (int)n;
  a.eos = eos;
  a.order = order;
  a.scores = scores;
  a.tokens = tokens_out;
  a.parents = parents_out;
  a.scores_out = scores_out;
  a.ended = ended_out;
  const BeamParts cut = beam_parts(batch * beams, n, dtype);
  a.parts = cut.parts;
  a.part_chunks = cut.chunks;
  a.stats = static_cast<float2*>(workspace);
  a.keys = reinterpret_cast<uint64_t*>(
      static_cast<unsigned char*>(workspace) +
      round_up((size_t)batch * beams * a.parts * sizeof(float2), 256));
  const cudaError_t e = launch_beam_select(a, stream);
  return e == cudaSuccess ? WQL_OK : cuda_fail(e);
}

wql_status wql_beam_reorder(const wql_state* states, int64_t count, const int32_t* parents,
                            int64_t batch, int64_t beams, const int32_t* lengths,
                            cudaStream_t stream) {
  if (count < 0 || batch < 0 || beams <= 0) return WQL_EINVAL;
  if ((count > 0 && !states) || (count > 0 && batch > 0 && !parents)) return WQL_EINVAL;
  if (beams > WQL_MAX_BEAMS || batch > 65535 || count > WQL_MAX_STATES) return WQL_EUNSUPPORTED;
  if (!aligned(parents, 4) || !aligned(lengths, 4)) return WQL_EUNSUPPORTED;
  constexpr int64_t kMaxStride = int64_t(1) << 40, kMaxSpan = int64_t(1) << 50,
                    kMaxBytes = (int64_t(1) << 32) - 1;
  for (int64_t i = 0; i < count; ++i) {
    const wql_state& s = states[i];
    if (s.outer < 0 || s.positions < 0 || s.position_bytes < 0 || s.row_stride < 0 ||
        s.outer_stride < 0 || s.position_stride < 0)
      return WQL_EINVAL;
    const bool empty = s.outer == 0 || s.positions == 0 || s.position_bytes == 0 || batch == 0;
    if (!empty && !s.data) return WQL_EINVAL;
    if (!empty && (s.outer_stride > kMaxSpan / s.outer || s.position_stride > kMaxSpan / s.positions ||
                   s.row_stride > kMaxSpan / (batch * beams)))
      return WQL_EUNSUPPORTED;
    if (s.row_stride >= kMaxStride || s.outer_stride >= kMaxStride || s.position_stride >= kMaxStride)
      return WQL_EUNSUPPORTED;
    if (!empty && (s.outer > kMaxBytes / s.positions ||
                   s.outer * s.positions > kMaxBytes / s.position_bytes))
      return WQL_EUNSUPPORTED;
  }
  if (count == 0 || batch == 0) return WQL_OK;
  if (states_overlap(states, count, batch * beams)) return WQL_EINVAL;
  if (beams == 1) return WQL_OK;
  const cudaError_t e = launch_beam_reorder(states, count, parents, (int)batch, (int)beams, lengths,
                                            stream);
  return e == cudaSuccess ? WQL_OK : cuda_fail(e);
}

wql_status wql_debug_set_waits(int64_t budget_cycles, int32_t stall_mma) {
  if (budget_cycles < 0 || (stall_mma != 0 && stall_mma != 1)) return WQL_EINVAL;
  g_wait_budget.store(budget_cycles, std::memory_order_relaxed);
  g_stall_mma.store(stall_mma, std::memory_order_relaxed);
  return WQL_OK;
}

}  // extern "C"
