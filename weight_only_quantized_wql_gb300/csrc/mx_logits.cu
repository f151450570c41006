// mx_logits.cu -- logits of a microscaled head: X (e4m3 or e2m1) times W^T
// (e2m1), both in blocks of 32 with power-of-two scales.
//
// The simplest form: a block of 256 threads computes 64 vocab rows x 16
// tokens, decoding 128 columns at a time into shared memory as fp32.
#include "mx.cuh"

namespace wql {
namespace {

constexpr int kRows = 64, kTokens = 16, kCols = 128, kThreads = 256;

template <int XFMT, typename OT>
__global__ void __launch_bounds__(kThreads) mx_logits_kernel(const MxLogitsArgs a) {
  __shared__ float ws[kRows][kCols + 1];
  __shared__ float xs[kTokens][kCols + 1];
  griddep_launch_dependents();
  griddep_wait();
  const int row0 = blockIdx.x * kRows, tok0 = blockIdx.y * kTokens;
  const int tile_cols = (a.k + 127) / 128;
  const int r = threadIdx.x % kRows, t4 = threadIdx.x / kRows;   // row, tokens t4 + 4 i
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int tc = 0; tc < tile_cols; ++tc) {
    __syncthreads();
    for (int i = threadIdx.x; i < (kRows + kTokens) * (kCols / 8); i += kThreads) {
      const int rr = i / (kCols / 8), c = (i % (kCols / 8)) * 8, col = tc * kCols + c;
      const bool is_w = rr < kRows;
      const int row = is_w ? row0 + rr : tok0 + rr - kRows;
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      float s = 0.f;
      if (row < (is_w ? a.n : a.m) && col < a.k) {
        const size_t vec = ((size_t)row * a.k + col) / 8;
        if (is_w)
          mx_values_fp4(__ldg(reinterpret_cast<const uint32_t*>(a.w_codes) + vec), v);
        else if (XFMT == WQL_MX_FP4)
          mx_values_fp4(__ldg(reinterpret_cast<const uint32_t*>(a.x_codes) + vec), v);
        else
          mx_values_fp8(__ldg(reinterpret_cast<const uint2*>(a.x_codes) + vec), v);
        s = mx_scale_value(reinterpret_cast<const uint8_t*>(
            is_w ? a.w_scales : a.x_scales)[mx_scale_at(row, tc, tile_cols) + c / kMxBlock]);
      }
      float* dst = is_w ? &ws[rr][c] : &xs[rr - kRows][c];
#pragma unroll
      for (int j = 0; j < 8; ++j) dst[j] = v[j] * s;
    }
    __syncthreads();
    for (int c = 0; c < kCols; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = fmaf(ws[r][c], xs[t4 + 4 * i][c], acc[i]);
  }
  const int row = row0 + r;
  if (row >= a.n) return;
  const float b = a.bias ? to_f32(reinterpret_cast<const OT*>(a.bias)[row]) : 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int tok = tok0 + t4 + 4 * i;
    if (tok < a.m) reinterpret_cast<OT*>(a.out)[(size_t)tok * a.n + row] = from_f32<OT>(acc[i] + b);
  }
}

template <int XFMT, typename OT>
cudaError_t launch_t(const MxLogitsArgs& a, cudaStream_t s) {
  const dim3 grid((a.n + kRows - 1) / kRows, (a.m + kTokens - 1) / kTokens);
  const cudaError_t e =
      launch_pdl(mx_logits_kernel<XFMT, OT>, grid, dim3(kThreads), 0, s, a);
  note_launch();
  return e;
}

}  // namespace

cudaError_t launch_mx_logits(const MxLogitsArgs& a, cudaStream_t s) {
  if (a.x_format == WQL_MX_FP4)
    return a.out_dtype == WQL_F16 ? launch_t<WQL_MX_FP4, __half>(a, s)
                                  : launch_t<WQL_MX_FP4, __nv_bfloat16>(a, s);
  return a.out_dtype == WQL_F16 ? launch_t<WQL_MX_FP8, __half>(a, s)
                                : launch_t<WQL_MX_FP8, __nv_bfloat16>(a, s);
}

}  // namespace wql
