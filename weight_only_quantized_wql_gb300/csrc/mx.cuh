// mx.cuh -- microscaled codes (blocks of 32 columns, a power-of-two scale):
// the arithmetic of a block, the place of a scale, and the launchers that the
// C-ABI layer calls.
#pragma once

#include <cuda.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "wql_common.cuh"

namespace wql {

constexpr int kMxBlock = 32;        // columns per scale
constexpr int kMxTileRows = 128;    // a scale tile: 128 rows x 4 blocks, 512 bytes
constexpr int kMxTileBytes = 512;
constexpr int kMxMaxK = 1 << 20;

__host__ __device__ __forceinline__ int64_t mx_tile_cols(int64_t k) { return (k + 127) / 128; }

// Byte of the first block of (row, tile column) in the scale tiles; the
// tile's other three blocks follow it.
__device__ __forceinline__ size_t mx_scale_at(int64_t row, int tile_col, int tile_cols) {
  return ((size_t)(row >> 7) * tile_cols + tile_col) * kMxTileBytes +
         (size_t)((row & 31) * 16 + ((row >> 5) & 3) * 4);
}

// Scale byte of a block whose largest |x| has these float bits (NaNs order
// above infinity): the exponent, less that of the largest element; 255 = NaN.
template <int FMT>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
  constexpr int kEmax = FMT == WQL_MX_FP4 ? 2 : 8;
  if (amax_bits >= 0x7F800000u) return 255u;
  return (uint32_t)max((int)(amax_bits >> 23) - kEmax, 0);
}

// 1 / 2^(byte - 127), exact (byte <= 252 here; a NaN block gives a NaN).
__device__ __forceinline__ float mx_inverse(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float((254u - byte) << 23);
}

// 2^(byte - 127): 2^-127 is a subnormal float.
__device__ __forceinline__ float mx_scale_value(uint32_t byte) {
  if (byte == 255u) return __uint_as_float(0x7FC00000u);
  return byte ? __uint_as_float(byte << 23) : __uint_as_float(0x00400000u);
}

// Eight values, already divided by the scale, to codes: 4 bytes (FP4, element
// 0 in the lowest nibble) or 8 (FP8); round to nearest even, saturating.
__device__ __forceinline__ uint32_t mx_codes_fp4(const float (&v)[8]) {
  uint32_t w;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(w)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return w;
}
__device__ __forceinline__ uint32_t mx_codes_fp8x4(float a, float b, float c, float d) {
  uint32_t w;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(w)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return w;
}
__device__ __forceinline__ uint2 mx_codes_fp8(const float (&v)[8]) {
  return make_uint2(mx_codes_fp8x4(v[0], v[1], v[2], v[3]), mx_codes_fp8x4(v[4], v[5], v[6], v[7]));
}

// Codes to their values as fp16 pairs (exact), element 0 in the low half of h[0].
__device__ __forceinline__ void mx_halves_fp4(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
__device__ __forceinline__ void mx_halves_fp8(uint2 w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b16 a, b, c, d;\n\t"
      "mov.b32 {a, b}, %4;\n\t"
      "mov.b32 {c, d}, %5;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t"
      "cvt.rn.f16x2.e4m3x2 %2, c;\n\t"
      "cvt.rn.f16x2.e4m3x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w.x), "r"(w.y));
}

// max(|a|, |b|), NaN if either is.
__device__ __forceinline__ float mx_max_abs(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}

// A group of four consecutive lanes holds a block, eight values each: encode
// this lane's eight (`x` in fp32, whose largest |x| has the float bits `amax`)
// and return the block's scale byte.
template <int FMT>
__device__ __forceinline__ uint32_t mx_encode8(const float (&x)[8], uint32_t amax, uint2* codes) {
  amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
  amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
  const uint32_t byte = mx_scale_byte<FMT>(amax);
  const float inv = mx_inverse(byte);
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = x[i] * inv;
  if constexpr (FMT == WQL_MX_FP4) {
    codes->x = byte == 255u ? 0u : mx_codes_fp4(v);
    codes->y = 0u;
  } else {
    *codes = mx_codes_fp8(v);
  }
  return byte;
}
__device__ __forceinline__ uint32_t mx_amax8(const float (&x)[8]) {
  const float m = mx_max_abs(mx_max_abs(mx_max_abs(x[0], x[1]), mx_max_abs(x[2], x[3])),
                             mx_max_abs(mx_max_abs(x[4], x[5]), mx_max_abs(x[6], x[7])));
  return __float_as_uint(m) & 0x7FFFFFFFu;
}

// Tensor map (host) of a row-major matrix of rows of row_bytes, seen as
// [blocks of columns][rows][one block], whose boxes of box_blocks x box_rows
// blocks land in shared memory as rows of 128 bytes, 128B-swizzled, block after
// block.  A block is 128 bytes of a row, or (spread) 64 bytes, 128 packed 4-bit
// codes, of which 16 (8 bytes) land at the start of every 16-byte unit.
// row_bytes: whole blocks; base 16-byte (spread: 32-byte) aligned.
cudaError_t make_tmap_blocks(CUtensorMap* map, bool spread, const void* base, uint64_t row_bytes,
                             uint64_t rows, uint32_t box_rows, uint32_t box_blocks);

struct MxQuantizeArgs {
  const void* x;
  int x_dtype;
  int rows, k;
  int format;
  void* codes;
  void* scales;
};
cudaError_t launch_mx_quantize(const MxQuantizeArgs& a, cudaStream_t s);

struct MxDequantizeArgs {
  const void* codes;
  const void* scales;
  int format;
  int rows, k;
  int out_dtype;
  void* out;
};
cudaError_t launch_mx_dequantize(const MxDequantizeArgs& a, cudaStream_t s);

struct MxLogitsArgs {
  const void* x_codes;
  const void* x_scales;
  int x_format;
  const void* w_codes;
  const void* w_scales;
  int m, n, k;
  const void* bias;           // [n] of out_dtype, or null
  int out_dtype;
  void* out;                  // [m, n]
  unsigned int* err;          // error word, or null
};
cudaError_t launch_mx_logits(const MxLogitsArgs& a, cudaStream_t s);

struct NormArgs {
  const void* x;
  const void* residual;       // or null
  const void* gamma;
  int dtype;
  int m, k;
  float eps;
  int out_format;             // wql_norm_out
  void* out;
  void* scales;
  void* residual_out;         // or null
};
cudaError_t launch_add_rmsnorm(const NormArgs& a, cudaStream_t s);

struct SampleArgs {
  const void* logits;
  int dtype;
  int m, n;
  const float* u;
  const float* temperature;   // null: 1
  const int32_t* top_k;       // null: off
  const float* top_p;         // null: off
  const float* min_p;         // null: off
  int32_t* ids;
  float* logp;                // or null
  long long wait_budget;      // SM cycles the wait for a slice's copies may take
  int diag_stall;             // diagnostics: that wait is for a barrier nothing arrives on
};
cudaError_t launch_sample(const SampleArgs& a, cudaStream_t s);

}  // namespace wql
