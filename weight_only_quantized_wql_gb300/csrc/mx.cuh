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
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t b =
        __nv_cvt_float2_to_fp4x2(make_float2(v[2 * i], v[2 * i + 1]), __NV_E2M1, cudaRoundNearest);
    w |= (b & 0xFFu) << (8 * i);
  }
  return w;
}
__device__ __forceinline__ uint2 mx_codes_fp8(const float (&v)[8]) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * h], v[4 * h + 1]),
                                                 __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * h + 2], v[4 * h + 3]),
                                                 __NV_SATFINITE, __NV_E4M3);
    w[h] = (lo & 0xFFFFu) | (hi << 16);
  }
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void mx_values_fp4(uint32_t w, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h =
        __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)((w >> (8 * i)) & 0xFFu), __NV_E2M1);
    const float2 f = __half22float2(__half2(h));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void mx_values_fp8(uint2 w, float (&v)[8]) {
  const uint32_t p[2] = {w.x, w.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        (__nv_fp8x2_storage_t)((p[i >> 1] >> (16 * (i & 1))) & 0xFFFFu), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

// max(|a|, |b|), NaN if either is.
__device__ __forceinline__ float mx_max_abs(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}

// A group of four consecutive lanes holds a block, eight values each: encode
// this lane's eight (`x` in fp32) and return the block's scale byte.
template <int FMT>
__device__ __forceinline__ uint32_t mx_encode8(const float (&x)[8], uint2* codes) {
  const float m = mx_max_abs(mx_max_abs(mx_max_abs(x[0], x[1]), mx_max_abs(x[2], x[3])),
                             mx_max_abs(mx_max_abs(x[4], x[5]), mx_max_abs(x[6], x[7])));
  uint32_t am = __float_as_uint(m) & 0x7FFFFFFFu;
  am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
  am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
  const uint32_t byte = mx_scale_byte<FMT>(am);
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
};
cudaError_t launch_sample(const SampleArgs& a, cudaStream_t s);

}  // namespace wql
