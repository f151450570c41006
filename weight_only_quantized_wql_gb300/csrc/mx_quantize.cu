// mx_quantize.cu -- microscaled codes from dense rows, and back.
//
// Per block of 32 columns: scale 2^e with e = floor(log2 max|x|) - emax (2 for
// e2m1, 8 for e4m3), codes x / 2^e rounded to nearest even.  Division by a
// power of two is exact, so the only rounding is the code's.
//
// HBM-bound: quantising reads 2 (4) bytes an element and writes 17/32 (FP4)
// or 33/32 (FP8).  Quantising, a thread takes sixteen columns (two 16-byte
// loads of 16-bit input), two lanes a block, eight lanes one scale tile's row
// (128 columns); with eight columns a thread it was bound by instructions
// (151936 x 1024 fp16 to e2m1 and back 128 us).  Dequantising, a thread takes
// eight columns.  Loads of several tiles are in flight per thread before the
// first is used; rows and tiles come from a multiplication by the reciprocal of
// the tile count.  Measured: 151936 x 1024 fp16 to e2m1 60.7 us (6.5 TB/s), back 58.8
// us (6.7 TB/s), one after the other 118.6 us; 4096 x 5120 bf16 to e4m3 and back 19.3
// us.
#include <type_traits>

#include "mx.cuh"

namespace wql {
namespace {

constexpr int kThreads = 256;
constexpr int kLanes = 8;                    // quantising: lanes per row of a scale tile
constexpr int kTeams = kThreads / kLanes;
constexpr int kTilesAhead = 2;               // per thread
constexpr int kHalfWarps = kThreads / 16;    // dequantising: the lanes per row are 16
constexpr int kUnroll = 4;

// Eight consecutive elements as loaded, their values, and the float bits of the
// largest magnitude (NaNs on top; 16-bit types two at a time).
template <typename T> struct Eight {
  uint4 raw;
  __device__ __forceinline__ void load(const T* p) { raw = ldg_stream_u4(p); }
  __device__ __forceinline__ void clear() { raw = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    const T* h = reinterpret_cast<const T*>(&raw);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32(h[i]);
  }
  __device__ __forceinline__ uint32_t amax(const float (&)[8]) const {
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2,
                                         __nv_bfloat162>::type;
    const T2* h = reinterpret_cast<const T2*>(&raw);
    const T2 m = __hmax2_nan(__hmax2_nan(__habs2(h[0]), __habs2(h[1])),
                             __hmax2_nan(__habs2(h[2]), __habs2(h[3])));
    return __float_as_uint(to_f32(__hmax_nan(m.x, m.y))) & 0x7FFFFFFFu;
  }
};
template <> struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  __device__ __forceinline__ uint32_t amax(const float (&v)[8]) const { return mx_amax8(v); }
};

// item / tile_cols, for items < 8 tile_cols + 64: exact with recip =
// ceil(2^32 / tile_cols) while item * tile_cols < 2^32 (tile_cols <= 2^13)
__device__ __forceinline__ int row_of(int item, int tile_cols, uint32_t recip) {
  return tile_cols == 1 ? item : (int)__umulhi((uint32_t)item, recip);
}
uint32_t recip_of(int tile_cols) {
  return (uint32_t)(((1ull << 32) + (uint64_t)tile_cols - 1) / (uint64_t)tile_cols);
}
static_assert(kMxMaxK / 128 <= 1 << 13, "row_of()");

// A block of threads takes `rows_per_cta` rows (of the rows padded to 128, so
// that every byte of the scale tiles is written) and all their tile columns.
template <typename T, int FMT>
__global__ void __launch_bounds__(kThreads)
    mx_quantize_kernel(const MxQuantizeArgs a, int tile_cols, uint32_t recip, int padded_rows,
                       int rows_per_cta) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & (kLanes - 1), team = threadIdx.x / kLanes;
  const int row0 = blockIdx.x * rows_per_cta;
  const int items = min(rows_per_cta, padded_rows - row0) * tile_cols;
  const T* x = reinterpret_cast<const T*>(a.x);
  // every warp makes the same number of passes (the shuffles need whole warps)
  for (int i0 = 0; i0 < items; i0 += kTilesAhead * kTeams) {
    Eight<T> x8[kTilesAhead][2];
    int row[kTilesAhead], tc[kTilesAhead];
    bool in[kTilesAhead];
#pragma unroll
    for (int u = 0; u < kTilesAhead; ++u) {
      const int item = i0 + u * kTeams + team;
      const int r = row_of(item, tile_cols, recip);
      row[u] = row0 + r;
      tc[u] = item - r * tile_cols;
      const int col = tc[u] * 128 + lane * 16;
      in[u] = item < items && row[u] < a.rows && col < a.k;
      x8[u][0].clear();
      x8[u][1].clear();
      if (in[u]) {
        const T* p = x + (size_t)row[u] * a.k + col;
        x8[u][0].load(p);
        x8[u][1].load(p + 8);
      }
    }
#pragma unroll
    for (int u = 0; u < kTilesAhead; ++u) {
      const int item = i0 + u * kTeams + team;
      float v[2][8];
      x8[u][0].values(v[0]);
      x8[u][1].values(v[1]);
      uint32_t amax = max(x8[u][0].amax(v[0]), x8[u][1].amax(v[1]));
      amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
      const uint32_t byte = mx_scale_byte<FMT>(amax);
      const float inv = mx_inverse(byte);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[h][j] *= inv;
      if (in[u]) {
        const size_t vec = ((size_t)row[u] * a.k + tc[u] * 128 + lane * 16) / 16;
        if constexpr (FMT == WQL_MX_FP4) {
          const uint2 q = make_uint2(mx_codes_fp4(v[0]), mx_codes_fp4(v[1]));
          reinterpret_cast<uint2*>(a.codes)[vec] = byte == 255u ? make_uint2(0u, 0u) : q;
        } else {
          const uint2 q0 = mx_codes_fp8(v[0]), q1 = mx_codes_fp8(v[1]);
          reinterpret_cast<uint4*>(a.codes)[vec] = make_uint4(q0.x, q0.y, q1.x, q1.y);
        }
      }
      if ((lane & 1) == 0 && item < items)
        reinterpret_cast<uint8_t*>(a.scales)[mx_scale_at(row[u], tc[u], tile_cols) +
                                             (lane >> 1)] = (uint8_t)byte;
    }
  }
}

template <typename T, int FMT>
__global__ void __launch_bounds__(kThreads)
    mx_dequantize_kernel(const MxDequantizeArgs a, int tile_cols, uint32_t recip,
                         int rows_per_cta) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 15, hw = threadIdx.x >> 4;
  const int row0 = blockIdx.x * rows_per_cta;
  const int items = min(rows_per_cta, a.rows - row0) * tile_cols;
  const uint8_t* scales = reinterpret_cast<const uint8_t*>(a.scales);
  for (int i0 = 0; i0 < items; i0 += kUnroll * kHalfWarps) {
    uint2 q[kUnroll];
    uint32_t sw[kUnroll];
    int row[kUnroll], col[kUnroll];
    bool in[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int item = i0 + u * kHalfWarps + hw;
      const int r = row_of(item, tile_cols, recip);
      row[u] = row0 + r;
      const int tc = item - r * tile_cols;
      col[u] = tc * 128 + lane * 8;
      in[u] = item < items && col[u] < a.k;
      q[u] = make_uint2(0u, 0u);
      sw[u] = 0u;
      if (in[u]) {
        const size_t vec = ((size_t)row[u] * a.k + col[u]) / 8;
        if constexpr (FMT == WQL_MX_FP4)
          q[u].x = __ldg(reinterpret_cast<const uint32_t*>(a.codes) + vec);
        else
          q[u] = __ldg(reinterpret_cast<const uint2*>(a.codes) + vec);
        sw[u] = __ldg(reinterpret_cast<const uint32_t*>(
            scales + mx_scale_at(row[u], tc, tile_cols)));
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (!in[u]) continue;
      const uint32_t byte = (sw[u] >> (8 * (lane >> 2))) & 0xFFu;
      uint32_t h[4];
      if constexpr (FMT == WQL_MX_FP4)
        mx_halves_fp4(q[u].x, h);
      else
        mx_halves_fp8(q[u], h);
      T* dst = reinterpret_cast<T*>(a.out) + (size_t)row[u] * a.k + col[u];
      if constexpr (std::is_same<T, __half>::value) {
        // 2^-24 .. 2^15 are fp16 numbers: the product rounds once, as from fp32
        if (byte >= 103u && byte <= 142u) {
          const __half2 s = __half2half2(__float2half_rn(mx_scale_value(byte)));
          uint4 o;
          __half2* o2 = reinterpret_cast<__half2*>(&o);
#pragma unroll
          for (int j = 0; j < 4; ++j) o2[j] = __hmul2(*reinterpret_cast<const __half2*>(&h[j]), s);
          *reinterpret_cast<uint4*>(dst) = o;
          continue;
        }
      }
      const float s = mx_scale_value(byte);
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
        v[2 * j] = f.x * s;
        v[2 * j + 1] = f.y * s;
      }
      if constexpr (sizeof(T) == 4) {
        reinterpret_cast<float4*>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
      } else {
        uint4 o;
        T* t = reinterpret_cast<T*>(&o);
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] = from_f32<T>(v[j]);
        *reinterpret_cast<uint4*>(dst) = o;
      }
    }
  }
}

// Rows per block: enough blocks for a few per SM, at most 8 rows each.
int rows_per_cta(int rows) {
  const int r = rows / (device_sm_count() * 8);
  return r < 1 ? 1 : r > 8 ? 8 : r;
}

template <typename T>
cudaError_t quantize_t(const MxQuantizeArgs& a, cudaStream_t s) {
  const int tile_cols = (int)mx_tile_cols(a.k);
  const int padded = (a.rows + kMxTileRows - 1) / kMxTileRows * kMxTileRows;
  const int rpc = rows_per_cta(padded);
  const dim3 grid((padded + rpc - 1) / rpc);
  const cudaError_t e =
      a.format == WQL_MX_FP4
          ? launch_pdl(mx_quantize_kernel<T, WQL_MX_FP4>, grid, dim3(kThreads), 0, s, a, tile_cols,
                       recip_of(tile_cols), padded, rpc)
          : launch_pdl(mx_quantize_kernel<T, WQL_MX_FP8>, grid, dim3(kThreads), 0, s, a, tile_cols,
                       recip_of(tile_cols), padded, rpc);
  note_launch();
  return e;
}

template <typename T>
cudaError_t dequantize_t(const MxDequantizeArgs& a, cudaStream_t s) {
  const int tile_cols = (int)mx_tile_cols(a.k);
  const int rpc = rows_per_cta(a.rows);
  const dim3 grid((a.rows + rpc - 1) / rpc);
  const cudaError_t e =
      a.format == WQL_MX_FP4
          ? launch_pdl(mx_dequantize_kernel<T, WQL_MX_FP4>, grid, dim3(kThreads), 0, s, a,
                       tile_cols, recip_of(tile_cols), rpc)
          : launch_pdl(mx_dequantize_kernel<T, WQL_MX_FP8>, grid, dim3(kThreads), 0, s, a,
                       tile_cols, recip_of(tile_cols), rpc);
  note_launch();
  return e;
}

}  // namespace

cudaError_t launch_mx_quantize(const MxQuantizeArgs& a, cudaStream_t s) {
  switch (a.x_dtype) {
    case WQL_F32: return quantize_t<float>(a, s);
    case WQL_F16: return quantize_t<__half>(a, s);
    default: return quantize_t<__nv_bfloat16>(a, s);
  }
}

cudaError_t launch_mx_dequantize(const MxDequantizeArgs& a, cudaStream_t s) {
  switch (a.out_dtype) {
    case WQL_F32: return dequantize_t<float>(a, s);
    case WQL_F16: return dequantize_t<__half>(a, s);
    default: return dequantize_t<__nv_bfloat16>(a, s);
  }
}

}  // namespace wql
