// norm.cu -- residual addition and root-mean-square norm in front of the
// head: h = x + residual, y = h * rsqrt(mean(h^2) + eps) * gamma, written in
// 16 bits, in e4m3 with a scale per row, or in microscaled codes.
//
// HBM-bound: 2 bytes each of x, residual and residual_out and 2, 1 or 17/32
// bytes of y an element.  One block per row: the row stays in registers
// between the sum of squares and the output, so every byte moves once.  Sums
// and the norm are fp32; y is rounded once, to the output.  Measured: 4096 x 5120
// bf16 to 16 bits 26.6 us (93 % of the copy rate), to e4m3 25.7 us (84 %), to
// microscaled e4m3 25.8 us (84 %), to e2m1 25.1 us (80 %); 1 x 1024 1.8 us, 32 x 5120
// to microscaled e4m3 2.6 us.
// Where a thread holds 64 elements (rows of more than 16384 when there are many,
// else of more than 32768) the 64 registers of a 1024-thread block spill, 236 to 456
// bytes a thread: 512 x 16384 bf16 to 16 bits takes 16.4 us (60 %), 512 x 16416 26.8
// us (37 %), 512 x 65536 70.5 us (56 %).  By elements the spill is 2376 to 2660
// bytes: 512 x 4096 off a 16-byte boundary takes 6.4 us, 512 x 16384 53 us, 512 x
// 65536 431 us (9 %).
#include "mx.cuh"

namespace wql {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int kMaxRagged = 65536 - 16;   // its groups may be two more than k / 8

// Sum or maximum over the block; every thread gets it.
template <bool MAX>
__device__ __forceinline__ float block_reduce(float v, float* red) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) {
    const float o = __shfl_xor_sync(0xFFFFFFFFu, v, m);
    // NaN-keeping maximum of non-negative values: their bits order, NaN on top
    v = MAX ? __uint_as_float(max(__float_as_uint(v), __float_as_uint(o))) : v + o;
  }
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;
  __syncthreads();                       // the buffer of an earlier reduction is free
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = (threadIdx.x & 31) < warps ? red[threadIdx.x & 31] : 0.f;
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) {
    const float o = __shfl_xor_sync(0xFFFFFFFFu, v, m);
    v = MAX ? __uint_as_float(max(__float_as_uint(v), __float_as_uint(o))) : v + o;
  }
  return v;
}

// max(a, |v|) for a >= 0, NaN if either is.
__device__ __forceinline__ float max_abs(float a, float v) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(v)));
  return r;
}

// One group of W consecutive elements: W = 8 as one 16-byte access, else
// single elements.
template <typename T, int W>
__device__ __forceinline__ void load_group(const T* p, float (&v)[W]) {
  if constexpr (W == 8) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const T* h = reinterpret_cast<const T*>(&a);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32(h[i]);
  } else {
    v[0] = to_f32(*p);
  }
}
template <typename T, int W>
__device__ __forceinline__ void store_group(T* p, const float (&v)[W]) {
  if constexpr (W == 8) {
    uint4 a;
    T* h = reinterpret_cast<T*>(&a);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = from_f32<T>(v[i]);
    *reinterpret_cast<uint4*>(p) = a;
  } else {
    *p = from_f32<T>(v[0]);
  }
}

// Scale bytes of a row past m in the last tile: zero.
__device__ __forceinline__ void pad_scales(const NormArgs& a, int64_t row) {
  const int tile_cols = (a.k + 127) / 128;
  for (int t = threadIdx.x; t < tile_cols; t += blockDim.x)
    *reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(a.scales) +
                                 mx_scale_at(row, t, tile_cols)) = 0u;
}

// A thread holds G groups of W elements: group g of the row is thread
// g % threads, slot g / threads.  W = 8: 16-byte accesses, for 16-byte aligned
// tensors; without RAGGED k % 8 == 0, with it groups start on 16-byte
// addresses, `mis` elements before the row's first one, and those at the ends
// (which share their 16 bytes with other rows) go element by element.  W = 1
// takes any alignment.  (2000 x 4099 fp16 took 34.9 us by elements.)
template <typename T, int OUT, int W, int G, bool RAGGED>
__global__ void __launch_bounds__(kMaxThreads) add_rmsnorm_kernel(const NormArgs a) {
  __shared__ float red[32];
  griddep_launch_dependents();
  griddep_wait();
  const int64_t row = blockIdx.x;
  if constexpr (OUT >= WQL_NORM_MX_FP8) {
    if (row >= a.m) {
      pad_scales(a, row);
      return;
    }
  }
  const int mis = RAGGED ? (int)((row * a.k) & 7) : 0;
  const int groups = RAGGED ? (a.k + mis + 7) / 8 : a.k / W;
  const T* x = reinterpret_cast<const T*>(a.x) + row * a.k - mis;
  const T* res = a.residual ? reinterpret_cast<const T*>(a.residual) + row * a.k - mis : nullptr;
  const T* gamma = reinterpret_cast<const T*>(a.gamma) - mis;
  // is group g all inside the row; is its element i
  auto whole = [&](int g) { return !RAGGED || (g * 8 >= mis && g * 8 + 8 <= a.k + mis); };
  auto inside = [&](int g, int i) { return g * 8 + i >= mis && g * 8 + i < a.k + mis; };
  auto load = [&](const T* p, int g, float (&v)[W]) {
    if (whole(g)) {
      load_group<T, W>(p + (size_t)g * W, v);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) v[i] = inside(g, i) ? to_f32(p[(size_t)g * W + i]) : 0.f;
    }
  };
  auto store = [&](void* out, int g, const float (&v)[W]) {
    T* p = reinterpret_cast<T*>(out) + row * a.k - mis + (size_t)g * W;
    if (whole(g)) {
      store_group<T, W>(p, v);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i)
        if (inside(g, i)) p[i] = from_f32<T>(v[i]);
    }
  };
  float h[G][W];
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < G; ++j) {
    const int g = j * blockDim.x + threadIdx.x;
#pragma unroll
    for (int i = 0; i < W; ++i) h[j][i] = 0.f;
    if (g < groups) load(x, g, h[j]);
  }
  if (res) {
#pragma unroll
    for (int j = 0; j < G; ++j) {
      const int g = j * blockDim.x + threadIdx.x;
      float r[W];
      if (g < groups) {
        load(res, g, r);
#pragma unroll
        for (int i = 0; i < W; ++i) h[j][i] += r[i];
      }
    }
  }
#pragma unroll
  for (int j = 0; j < G; ++j)
#pragma unroll
    for (int i = 0; i < W; ++i) sum = fmaf(h[j][i], h[j][i], sum);
  // (every thread's loads of the row precede this reduction's barrier and
  // every store follows it, so out and residual_out may be x or residual;
  // a one-warp block converges at the shuffles)
  sum = block_reduce<false>(sum, red);
  const float scale = rsqrtf(sum / (float)a.k + a.eps);
  float amax = 0.f;
#pragma unroll
  for (int j = 0; j < G; ++j) {
    const int g = j * blockDim.x + threadIdx.x;
    if (g < groups) {
      if (a.residual_out) store(a.residual_out, g, h[j]);
      float gm[W];
      if constexpr (RAGGED) {             // gamma starts on its own boundary: by elements
#pragma unroll
        for (int i = 0; i < W; ++i) gm[i] = inside(g, i) ? to_f32(gamma[g * W + i]) : 0.f;
      } else {
        load_group<T, W>(gamma + (size_t)g * W, gm);
      }
#pragma unroll
      for (int i = 0; i < W; ++i) {
        h[j][i] = h[j][i] * scale * gm[i];
        if constexpr (OUT == WQL_NORM_E4M3)
          amax = max_abs(amax, h[j][i]);
      }
    }
  }
  if constexpr (OUT == WQL_NORM_SAME) {
#pragma unroll
    for (int j = 0; j < G; ++j) {
      const int g = j * blockDim.x + threadIdx.x;
      if (g < groups) store(a.out, g, h[j]);
    }
  } else if constexpr (OUT == WQL_NORM_E4M3) {
    amax = block_reduce<true>(amax, red);
    const float s0 = __fmul_rn(amax, 1.0f / 448.0f);
    const float s = s0 < 1e-8f ? 1e-8f : s0;          // (a NaN stays)
    const float inv = __fdiv_rn(1.f, s);
    if (threadIdx.x == 0) reinterpret_cast<float*>(a.scales)[row] = s;
    uint8_t* out = reinterpret_cast<uint8_t*>(a.out) + row * a.k - mis;
#pragma unroll
    for (int j = 0; j < G; ++j) {
      const int g = j * blockDim.x + threadIdx.x;
      if (g >= groups) continue;
      if constexpr (W == 8) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = h[j][i] * inv;
        const uint2 q = mx_codes_fp8(v);
        if (whole(g)) {
          *reinterpret_cast<uint2*>(out + (size_t)g * 8) = q;
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (inside(g, i))
              out[(size_t)g * 8 + i] = (uint8_t)((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
        }
      } else {
        out[g] = (uint8_t)__nv_cvt_float_to_fp8(h[j][0] * inv, __NV_SATFINITE, __NV_E4M3);
      }
    }
  } else {
    static_assert(W == 8 || OUT < WQL_NORM_MX_FP8, "microscaled rows are whole 8-element groups");
    constexpr int FMT = OUT == WQL_NORM_MX_FP4 ? WQL_MX_FP4 : WQL_MX_FP8;
    const int tile_cols = (a.k + 127) / 128;
#pragma unroll
    for (int j = 0; j < G; ++j) {
      // four lanes hold a block, a half warp one tile column (blockDim is a
      // multiple of 32, so group g is lane g % 32); groups past the row are
      // zeros with scale 0
      const int g = j * blockDim.x + threadIdx.x;
      uint2 q;
      const uint32_t byte = mx_encode8<FMT>(h[j], mx_amax8(h[j]), &q);
      if (g < groups) {
        const size_t vec = (size_t)row * groups + g;
        if constexpr (FMT == WQL_MX_FP4)
          reinterpret_cast<uint32_t*>(a.out)[vec] = q.x;
        else
          reinterpret_cast<uint2*>(a.out)[vec] = q;
      }
      if ((threadIdx.x & 3) == 0 && (g >> 4) < tile_cols)
        reinterpret_cast<uint8_t*>(a.scales)[mx_scale_at(row, g >> 4, tile_cols) +
                                             ((g >> 2) & 3)] = (uint8_t)byte;
    }
  }
}

template <typename T, int OUT, int W, int G, bool RAGGED>
cudaError_t launch_g(const NormArgs& a, int threads, cudaStream_t s) {
  const int rows = OUT >= WQL_NORM_MX_FP8
                       ? (a.m + kMxTileRows - 1) / kMxTileRows * kMxTileRows : a.m;
  const cudaError_t e =
      launch_pdl(add_rmsnorm_kernel<T, OUT, W, G, RAGGED>, dim3((unsigned)rows), dim3(threads), 0, s, a);
  note_launch();
  return e;
}

template <typename T, int OUT, int W, bool RAGGED = false>
cudaError_t launch_w(const NormArgs& a, cudaStream_t s) {
  // Threads per row: few rows want all their loads out at once (1 x 5120: 640
  // threads, one group each), many rows several loads per thread (4096 x 5120
  // to e4m3: 25.9 us with at most 512 threads, 29.2 with 256, 29.0 with 1024).
  const int groups = RAGGED ? a.k / W + 2 : a.k / W;
  const int most = a.m < 2 * device_sm_count() ? kMaxThreads : 512;
  int g = 1;
  while (g < 64 / W && groups > most * g) g *= 2;
  int threads = ((groups + g - 1) / g + 31) / 32 * 32;
  if (threads > kMaxThreads) return cudaErrorInvalidConfiguration;
  if constexpr (W == 8) {
    switch (g) {
      case 1: return launch_g<T, OUT, W, 1, RAGGED>(a, threads, s);
      case 2: return launch_g<T, OUT, W, 2, RAGGED>(a, threads, s);
      case 4: return launch_g<T, OUT, W, 4, RAGGED>(a, threads, s);
      default: return launch_g<T, OUT, W, 8, RAGGED>(a, threads, s);
    }
  } else {
    switch (g) {
      case 1: return launch_g<T, OUT, W, 1, RAGGED>(a, threads, s);
      case 2: return launch_g<T, OUT, W, 2, RAGGED>(a, threads, s);
      case 4: return launch_g<T, OUT, W, 4, RAGGED>(a, threads, s);
      case 8: return launch_g<T, OUT, W, 8, RAGGED>(a, threads, s);
      case 16: return launch_g<T, OUT, W, 16, RAGGED>(a, threads, s);
      case 32: return launch_g<T, OUT, W, 32, RAGGED>(a, threads, s);
      default: return launch_g<T, OUT, W, 64, RAGGED>(a, threads, s);
    }
  }
}

template <typename T>
cudaError_t launch_t(const NormArgs& a, cudaStream_t s) {
  auto ok = [](const void* p, size_t al) { return (reinterpret_cast<uintptr_t>(p) % al) == 0; };
  const bool wide = ok(a.x, 16) && ok(a.residual, 16) && ok(a.residual_out, 16) &&
                    ok(a.out, a.out_format == WQL_NORM_E4M3 ? 8 : 16);
  const bool even = wide && a.k % 8 == 0 && ok(a.gamma, 16);
  const bool ragged = wide && a.k <= kMaxRagged;
  switch (a.out_format) {
    case WQL_NORM_SAME:
      return even ? launch_w<T, WQL_NORM_SAME, 8>(a, s)
             : ragged ? launch_w<T, WQL_NORM_SAME, 8, true>(a, s) : launch_w<T, WQL_NORM_SAME, 1>(a, s);
    case WQL_NORM_E4M3:
      return even ? launch_w<T, WQL_NORM_E4M3, 8>(a, s)
             : ragged ? launch_w<T, WQL_NORM_E4M3, 8, true>(a, s) : launch_w<T, WQL_NORM_E4M3, 1>(a, s);
    case WQL_NORM_MX_FP8: return launch_w<T, WQL_NORM_MX_FP8, 8>(a, s);
    default: return launch_w<T, WQL_NORM_MX_FP4, 8>(a, s);
  }
}

}  // namespace

cudaError_t launch_add_rmsnorm(const NormArgs& a, cudaStream_t s) {
  return a.dtype == WQL_F16 ? launch_t<__half>(a, s) : launch_t<__nv_bfloat16>(a, s);
}

}  // namespace wql
