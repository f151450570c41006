// lora.cu -- low-rank adapters of many requests beside a shared projection:
//   out[m, n] = RN(y[m, n] + s_i * sum_j u[m, j] b[i, n, j]),
//   u[m, j]   = sum_k x[m, k] a[i, j, k],        i = ids[m].
//
// Two launches: lora_down_kernel makes u, lora_up_kernel adds its product.
// Tokens of one adapter are taken 16 at a time, the rows of one mma.sync
// m16n8k16; the work is far below what the tensor cores need to be fed from
// tensor memory for (16 to 64 operations a byte), so both kernels load their
// fragments from global memory straight into registers: which k a lane's
// 16 bytes stand for is free, as long as both operands agree.
#include "requests.cuh"

namespace wql {
namespace {

constexpr int kTokens = 256;             // a slice of tokens is grouped by adapter at a time
constexpr int kDownThreads = 256;
constexpr int kUpThreads = 128;
static_assert(kDownThreads == kTokens, "a thread looks at one token of the slice");

// D += A B, 16 x 8 x 16, 16-bit operands, fp32 sums.
template <typename T>
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                      uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <typename T> __device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const T a = from_f32<T>(lo), b = from_f32<T>(hi);
  return (uint32_t)*reinterpret_cast<const uint16_t*>(&a) |
         ((uint32_t)*reinterpret_cast<const uint16_t*>(&b) << 16);
}
template <typename T> __device__ __forceinline__ float low(uint32_t v) {
  const uint16_t h = (uint16_t)v;
  return to_f32(*reinterpret_cast<const T*>(&h));
}
template <typename T> __device__ __forceinline__ float high(uint32_t v) {
  const uint16_t h = (uint16_t)(v >> 16);
  return to_f32(*reinterpret_cast<const T*>(&h));
}

// The four ranks that lane t's share of chunk c holds.  Chunks come in pairs
// of 32 ranks, of which a lane has 8 in a row (16 bytes of b); a lone chunk of
// 16 gives each lane four.
template <int CHUNKS> __device__ __forceinline__ int first_rank(int c, int t) {
  return CHUNKS == 1 ? 4 * t : 32 * (c / 2) + 8 * t + 4 * (c & 1);
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
               ::: "memory");
}
// A float4 of shared memory of another block of the cluster.
__device__ __forceinline__ float4 remote_f4(const void* p, uint32_t rank) {
  uint32_t at;
  asm("mapa.shared::cluster.u32 %0, %1, %2;"
      : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
  return v;
}

// ---------------------------------------------------------------------------
// u: a cluster of `splits` blocks per token, which share the hidden columns.
// Of a slice's tokens with one adapter, in order, every sixteenth leads a
// group; the clusters of the others have nothing to do.  (Finding its group
// takes a block one comparison a thread; a sorted list would be another
// launch.)  u is written as the mma fragments that lora_up_kernel loads: per
// token, chunk and lane of four, the high parts of four ranks and what they
// leave of them, and the factor that the products are multiplied with.
// ---------------------------------------------------------------------------
template <typename T, int CHUNKS>
__global__ void __launch_bounds__(kDownThreads) lora_down_kernel(const LoraArgs a, int splits) {
  constexpr int kRank = 16 * CHUNKS, kTiles = 2 * CHUNKS, kWarps = kDownThreads / 32;
  constexpr int kBufs = CHUNKS == 8 ? 4 : kWarps;
  __shared__ alignas(16) float part[kBufs][16][kRank];
  __shared__ uint32_t mask[kTokens / 32];
  __shared__ int group[16];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int token = blockIdx.x / splits, split = blockIdx.x % splits;
  griddep_wait();
  griddep_launch_dependents();
  const int base = token / kTokens * kTokens, mine = token - base;
  const int id = a.ids[token];
  if ((uint32_t)id >= (uint32_t)a.count) return;
  const bool same = base + tid < a.m && a.ids[base + tid] == id;
  const uint32_t bits = __ballot_sync(0xFFFFFFFFu, same);
  if (lane == 0) mask[warp] = bits;
  if (tid < 16) group[tid] = -1;
  __syncthreads();
  int before = 0, lead = 0, total = 0;   // of this thread's token, of the cluster's, of the adapter
#pragma unroll
  for (int w = 0; w < kTokens / 32; ++w) {
    const uint32_t v = mask[w];
    const int all = __popc(v);
    total += all;
    before += w < warp ? all : w == warp ? __popc(v & ((1u << lane) - 1u)) : 0;
    lead += w < (mine >> 5) ? all : w == (mine >> 5) ? __popc(v & ((1u << (mine & 31)) - 1u)) : 0;
  }
  if (lead % 16 != 0) return;
  if (same && before >= lead && before < lead + 16) group[before - lead] = base + tid;
  __syncthreads();
  const int count = min(16, total - lead);

  const int g = lane >> 2, t = lane & 3;
  const T* x0 = g < count ? static_cast<const T*>(a.x) + (size_t)group[g] * a.k : nullptr;
  const T* x1 = g + 8 < count ? static_cast<const T*>(a.x) + (size_t)group[g + 8] * a.k : nullptr;
  const T* w = static_cast<const T*>(a.a) + (size_t)id * a.rank * a.k;
  float acc[kTiles][4];
#pragma unroll
  for (int i = 0; i < kTiles; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
  // units of 32 columns, 8 a lane, split evenly over the cluster's warps
  const int units = (a.k + 31) / 32, shares = splits * kWarps, share = split * kWarps + warp;
  const int u1 = (int)((long long)units * (share + 1) / shares);
#pragma unroll 4
  for (int u = (int)((long long)units * share / shares); u < u1; ++u) {
    const int col = u * 32 + 8 * t;
    const bool in = col < a.k;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const uint4 xa = in && x0 ? *reinterpret_cast<const uint4*>(x0 + col) : zero;
    const uint4 xb = in && x1 ? *reinterpret_cast<const uint4*>(x1 + col) : zero;
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      const int rank = 8 * i + g;
      const uint4 v = in && rank < a.rank
                          ? *reinterpret_cast<const uint4*>(w + (size_t)rank * a.k + col) : zero;
      mma16<T>(acc[i], xa.x, xb.x, xa.y, xb.y, v.x, v.y);
      mma16<T>(acc[i], xa.z, xb.z, xa.w, xb.w, v.z, v.w);
    }
  }

  // sums over the warps: part[b][token][rank]
  auto put = [&](int b) {
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      *reinterpret_cast<float2*>(&part[b][g][8 * i + 2 * t]) = make_float2(acc[i][0], acc[i][1]);
      *reinterpret_cast<float2*>(&part[b][g + 8][8 * i + 2 * t]) = make_float2(acc[i][2], acc[i][3]);
    }
  };
  if constexpr (kBufs < kWarps) {
    if (warp >= kBufs) put(warp - kBufs);
    __syncthreads();
    if (warp < kBufs) {
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        acc[i][0] += part[warp][g][8 * i + 2 * t];
        acc[i][1] += part[warp][g][8 * i + 2 * t + 1];
        acc[i][2] += part[warp][g + 8][8 * i + 2 * t];
        acc[i][3] += part[warp][g + 8][8 * i + 2 * t + 1];
      }
      put(warp);                       // (read and written by the same lanes)
    }
  } else {
    put(warp);
  }
  if (splits > 1) cluster_sync();
  else __syncthreads();
  // fragments of this block's share of the tokens: four ranks a thread
  constexpr int kFrags = 4 * CHUNKS;
  const int share_tokens = 16 / splits;
  const float scale = a.scale ? a.scale[id] : 1.f;
  for (int e = tid; e < share_tokens * kFrags; e += kDownThreads) {
    const int row = split * share_tokens + e / kFrags, f = e % kFrags;
    const int rank = first_rank<CHUNKS>(f >> 2, f & 3);
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = 0; c < splits; ++c) {
#pragma unroll
      for (int b = 0; b < kBufs; ++b) {
        const float4 v = splits > 1 ? remote_f4(&part[b][row][rank], (uint32_t)c)
                                    : *reinterpret_cast<const float4*>(&part[b][row][rank]);
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
      }
    }
    float factor = scale;
    float v[4] = {s.x, s.y, s.z, s.w};
    if constexpr (std::is_same<T, __half>::value) {
      // by a power of two to at most 2: fp16 holds neither a large u nor the
      // parts of a small one
      uint32_t top = 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t m = __float_as_uint(v[i]) & 0x7FFFFFFFu;
        if (m < 0x7F800000u) top = max(top, m);
      }
      const uint32_t lanes = (kFrags == 32 ? 0xFFFFFFFFu : (1u << (kFrags & 31)) - 1u)
                             << (lane / kFrags * kFrags);
#pragma unroll
      for (int d = 1; d < kFrags; d *= 2) top = max(top, __shfl_xor_sync(lanes, top, d));
      const int e2 = min(max((int)(top >> 23), 1), 253);      // biased; u = 0: anything
      const float down = __uint_as_float((uint32_t)(254 - e2) << 23);
      factor = scale * __uint_as_float((uint32_t)e2 << 23);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] *= down;
    }
    if (row >= count) continue;
    const int to = group[row];
    const uint4 q = [&] {
      uint4 r;
      r.x = pack2<T>(v[0], v[1]);
      r.y = pack2<T>(v[2], v[3]);
      const float h[4] = {low<T>(r.x), high<T>(r.x), low<T>(r.y), high<T>(r.y)};
      float l[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)       // an infinity or NaN leaves nothing
        l[i] = fabsf(h[i]) <= 3.4028235e38f ? v[i] - h[i] : 0.f;
      r.z = pack2<T>(l[0], l[1]);
      r.w = pack2<T>(l[2], l[3]);
      return r;
    }();
    a.u[(size_t)to * kFrags + f] = q;
    if (f == 0) a.factor[to] = factor;
  }
  if (splits > 1) cluster_sync();        // the others have read this block's sums
}

// ---------------------------------------------------------------------------
// out = y + factor * u b: a warp has 32 * UNITS columns for all tokens of a
// slice, grouped by adapter, so that it loads b once per adapter.  The mma's
// columns are dealt so that a lane ends up with 8 consecutive ones of a token:
// column j of n-tile i is 8 * (j / 2) + 2 i + j % 2 of the 32.
// ---------------------------------------------------------------------------
template <typename T, int CHUNKS, int UNITS, bool WIDE>
__global__ void __launch_bounds__(kUpThreads) lora_up_kernel(const LoraArgs a) {
  constexpr int kFrags = 4 * CHUNKS;
  constexpr uint32_t kNone = 0x7FFFFFu;
  __shared__ alignas(16) uint32_t key[kTokens], sorted[kTokens];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  griddep_launch_dependents();
  griddep_wait();
  const int base = blockIdx.y * kTokens, m = min(kTokens, a.m - base);
  // tokens ordered by adapter: (adapter, token) is unique, its place is the
  // number of smaller ones
  for (int i = tid; i < kTokens; i += kUpThreads) {
    const int id = i < m ? a.ids[base + i] : -1;
    key[i] = i < m ? ((uint32_t)id < (uint32_t)a.count ? (uint32_t)id : kNone) << 8 | (uint32_t)i
                   : 0xFFFFFFFFu;
  }
  __syncthreads();
  for (int i = tid; i < m; i += kUpThreads) {
    const uint32_t mine = key[i];
    int place = 0;
    for (int j = 0; j < m; j += 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(&key[j]);
      place += (v.x < mine) + (v.y < mine) + (v.z < mine) + (v.w < mine);
    }
    sorted[place] = mine;
  }
  __syncthreads();

  const long long col0 = (long long)blockIdx.x * (kUpThreads * UNITS) + warp * (32 * UNITS);
  if (col0 >= a.n) return;
  uint32_t b[UNITS][4][CHUNKS][2];
  uint32_t current = kNone;
  for (int p = 0; p < m;) {
    const uint32_t first = sorted[p], id = first >> 8;
    const bool like = lane < 16 && p + lane < m && (sorted[min(p + lane, m - 1)] >> 8) == id;
    const int count = __popc(__ballot_sync(0xFFFFFFFFu, like));
    if (id == kNone) {
      if (a.out == a.y) break;            // the last ones; nothing to add
    } else if (id != current) {
      current = id;
#pragma unroll
      for (int u = 0; u < UNITS; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const long long col = col0 + 32 * u + 8 * (g >> 1) + 2 * i + (g & 1);
          const T* row = static_cast<const T*>(a.b) + ((size_t)id * a.n + col) * a.rank;
          if constexpr (CHUNKS == 1) {
            const bool in = col < a.n && 4 * t < a.rank;
            const uint2 v = in ? *reinterpret_cast<const uint2*>(row + 4 * t) : make_uint2(0u, 0u);
            b[u][i][0][0] = v.x;
            b[u][i][0][1] = v.y;
          } else {
#pragma unroll
            for (int c = 0; c < CHUNKS; c += 2) {
              const bool in = col < a.n && 16 * c + 8 * t < a.rank;
              const uint4 v = in ? *reinterpret_cast<const uint4*>(row + 16 * c + 8 * t)
                                 : make_uint4(0u, 0u, 0u, 0u);
              b[u][i][c][0] = v.x;
              b[u][i][c][1] = v.y;
              b[u][i][c + 1][0] = v.z;
              b[u][i][c + 1][1] = v.w;
            }
          }
        }
    }
    const int r0 = g < count ? base + (int)(sorted[p + g] & 255u) : -1;
    const int r1 = g + 8 < count ? base + (int)(sorted[p + g + 8] & 255u) : -1;
    float f0 = 0.f, f1 = 0.f;
    uint4 ua[CHUNKS], ub[CHUNKS];
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) ua[c] = ub[c] = make_uint4(0u, 0u, 0u, 0u);
    if (id != kNone) {
      if (r0 >= 0) {
        f0 = a.factor[r0];
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) ua[c] = a.u[(size_t)r0 * kFrags + 4 * c + t];
      }
      if (r1 >= 0) {
        f1 = a.factor[r1];
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) ub[c] = a.u[(size_t)r1 * kFrags + 4 * c + t];
      }
    }
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      float acc[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
      if (id != kNone) {
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            mma16<T>(acc[i], ua[c].z, ub[c].z, ua[c].w, ub[c].w, b[u][i][c][0], b[u][i][c][1]);
            mma16<T>(acc[i], ua[c].x, ub[c].x, ua[c].y, ub[c].y, b[u][i][c][0], b[u][i][c][1]);
          }
      }
      const long long col = col0 + 32 * u + 8 * t;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = h ? r1 : r0;
        const float f = h ? f1 : f0;
        if (r < 0 || col >= a.n) continue;
        const T* y = static_cast<const T*>(a.y) + (size_t)r * a.n + col;
        T* out = static_cast<T*>(a.out) + (size_t)r * a.n + col;
        if constexpr (WIDE) {
          const uint4 q = *reinterpret_cast<const uint4*>(y);
          const uint32_t in[4] = {q.x, q.y, q.z, q.w};
          uint32_t to[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            to[i] = id == kNone ? in[i]
                                : pack2<T>(fmaf(f, acc[i][2 * h], low<T>(in[i])),
                                           fmaf(f, acc[i][2 * h + 1], high<T>(in[i])));
          *reinterpret_cast<uint4*>(out) = make_uint4(to[0], to[1], to[2], to[3]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (col + i < a.n)
              out[i] = id == kNone ? y[i]
                                   : from_f32<T>(fmaf(f, acc[i / 2][2 * h + i % 2], to_f32(y[i])));
        }
      }
    }
    p += count;
  }
}

template <typename T, int CHUNKS>
cudaError_t launch_c(const LoraArgs& a, cudaStream_t s) {
  // Blocks of a cluster: few groups of tokens leave SMs idle, and a long row
  // of a is then read by more of them.
  int splits = 1;
  while (splits < 8 && (long long)a.m * splits < device_sm_count() && a.k / splits > 512) splits *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.m * splits);
  cfg.blockDim = dim3(kDownThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)splits;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, lora_down_kernel<T, CHUNKS>, a, splits);
  if (e != cudaSuccess) return e;
  note_launch();
  constexpr int kUnits = CHUNKS <= 4 ? 2 : 1;
  const bool wide = a.n % 8 == 0 && reinterpret_cast<uintptr_t>(a.y) % 16 == 0 &&
                    reinterpret_cast<uintptr_t>(a.out) % 16 == 0;
  const unsigned cols = kUpThreads * kUnits;
  const dim3 grid((a.n + cols - 1) / cols, (a.m + kTokens - 1) / kTokens);
  e = wide ? launch_pdl(lora_up_kernel<T, CHUNKS, kUnits, true>, grid, dim3(kUpThreads), 0, s, a)
           : launch_pdl(lora_up_kernel<T, CHUNKS, kUnits, false>, grid, dim3(kUpThreads), 0, s, a);
  if (e == cudaSuccess) note_launch();
  return e;
}

template <typename T> cudaError_t launch_t(const LoraArgs& a, cudaStream_t s) {
  switch (a.chunks) {
    case 1: return launch_c<T, 1>(a, s);
    case 2: return launch_c<T, 2>(a, s);
    case 4: return launch_c<T, 4>(a, s);
    default: return launch_c<T, 8>(a, s);
  }
}

}  // namespace

cudaError_t launch_lora_add(const LoraArgs& a, cudaStream_t s) {
  return a.dtype == WQL_F16 ? launch_t<__half>(a, s) : launch_t<__nv_bfloat16>(a, s);
}

}  // namespace wql
