// lora.cu -- low-rank adapters of many requests beside a shared projection:
//   out[m, n] = RN(y[m, n] + s_i * sum_j u[m, j] b[i, n, j]),
//   u[m, j]   = sum_k x[m, k] a[i, j, k],        i = ids[m].
//
// Two launches: lora_down_kernel makes u, lora_up_kernel adds its product.
// Tokens of one adapter are taken 16 at a time, the rows of one mma.sync
// m16n8k16.  The work is far below what the tensor cores need to be fed from
// tensor memory for (16 to 128 operations a byte; 23 % of the legacy pipe at rank
// 64): which k a lane's 16 bytes stand for is free, as long as both operands agree,
// so fragments are 16-byte pieces of rows as they lie.
//
// HBM-bound, in the large: b, y and out each move once.  64 rows, each with its
// own adapter of rank 16, x 248320 x 5120 120 us (67 % of the copy rate); 256 rows, 8
// adapters of rank 64, x 151936 x 1024 73.5 us (63 %); 4096 rows in 4 runs, rank 32, x
// 5120 x 5120 41 us (46 %; the first kernel, which reads a again for every 16 rows from
// L2, has half of it).  One row x 151936 x 1024, rank 16, 5.1 us.
// What bounds the large ones now is instructions as much as memory: issue 54 %,
// with 16 warps on an SM.
#include <type_traits>
#include <utility>

#include "requests.cuh"
#include "sm100.cuh"

namespace wql {
namespace {

constexpr int kTokens = kLoraSlice;      // a slice of tokens is grouped by adapter at a time
constexpr int kDownThreads = 256;
constexpr int kUpThreads = 256;
static_assert(kDownThreads == kTokens && kUpThreads == kTokens, "a thread looks at one token of the slice");

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
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
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
// Tokens of a slice by adapter: a key is an adapter and a token of the slice,
// and its place the number of smaller ones.  A group is up to 16 tokens of one
// adapter (more where lora_down_kernel works on many); those without an adapter
// come last, in groups of their own.
// ---------------------------------------------------------------------------
constexpr uint32_t kNone = 0x7FFFFFu;
__device__ __forceinline__ uint32_t key_id(uint32_t key) { return key >> 8; }

struct Sorted {
  alignas(16) uint32_t key[kTokens];     // in order
  alignas(16) uint32_t given[kTokens];   // as they come
  uint32_t begin[kTokens / 32];          // which of the tokens in order begin something
  int start[kTokens + 1];                // where the groups begin, and the end
  int groups, products;                  // all, and those that have an adapter (the first ones)
};

// Sorts the m tokens of a slice and lists their groups of up to SIZE (a block of
// kTokens threads).
template <int SIZE>
__device__ __forceinline__ void sort_tokens(Sorted& s, const int32_t* ids, int m, int count) {
  const int tid = threadIdx.x, lane = tid & 31;
  uint32_t mine = 0xFFFFFFFFu;
  if (tid < m) {
    const int id = __ldcg(ids + tid);
    mine = ((uint32_t)id < (uint32_t)count ? (uint32_t)id : kNone) << 8 | (uint32_t)tid;
  }
  s.given[tid] = mine;
  __syncthreads();
  if (tid < m) {
    int smaller = 0;
#pragma unroll 8
    for (int j = 0; j < m; j += 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(&s.given[j]);
      smaller += (v.x < mine) + (v.y < mine) + (v.z < mine) + (v.w < mine);
    }
    s.key[smaller] = mine;
  }
  __syncthreads();
  // runs of one adapter
  const uint32_t id = tid < m ? key_id(s.key[tid]) : 0u;
  const bool run = tid < m && (tid == 0 || key_id(s.key[tid - 1]) != id);
  const uint32_t runs = __ballot_sync(0xFFFFFFFFu, run);
  if (lane == 0) s.begin[tid >> 5] = runs;
  __syncthreads();
  int w = tid >> 5;
  uint32_t before = runs & (0xFFFFFFFFu >> (31 - lane));
  while (before == 0u && w > 0) before = s.begin[--w];
  const int from = 32 * w + 31 - __clz(before | 1u);
  // groups: every SIZE-th token of a run
  const bool first = tid < m && (tid - from) % SIZE == 0;
  const uint32_t firsts = __ballot_sync(0xFFFFFFFFu, first);
  __syncthreads();
  if (lane == 0) s.begin[tid >> 5] = firsts;
  __syncthreads();
  int here = __popc(firsts & ((1u << lane) - 1u)), all = 0;
#pragma unroll
  for (int v = 0; v < kTokens / 32; ++v) {
    const int n = __popc(s.begin[v]);
    here += v < (tid >> 5) ? n : 0;
    all += n;
  }
  if (first) s.start[here] = tid;
  if (tid == 0) {
    s.start[all] = m;
    s.groups = all;
  }
  // (the last run is the one without an adapter, if there is one)
  if (run && id == kNone) s.products = here;
  if (tid == m - 1 && id != kNone) s.products = all;
  __syncthreads();
}

// ---------------------------------------------------------------------------
// u: a cluster of `splits` blocks per group of tokens, which share the hidden
// columns; as many clusters as a slice can have groups.  Every block sorts the
// slice's tokens for itself (0.8 to 2.5 us; one list for all would be another
// launch).  u is written as the mma fragments that lora_up_kernel loads: per token,
// chunk and lane of four, the high parts of four ranks and what they leave of them
// (so that u keeps 16 bits or more), and the factor that the products are
// multiplied with.
// ---------------------------------------------------------------------------
template <typename T, int CHUNKS, int SIZE>
__global__ void __launch_bounds__(kDownThreads) lora_down_kernel(const LoraArgs a, int splits,
                                                                 int most_groups) {
  constexpr int kRank = 16 * CHUNKS, kTiles = 2 * CHUNKS, kWarps = kDownThreads / 32;
  constexpr int kBufs = SIZE * kRank > 1024 ? 4 : kWarps;      // 32 KB of sums
  constexpr int kSub = SIZE / 16;        // of the mma's 16 rows
  constexpr int kUnits = 2 * kSub + kTiles > 16 ? 1 : 16 / (2 * kSub + kTiles);    // 16 loads at a time
  static_assert(SIZE * kRank <= 2048, "sums of four warps");
  __shared__ alignas(16) float part[kBufs][SIZE][kRank];
  __shared__ Sorted sorted;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cluster = blockIdx.x / splits, split = blockIdx.x % splits;
  const int slice = cluster / most_groups, tile = cluster % most_groups;
  const int base = slice * kTokens, m = min(kTokens, a.m - base);
  griddep_wait();
  griddep_launch_dependents();
  sort_tokens<SIZE>(sorted, a.ids + base, m, a.count);
  if (tile >= sorted.products) return;
  const int start = sorted.start[tile], count = sorted.start[tile + 1] - start;
  const int id = (int)key_id(sorted.key[start]);
  const float scale = a.scale ? a.scale[id] : 1.f;
  auto token = [&](int i) { return base + (int)(sorted.key[start + i] & 255u); };

  const int g = lane >> 2, t = lane & 3;
  // rows g, g + 8, ... and ranks g, g + 8, ...: those that are not there are
  // others again, and dropped at the end
  const T* x[2 * kSub];
#pragma unroll
  for (int i = 0; i < 2 * kSub; ++i)
    x[i] = static_cast<const T*>(a.x) + (size_t)token(min(g + 8 * i, count - 1)) * a.k;
  const T* w[kTiles];
#pragma unroll
  for (int i = 0; i < kTiles; ++i)
    w[i] = static_cast<const T*>(a.a) + ((size_t)id * a.rank + min(8 * i + g, a.rank - 1)) * a.k;
  float acc[kSub][kTiles][4];
#pragma unroll
  for (int r = 0; r < kSub; ++r)
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[r][i][j] = 0.f;
  // units of 32 columns, 8 a lane, split evenly over the cluster's blocks and
  // dealt to the warps in turn; all of a step's loads go out before its products
  // (left to the compiler, a third of them did: 4096 x 5120 at rank 32 8 us more)
  const int units = (a.k + 31) / 32;
  const int u1 = (int)((long long)units * (split + 1) / splits);
  for (int u = (int)((long long)units * split / splits) + warp * kUnits; u < u1; u += kWarps * kUnits) {
    uint4 xv[kUnits][2 * kSub], v[kUnits][kTiles];
#pragma unroll
    for (int q = 0; q < kUnits; ++q) {
      const int col = min((u + q) * 32 + 8 * t, a.k - 8);
#pragma unroll
      for (int i = 0; i < 2 * kSub; ++i) xv[q][i] = ldg_stream_u4(x[i] + col);
#pragma unroll
      for (int i = 0; i < kTiles; ++i) v[q][i] = ldg_stream_u4(w[i] + col);
    }
    if (u + kUnits > u1 || (u + kUnits) * 32 > a.k) {    // the end: nothing from columns past it
#pragma unroll
      for (int q = 0; q < kUnits; ++q)
        if (u + q >= u1 || (u + q) * 32 + 8 * t >= a.k)
#pragma unroll
          for (int i = 0; i < 2 * kSub; ++i) xv[q][i] = make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int q = 0; q < kUnits; ++q)
#pragma unroll
      for (int r = 0; r < kSub; ++r)
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
          const uint4 &xa = xv[q][2 * r], &xb = xv[q][2 * r + 1];
          mma16<T>(acc[r][i], xa.x, xb.x, xa.y, xb.y, v[q][i].x, v[q][i].y);
          mma16<T>(acc[r][i], xa.z, xb.z, xa.w, xb.w, v[q][i].z, v[q][i].w);
        }
  }

  // sums over the warps: part[b][token][rank]
  auto put = [&](int b, bool more) {     // more: to what is there
#pragma unroll
    for (int r = 0; r < kSub; ++r)
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float2* at = reinterpret_cast<float2*>(&part[b][16 * r + 8 * h + g][8 * i + 2 * t]);
          float2 v = make_float2(acc[r][i][2 * h], acc[r][i][2 * h + 1]);
          if (more) v = make_float2(v.x + at->x, v.y + at->y);
          *at = v;
        }
  };
  if constexpr (kBufs < kWarps) {
    if (warp >= kBufs) put(warp - kBufs, false);
    __syncthreads();
    if (warp < kBufs) put(warp, true);
  } else {
    put(warp, false);
  }
  __syncthreads();
  if (splits > 1) {
    // the block's own sum, so that the others read one number each
    for (int e = tid; e < SIZE / 4 * kRank; e += kDownThreads) {
      float4* at = reinterpret_cast<float4*>(&part[0][0][0]) + e;
      float4 s = *at;
#pragma unroll
      for (int b = 1; b < kBufs; ++b) {
        const float4 v = at[b * (SIZE / 4) * kRank];
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
      }
      *at = s;
    }
    cluster_sync();
  }
  // fragments of this block's share of the tokens: four ranks a thread
  constexpr int kFrags = 4 * CHUNKS;
  const int share_tokens = SIZE / splits;
  for (int e = tid; e < share_tokens * kFrags; e += kDownThreads) {
    const int row = split * share_tokens + e / kFrags, f = e % kFrags;
    const int rank = first_rank<CHUNKS>(f >> 2, f & 3);
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (splits > 1) {
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        if (c >= splits) break;
        const float4 v = remote_f4(&part[0][row][rank], (uint32_t)c);
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
      }
    } else {
#pragma unroll
      for (int b = 0; b < kBufs; ++b) {
        const float4 v = *reinterpret_cast<const float4*>(&part[b][row][rank]);
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
      }
    }
    float factor = scale;
    float v[4] = {s.x, s.y, s.z, s.w};
    if (rank >= a.rank) v[0] = v[1] = v[2] = v[3] = 0.f;      // (ranks come in eights)
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
      // a finite scale stays finite: an infinite one would make sums that are 0 NaN (all
      // others, multiples of 2^-48, overflow the result with this one too)
      if (fabsf(scale) <= 3.4028235e38f) factor = fminf(fmaxf(factor, -3.4028235e38f), 3.4028235e38f);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] *= down;
    }
    if (row >= count) continue;
    const int to = token(row);
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

// The first of a chain: D = A B.
template <typename T>
__device__ __forceinline__ void mma16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// ---------------------------------------------------------------------------
// out = y + factor * u b.  A warp has 32 * UNITS columns and goes through groups in
// the order of their adapters, so that it reads b once per adapter.  The mma's
// columns are dealt so that a lane ends up with 8 consecutive ones of a token:
// column j of n-tile i is 8 * (j / 2) + 2 i + j % 2 of the 32.  Rows off a 16-byte
// boundary (WIDE unset) pass through shared memory, a lane per column of a unit; what
// they cost is instructions, so their places are worked out once for a group (4001
// rows x 24697, rank 8, 175 us for the call, 224 with an address for every access;
// x 24696 108).
// ---------------------------------------------------------------------------
// A warp's ring of what groups need, copied ahead: the adapter's b for the
// warp's columns, where it is another than the group's before, and the rows of y
// (WIDE).  Both lie so that the eight lanes that are served together find their
// 16 bytes (8 for a lone chunk) in different banks.
template <int CHUNKS, int UNITS, bool WIDE> struct Stage {
  static constexpr int kPieces = 2 * CHUNKS;             // of 16 bytes in a row of b
  static constexpr int kRows = 32 / kPieces;             // rows of b the warp copies at a time
  static constexpr int kB = 32 * UNITS * 32 * CHUNKS;    // bytes of b
  static constexpr int kY = WIDE ? 16 * 64 * UNITS : 0;  // of y
  static constexpr int kBytes = kB + kY;
  static constexpr int kStages = 2;
  // Column 8 q + 2 i + e of a unit's 32 is row 8 i + 2 q + e of b: a lane's 4
  // n-tiles are 8 rows apart.  (The bits of a column change places: the row of a
  // sum without carries is the sum of the rows.)
  static __host__ __device__ constexpr int b_row(int column) {
    return 32 * (column >> 5) + 8 * ((column >> 1) & 3) + 2 * ((column >> 3) & 3) + (column & 1);
  }
  // Pieces 4 apart change places in odd rows, where a row is 128 bytes or more.
  static constexpr bool kSwapB = CHUNKS >= 4, kSwapY = UNITS == 2;
  static __device__ __forceinline__ int b_at(int row, int piece) {
    return row * 32 * CHUNKS + (kSwapB ? piece ^ ((row & 1) << 2) : piece) * 16;
  }
  static __device__ __forceinline__ int y_at(int row, int piece) {
    return kB + row * 64 * UNITS + (kSwapY ? piece ^ ((row & 1) << 2) : piece) * 16;
  }
};

// 16 bytes to shared memory, at constant distances from two addresses.
template <int TO, int FROM>
__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0+%2], [%1+%3], 16;" ::"r"(to), "l"(from), "n"(TO), "n"(FROM)
               : "memory");
}
template <int... K, typename F>
__device__ __forceinline__ void each_of(std::integer_sequence<int, K...>, F f) {
  (f(std::integral_constant<int, K>()), ...);
}
template <int N, typename F> __device__ __forceinline__ void for_each(F f) {
  each_of(std::make_integer_sequence<int, N>(), f);
}


// A lane's columns of a group's rows, four rows at a time; no branch waits for
// what the ones before it load.  `rows`: where the rows lie, in bytes.  (Pairs of
// columns on 4-byte addresses, or 16-byte pieces put together in shared memory,
// save accesses and cost more in finding them: 200 rows x 151935, rank 32, 90 and
// 79 us for the call when this took 77.)
template <int UNITS>
__device__ __forceinline__ void load_columns(const char* const (&y)[UNITS], const int64_t* rows, int count,
                                             uint32_t (&v)[UNITS][16]) {
#pragma unroll
  for (int j = 0; j < 16; j += 4)
    if (j < count) {
#pragma unroll
      for (int i = j; i < j + 4; ++i) {
        const int64_t row = rows[i];
#pragma unroll
        for (int u = 0; u < UNITS; ++u) v[u][i] = __ldcg(reinterpret_cast<const unsigned short*>(y[u] + row));
      }
    }
}

template <typename T, int CHUNKS, int UNITS, bool WIDE>
__global__ void __launch_bounds__(kUpThreads, CHUNKS <= 4 ? 2 : 1)
    lora_up_kernel(const LoraArgs a) {
  using S = Stage<CHUNKS, UNITS, WIDE>;
  constexpr int kFrags = 4 * CHUNKS, kWarps = kUpThreads / 32, kStages = S::kStages;
  extern __shared__ uint4 ring[];              // [warp][stage][S::kBytes]
  __shared__ Sorted sorted;
  __shared__ float turn[WIDE ? 1 : kWarps][WIDE ? 1 : 16][WIDE ? 1 : 32 * UNITS + 1];
  __shared__ int64_t rows[2][WIDE ? 1 : kWarps][WIDE ? 1 : 16];   // of a group and the next, in bytes
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int base = blockIdx.y * kTokens, m = min(kTokens, a.m - base);
  griddep_launch_dependents();
  // The tokens are sorted again here, while lora_down_kernel works on them, and
  // what does not come from it is copied: its blocks let this kernel begin when
  // the kernels before it are done and seen.  (All of it past the L1, which may
  // hold what was there before.)
  sort_tokens<16>(sorted, a.ids + base, m, a.count);
  auto token = [&](int place) { return base + (int)(sorted.key[place] & 255u); };
  // The blocks share pairs of a strip of columns (32 * UNITS a warp) and a group
  // evenly, a block's in a row: the groups of its first strip, those of the next.
  constexpr int kStrip = kWarps * 32 * UNITS;
  const int last = sorted.products;
  const int64_t pairs = ((int64_t)a.n + kStrip - 1) / kStrip * last;
  const int64_t lo = pairs * blockIdx.x / gridDim.x, hi = pairs * (blockIdx.x + 1) / gridDim.x;

  // Copies run kStages pairs ahead.
  const uint32_t slots = (uint32_t)__cvta_generic_to_shared(ring) + warp * (kStages * S::kBytes);
  const int b_column = lane / S::kPieces, b_piece = lane % S::kPieces;
  const int64_t b_adapter = (int64_t)a.n * a.rank * 2;
  const bool b_in = 8 * b_piece < a.rank, full = a.rank == 16 * CHUNKS;
  constexpr int kYPieces = 4 * UNITS, kYRows = 32 / kYPieces;
  const int y_row = lane / kYPieces, y_piece = lane % kYPieces;
  const uint32_t b_to = S::b_at(S::b_row(b_column), b_piece), y_to = S::y_at(y_row, y_piece);
  int left = (int)(hi - lo);                   // pairs to copy
  int i_copy = 0;
  uint32_t copied = kNone;                     // the adapter of the pair before, for these columns
  int64_t col_copy = 0;
  const char* b_copy = nullptr;                // this lane's part of b for these columns, of adapter 0
  const T* y_copy = nullptr;
  auto copy_columns = [&](int64_t col) {
    col_copy = col;
    b_copy = static_cast<const char*>(a.b) + ((col + b_column) * a.rank + 8 * b_piece) * 2;
    y_copy = static_cast<const T*>(a.y) + col + 8 * y_piece;
    copied = kNone;
  };
  auto copy = [&](uint32_t slot) {
    if (left > 0) {
      --left;
      const int p = sorted.start[i_copy], count = sorted.start[i_copy + 1] - p;
      const uint32_t id = key_id(sorted.key[p]);
      const bool inside = col_copy + 32 * UNITS <= a.n;
      if (id != copied) {
        const char* at = b_copy + id * b_adapter;
        if (full && inside) {
          for_each<UNITS * S::kPieces>([&](auto k) {
            copy16<S::b_row(k * S::kRows) * 32 * CHUNKS, k * 512>(slot + b_to, at);
          });
        } else {
          const int b_step = S::kRows * 2 * a.rank;
          for_each<UNITS * S::kPieces>([&](auto k) {
            if (b_in && col_copy + b_column + k * S::kRows < a.n)
              copy16<S::b_row(k * S::kRows) * 32 * CHUNKS, 0>(slot + b_to, at + k * b_step);
          });
        }
        copied = id;
      }
      if constexpr (WIDE) {
        const bool y_in = inside || col_copy + 8 * y_piece < a.n;
        auto row = [&](auto k) {
          if (y_row + k * kYRows < count && y_in)
            copy16<k * kYRows * 64 * UNITS, 0>(slot + y_to, y_copy + (int64_t)token(p + y_row + k * kYRows) * a.n);
        };
        if (count <= kYRows) row(std::integral_constant<int, 0>());
        else for_each<16 / kYRows>(row);
      }
      if (++i_copy == last) {
        i_copy = 0;
        copy_columns(col_copy + kStrip);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  if (!full) {                                 // ranks that are never copied are zero
    for (int k = lane; k < kStages * S::kBytes / 16; k += 32)
      ring[warp * (kStages * S::kBytes / 16) + k] = make_uint4(0u, 0u, 0u, 0u);
    __syncwarp();
  }
  int i = 0;
  int64_t col0 = 0;
  if (left > 0) {
    i = i_copy = (int)(lo % last);
    col0 = lo / last * kStrip + warp * (32 * UNITS);
    copy_columns(col0);
  }
#pragma unroll
  for (int k = 0; k < kStages; ++k) copy(slots + k * S::kBytes);
  griddep_wait();

  uint32_t b[UNITS][4][CHUNKS][2];
  uint32_t current = kNone;                    // b's adapter
  uint32_t offset = 0;                         // of the slot
  const char* const mine = reinterpret_cast<const char*>(ring) + warp * (kStages * S::kBytes);
  // where this lane reads: the first piece of a pair that changes places, the other
  const uint32_t b_even = S::b_at(g, 0) + (CHUNKS == 1 ? 8 : 16) * t, b_odd = b_even ^ 64u;
  const uint32_t y_even = S::y_at(g, t), y_odd = S::kSwapY ? y_even ^ 64u : 0u;
  if (!WIDE && hi > lo && lane < 16)
    rows[(hi - lo) & 1][warp][lane] = 2 * ((int64_t)token(min(sorted.start[i] + lane, sorted.start[i + 1] - 1)) * a.n);
  __syncwarp();
  for (int todo = (int)(hi - lo); todo > 0; --todo) {
    const int p = sorted.start[i], count = sorted.start[i + 1] - p;
    const uint32_t id = key_id(sorted.key[p]);
    const int columns = (int)min((int64_t)(32 * UNITS), a.n - col0);
    // rows past the group's are its last token's again, and are not stored
    const int r0 = token(p + min(g, count - 1)), r1 = token(p + min(g + 8, count - 1));
    const float f0 = a.factor[r0], f1 = a.factor[r1];
    const uint4* u0 = a.u + (int64_t)r0 * kFrags + t;
    const uint4* u1 = a.u + (int64_t)r1 * kFrags + t;
    uint4 ua[CHUNKS], ub[CHUNKS];
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      ua[c] = u0[4 * c];
      ub[c] = u1[4 * c];
    }
    // y: WIDE, rows g and g + 8, 8 columns a unit; else a column a lane and unit
    uint32_t y[UNITS][WIDE ? 8 : 16];
    if constexpr (!WIDE) {
      const char* columns_of[UNITS];           // (past the last column: the last one again)
#pragma unroll
      for (int u = 0; u < UNITS; ++u)
        columns_of[u] = static_cast<const char*>(a.y) + 2 * min(col0 + 32 * u + lane, (int64_t)a.n - 1);
      __syncwarp();                            // the group before is stored
      if (lane < 16 && todo > 1) {
        const int k = i + 1 == last ? 0 : i + 1, q = sorted.start[k];
        rows[(todo & 1) ^ 1][warp][lane] = 2 * ((int64_t)token(min(q + lane, sorted.start[k + 1] - 1)) * a.n);
      }
      load_columns<UNITS>(columns_of, rows[todo & 1][warp], count, y);
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    __syncwarp();
    const char* slot = mine + offset;
    if (id != current) {
      current = id;
      const char* even = slot + b_even;
      const char* odd = slot + b_odd;
#pragma unroll
      for (int u = 0; u < UNITS; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int row = (32 * u + 8 * j) * 32 * CHUNKS;
          if constexpr (CHUNKS == 1) {
            const uint2 q = *reinterpret_cast<const uint2*>(even + row);
            b[u][j][0][0] = q.x;
            b[u][j][0][1] = q.y;
          } else {
#pragma unroll
            for (int c = 0; c < CHUNKS; c += 2) {
              const uint4 q = *reinterpret_cast<const uint4*>((c & 2 ? odd : even) + row + 128 * (c / 4));
              b[u][j][c][0] = q.x;
              b[u][j][c][1] = q.y;
              b[u][j][c + 1][0] = q.z;
              b[u][j][c + 1][1] = q.w;
            }
          }
        }
    }
    if constexpr (WIDE) {
#pragma unroll
      for (int u = 0; u < UNITS; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 q = *reinterpret_cast<const uint4*>(slot + (u ? y_odd : y_even) + 8 * h * 64 * UNITS);
          y[u][4 * h] = q.x;
          y[u][4 * h + 1] = q.y;
          y[u][4 * h + 2] = q.z;
          y[u][4 * h + 3] = q.w;
        }
    }
    __syncwarp();                              // read by all before it is written again
    copy(slots + offset);
    offset = offset == (kStages - 1) * S::kBytes ? 0u : offset + S::kBytes;

#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      float acc[4][4];
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (c == 0) mma16_first<T>(acc[j], ua[c].z, ub[c].z, ua[c].w, ub[c].w, b[u][j][c][0], b[u][j][c][1]);
          else mma16<T>(acc[j], ua[c].z, ub[c].z, ua[c].w, ub[c].w, b[u][j][c][0], b[u][j][c][1]);
          mma16<T>(acc[j], ua[c].x, ub[c].x, ua[c].y, ub[c].y, b[u][j][c][0], b[u][j][c][1]);
        }
      if constexpr (WIDE) {
        const int column = 32 * u + 8 * t;
        T* to = static_cast<T*>(a.out) + col0 + column;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (8 * h >= count) break;
          const float f = h ? f1 : f0;
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            w[j] = pack2<T>(fmaf(f, acc[j][2 * h], low<T>(y[u][4 * h + j])),
                            fmaf(f, acc[j][2 * h + 1], high<T>(y[u][4 * h + j])));
          if (g + 8 * h < count && column < columns)
            *reinterpret_cast<uint4*>(to + (int64_t)(h ? r1 : r0) * a.n) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            turn[warp][g][32 * u + 8 * t + 2 * j + e] = acc[j][e];
            turn[warp][g + 8][32 * u + 8 * t + 2 * j + e] = acc[j][2 + e];
          }
      }
    }
    if constexpr (!WIDE) {
      __syncwarp();
      char* to = static_cast<char*>(a.out) + 2 * (col0 + lane);
#pragma unroll
      for (int j = 0; j < 16; j += 4) {
        if (j >= count) break;
#pragma unroll
        for (int r = j; r < j + 4; ++r) {
          const float f = __shfl_sync(0xFFFFFFFFu, r < 8 ? f0 : f1, 4 * (r & 7));
          T* at = reinterpret_cast<T*>(to + rows[todo & 1][warp][r]);
#pragma unroll
          for (int u = 0; u < UNITS; ++u)
            if (r < count && 32 * u + lane < columns)
              at[32 * u] = from_f32<T>(fmaf(f, turn[warp][r][32 * u + lane], low<T>(y[u][r])));
        }
      }
    }
    if (++i == last) {
      i = 0;
      col0 += kStrip;
      current = kNone;
    }
  }

  // rows without an adapter, 256 columns at a time
  if (a.out != a.y && last < sorted.groups) {
    const int p = sorted.start[last];
    const int64_t parts = ((int64_t)a.n + 255) / 256, all = parts * (m - p);
    for (int64_t k = (int64_t)blockIdx.x * kWarps + warp; k < all; k += (int64_t)gridDim.x * kWarps) {
      const int64_t column = k % parts * 256, row = (int64_t)token(p + (int)(k / parts)) * a.n;
      const T* y = static_cast<const T*>(a.y) + row;
      T* to = static_cast<T*>(a.out) + row;
      if constexpr (WIDE) {
        if (column + 8 * lane < a.n)
          *reinterpret_cast<uint4*>(to + column + 8 * lane) =
              __ldcg(reinterpret_cast<const uint4*>(y + column + 8 * lane));
      } else {
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (column + 32 * u + lane < a.n) to[column + 32 * u + lane] = y[column + 32 * u + lane];
      }
    }
  }
}

template <typename T, int CHUNKS, bool WIDE>
cudaError_t launch_up(const LoraArgs& a, int groups, int slices, cudaStream_t s) {
  // (as ranks leave registers for two.  Off the boundary 64 rows x 50303 with an
  // adapter each, rank 16: 41 us for the call, 43.5 with one; 1000 rows x 50303, rank
  // 32: 117, 132 with one.)
  constexpr int kUnits = CHUNKS == 1 || (CHUNKS == 2 && !WIDE) ? 2 : 1;
  using S = Stage<CHUNKS, kUnits, WIDE>;
  constexpr size_t kRing = (size_t)kUpThreads / 32 * S::kStages * S::kBytes;
  auto kern = lora_up_kernel<T, CHUNKS, kUnits, WIDE>;
  static LargestPerDevice limit;
  const cudaError_t e = allow_smem(limit, kern, kRing);
  if (e != cudaSuccess) return e;
  // As many blocks as the SMs hold, or fewer where the pairs are fewer.
  constexpr int kResident = CHUNKS <= 4 ? 2 : 1;
  const int64_t most = ((int64_t)a.n + kUpThreads * kUnits - 1) / (kUpThreads * kUnits) * groups;
  int64_t blocks = ((int64_t)kResident * device_sm_count() + slices - 1) / slices;
  if (blocks > most) blocks = most;
  return launch_pdl(kern, dim3((unsigned)blocks, (unsigned)slices), dim3(kUpThreads), kRing, s, a);
}

// The most groups of `size` tokens that a slice can have: one of every adapter
// may be smaller.
int most_groups(const LoraArgs& a, int size) {
  const int in_slice = a.m < kTokens ? a.m : kTokens;
  const int kinds = a.count < in_slice ? a.count + 1 : in_slice;
  const int most = in_slice / size + kinds;
  return most < in_slice ? most : in_slice;
}

template <typename T, int CHUNKS, int SIZE> cudaError_t launch_down(const LoraArgs& a, int slices, cudaStream_t s) {
  const int groups = most_groups(a, SIZE);
  // Blocks of a cluster, which share the columns: while a block has more than 32 KB
  // of a to read, and two blocks to an SM are not reached.  (151936 x 1024,
  // rank 16, one token: 5.2 us with one, 5.7 with two; 256 tokens at rank 64 79 us
  // with two, 72 with four.)
  int splits = 1;
  while (splits < 8 && (long long)groups * slices * splits <= device_sm_count() &&
         (long long)a.k / splits * 16 * CHUNKS > 16384)
    splits *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)slices * groups * splits);
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
  const cudaError_t e = cudaLaunchKernelEx(&cfg, lora_down_kernel<T, CHUNKS, SIZE>, a, splits, groups);
  if (e == cudaSuccess) note_launch();
  return e;
}

template <typename T, int CHUNKS>
cudaError_t launch_c(const LoraArgs& a, cudaStream_t s) {
  const int slices = (a.m + kTokens - 1) / kTokens;
  // Prompts come in long runs: at rank 64 groups of 32 read a half as often (2000
  // tokens, 5120 x 5120: 38 us for the call, 48 with groups of 16; at rank 32 41.7
  // and 40.4).
  constexpr int kLarge = CHUNKS == 4 ? 32 : 16;
  cudaError_t e = a.m > 2 * kTokens ? launch_down<T, CHUNKS, kLarge>(a, slices, s)
                                    : launch_down<T, CHUNKS, 16>(a, slices, s);
  if (e != cudaSuccess) return e;
  const int groups = most_groups(a, 16);
  const bool wide = a.n % 8 == 0 && reinterpret_cast<uintptr_t>(a.y) % 16 == 0 &&
                    reinterpret_cast<uintptr_t>(a.out) % 16 == 0;
  e = wide ? launch_up<T, CHUNKS, true>(a, groups, slices, s) : launch_up<T, CHUNKS, false>(a, groups, slices, s);
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
