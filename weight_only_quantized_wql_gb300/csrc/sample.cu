// sample.cu -- draw the next token of every row: temperature, top-k, top-p
// and min-p, from a given random number.
//
// Weights are integers, W = floor(2^31 * exp2((l - max) * log2e / t)), so
// every sum is exact and the same in any order; ranks go by logit descending,
// then index ascending.  Each filter keeps a prefix of that order, so a row's
// filters come down to one cut, the rank key of the last kept token:
// (order-preserving bits of the logit, inverted index).
//
// One cluster of 1 to 8 blocks per row, each over a contiguous slice, which
// stays in shared memory when it fits (76 KB, so that two blocks share an SM
// and one's copies run under the other's passes):
//  * the maximum (and those of four shares of each thread's elements);
//  * top-k up to 512: a bound that about k logits reach, from a histogram of
//    the share maxima (k values at least as large exist if k maxima do); one
//    pass gathers the logits above it; the first block ranks that list,
//    applies the filters by prefix sums and draws;
//  * a nucleus: a histogram of the weights over quarter octaves below the
//    maximum finds the one that holds the cut; a second pass sums the weights
//    above it per stretch of the row and gathers its own tokens, which the
//    first block ranks to find the cut; their kept weights join the stretches'
//    sums, and the draw walks the one stretch that holds it;
//  * a larger top-k, or more open tokens than the list holds: histograms of
//    counts or weights, first over quarter octaves, then over seven bits of the
//    rank key at a time, until the open tokens fit; then, as when temperature
//    or min-p alone is on, one pass for the stretches' sums and the walk.
//
// What bounds it: one row, the barriers between its dependent steps; many rows,
// the latency of two or three passes' loads (all but the first from L2) at 27 warps
// an SM, and at 256 rows that 104 of 152 SMs have two of them: the schedulers issue
// in 30 to 47 % of the cycles, shared memory's pipe is 11 % busy.  The loops over a
// row are kept short (one 16-byte piece a turn): unrolled by four they were bound by
// instruction fetches.  Measured: 1 x 151936 bf16 top-k 10.7 us, temperature alone
// 9.3, a nucleus 19.2; 64 x 248320 fp32, temperature alone, 31 us; 256 x 151936 bf16
// top-k 31 us (2.5 TB/s), a nucleus 100 us.
// Histograms keep 16 copies, one per lane and its half warp's partner, so that a
// warp's additions hardly meet in a bank; a copy's sums (16 low and 15 high bits
// of the weights apart) stay below 2^32 for 2^20 tokens.
#include <cooperative_groups.h>
#include <stddef.h>

#include <type_traits>

#include "mx.cuh"
#include "sm100.cuh"

namespace cg = cooperative_groups;

namespace wql {
namespace {

typedef unsigned long long u64;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kList = 2048;          // tokens the joined list holds with their weights
constexpr int kOpen = 4096;          // and without
constexpr int kLocal = 1024;         // a block's own list, in a cluster
constexpr int kBins = 128;
constexpr int kCopies = 16;          // of a histogram
constexpr int kShares = 4;           // maxima kept per thread
constexpr int kSegs = 16;            // stretches of a warp's part of the row
constexpr int kChunks = 4;           // copies that bring a slice in, four warps' parts each
constexpr int kMaxCluster = 8;
constexpr int kMaxListK = 512;       // largest top-k that goes by a bound and a list
constexpr int kCountRank = 128;      // lists up to this long are ranked by counting
constexpr int kIndexBits = 20;
constexpr int kHeldBytes = 76 * 1024;
constexpr float kLog2e = 1.44269504088896340736f;
static_assert(WQL_SAMPLE_MAX_N == 1 << kIndexBits, "rank keys hold an index");

struct alignas(16) Shared {
  u64 seg[kWarps][kSegs];
  u64 red[kWarps];
  float redf[kWarps];
  uint64_t bars[kChunks];
  uint64_t stall;                      // diagnostics: nothing arrives here
  // read by the other blocks of the cluster
  u64 bin_mass[kBins];
  uint32_t bin_count[kBins];
  float max;
  int failed;                          // a wait for this block's copies ran out
  u64 sum;
  uint32_t listed;
  u64 cut;                             // of the first block
  // block-wide results
  int digit;
  u64 before_count, before_mass;
  // this block's list; in the first block, the joined one, which goes on where
  // the histograms are, once they are folded: kOpen rank keys, or kList and
  // their weights
  u64 list[kLocal];
  struct {
    uint32_t low[kBins][kCopies];      // sums of weights' low 16 bits
    uint32_t high[kBins][kCopies];     // and of the bits above
    uint32_t count[kBins][kCopies];
  } hist;
};
static_assert(offsetof(Shared, hist) == offsetof(Shared, list) + kLocal * 8 &&
                  sizeof(Shared::hist) >= (kOpen - kLocal) * 8 && kList * 12 <= kOpen * 8,
              "the joined list goes on into the histograms");

// Through the symbol, so that the compiler sees shared memory in functions that
// are not inlined too (as a reference argument it made every access generic
// and every addition to a histogram a branch).
extern __shared__ __align__(16) uint8_t sample_smem[];
__device__ __forceinline__ Shared& shared() { return *reinterpret_cast<Shared*>(sample_smem); }
__device__ __forceinline__ uint4* held_pieces() {
  return reinterpret_cast<uint4*>(sample_smem + sizeof(Shared));
}

__device__ __forceinline__ u64* keys() { return shared().list; }
__device__ __forceinline__ uint32_t* weights() {
  return reinterpret_cast<uint32_t*>(keys() + kList);
}

__device__ __forceinline__ uint32_t logit_key(float l) {
  const uint32_t b = __float_as_uint(l + 0.f);        // -0 ranks as +0
  return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
constexpr uint32_t kIndexMask = (1u << kIndexBits) - 1u;
__device__ __forceinline__ u64 rank_key(float l, uint32_t idx) {
  return ((u64)logit_key(l) << kIndexBits) | (~idx & kIndexMask);
}
__device__ __forceinline__ float rank_logit(u64 key) {
  return key_logit((uint32_t)(key >> kIndexBits));
}
__device__ __forceinline__ uint32_t rank_index(u64 key) { return ~(uint32_t)key & kIndexMask; }

// What a row is drawn with.
struct Row {
  float top;       // largest logit
  float c;         // log2e / temperature
  float min_p;     // 0: off
  // log2 of a token's weight over the likeliest's (top and c are finite here; a
  // NaN stays, converts to weight 0 and compares false)
  __device__ __forceinline__ float depth(float l) const {
    return __fmul_rn(__fsub_rn(l, top), c);
  }
  // 2^x; the same bits as exp2f() from -126 up, and W = 0 below -31 anyway
  static __device__ __forceinline__ float e(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
  }
  static __device__ __forceinline__ uint32_t weight(float e) {
    return __float2uint_rz(e * 2147483648.f);
  }
  // The same in two halves without the conversion, which shares the slow unit
  // with the exponential: floats 2^23 + W / 2^16 and 2^23 + W % 2^16 (each
  // product is exact, each sum truncates), whose bits are kOne + the half.  Not
  // for a NaN.
  static constexpr uint32_t kOne = 0x4B000000u;
  static __device__ __forceinline__ void halves(float e, uint32_t* high, uint32_t* low) {
    const float h = __fmaf_rz(e, 32768.f, 8388608.f);
    const float rest = __fmaf_rn(__fsub_rn(h, 8388608.f), -1.f / 32768.f, e);
    *high = __float_as_uint(h);
    *low = __float_as_uint(__fmaf_rz(rest, 2147483648.f, 8388608.f));
  }
  // quarter octaves below the maximum, rounded to the nearest: never
  // decreasing with the logit's rank, at most 124 for a token with a weight
  static __device__ __forceinline__ uint32_t bin_if_weight(float x) {
    return __float_as_uint(fmaf(x, -4.f, 8388608.f)) - 0x4B000000u;
  }
  static __device__ __forceinline__ int bin(float x) {
    return (int)min(bin_if_weight(x), (uint32_t)(kBins - 1));
  }
};

// A row of logits in 16-byte pieces on 16-byte addresses: piece q holds
// elements q*V - mis .. + V-1; those outside the row read as -inf.  kHeld: this
// block's pieces, from s0 on, are in shared memory.  kWhole: rows are whole
// pieces in global memory.  kRagged: they may not be, and the first and the last
// one are made up in shared memory.
enum Mode { kHeld, kWhole, kRagged };
template <typename T, Mode MODE> struct Pieces {
  static constexpr bool HELD = MODE == kHeld;
  static constexpr int V = 16 / (int)sizeof(T);
  const T* base;       // 16-byte aligned, mis elements before the row
  int mis, n, pieces, s0;
  __device__ __forceinline__ Pieces(const T* row, int n_) : n(n_) {
    mis = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    base = row - mis;
    pieces = (n + mis + V - 1) / V;
    s0 = 0;
  }
  // first piece of a warp's part
  __device__ __forceinline__ int first(int part, int parts) const {
    return (int)((uint32_t)pieces * (uint32_t)part / (uint32_t)parts);     // 2^18 * 128 at most
  }
  // the part that piece q lies in: the last that starts at or before q
  __device__ __forceinline__ int part_of(int q, int parts) const {
    return (int)((((uint32_t)q + 1u) * (uint32_t)parts - 1u) / (uint32_t)pieces);
  }
  __device__ __forceinline__ uint4 load(int q) const {
    if constexpr (HELD) {
      return held_pieces()[q - s0];
    } else {
      if constexpr (MODE == kRagged) {
        if (q == 0 || q == pieces - 1) return held_pieces()[q == 0 ? 0 : 1];
      }
      return __ldg(reinterpret_cast<const uint4*>(base) + q);
    }
  }
  // an element of the row, of a piece that this block has
  __device__ __forceinline__ float element(int idx) const {
    const int at = idx + mis;
    if constexpr (HELD) return to_f32(reinterpret_cast<const T*>(held_pieces())[at - s0 * V]);
    return to_f32(base[at]);
  }
  // the first or last piece, element by element
  __device__ __noinline__ uint4 load_end(int q) const {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    for (int j = 0; j < V; ++j) {
      const int i = q * V - mis + j;
      uint32_t bits;
      if constexpr (sizeof(T) == 4) {
        bits = i >= 0 && i < n ? __float_as_uint(base[(size_t)q * V + j]) : 0xFF800000u;
        w[j] = bits;
      } else {
        const T none = from_f32<T>(__int_as_float(0xFF800000));
        const T l = i >= 0 && i < n ? base[(size_t)q * V + j] : none;
        bits = *reinterpret_cast<const uint16_t*>(&l);
        w[j >> 1] |= bits << (16 * (j & 1));
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ void values(const uint4& r, float (&v)[V]) {
    const T* h = reinterpret_cast<const T*>(&r);
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = to_f32(h[j]);
  }
  // Largest value of a piece (NaNs apart: -inf or less than any other).
  static __device__ __forceinline__ float max_of(const uint4& r) {
    if constexpr (sizeof(T) == 4) {
      float v[V];
      values(r, v);
      return fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
    } else {
      using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2,
                                           __nv_bfloat162>::type;
      const T2* h = reinterpret_cast<const T2*>(&r);
      const T2 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
      return fmaxf(to_f32(m.x), to_f32(m.y));
    }
  }
  // This lane's pieces of the batch at b (32 * kShares consecutive pieces).
  __device__ __forceinline__ void batch(int b, int q1, uint4 (&r)[kShares]) const {
#pragma unroll
    for (int u = 0; u < kShares; ++u) {
      const int q = b + u * 32 + (int)(threadIdx.x & 31);
      r[u] = q < q1 ? load(q) : make_uint4(0u, 0u, 0u, 0u);
    }
  }
  // f(piece, its number, u) for this warp's pieces q0 .. q1, D a turn without a
  // check (u = 0 .. D-1), then the rest
  template <int D, typename F>
  __device__ __forceinline__ void each_piece(int q0, int q1, F f) const {
    const int lane = threadIdx.x & 31;
    int q = q0;
    if constexpr (MODE == kRagged && D > 1) {
      if (q == 0) {                    // with the row's first piece: by themselves
#pragma unroll 1
        for (const int q2 = min(q1, 32 * D); q < q2; q += 32)
          if (q + lane < q2) f(load(q + lane), q + lane, 0);
        q = min(q1, 32 * D);
      }
    }
    const int whole = MODE == kRagged && q1 == pieces ? q1 - 1 : q1;
    if constexpr (D > 1) {
#pragma unroll 1
      for (; q + 32 * D <= whole; q += 32 * D) {
        uint4 r[D];
        if constexpr (HELD) {
          const uint4* p = held_pieces() + (q + lane - s0);
#pragma unroll
          for (int u = 0; u < D; ++u) r[u] = p[u * 32];
        } else {
          const uint4* p = reinterpret_cast<const uint4*>(base) + (q + lane);
#pragma unroll
          for (int u = 0; u < D; ++u) r[u] = __ldg(p + u * 32);
        }
#pragma unroll
        for (int u = 0; u < D; ++u) f(r[u], q + u * 32 + lane, u);
      }
    }
#pragma unroll 1
    for (q += lane; q < q1; q += 32) f(load(q), q, 0);
  }
  // f(values, index of the first) for them
  template <typename F> __device__ __forceinline__ void each(int q0, int q1, F f) const {
    each_piece<HELD ? 1 : 16 / V>(q0, q1, [&](const uint4& r, int q, int) {
      float v[V];
      values(r, v);
      f(v, q * V - mis);
    });
  }
  // and for those whose largest value reaches `low`, D a turn
  template <int D, typename F>
  __device__ __forceinline__ void each_above(int q0, int q1, float low, F f) const {
    each_piece<HELD ? 1 : D>(q0, q1, [&](const uint4& r, int q, int) {
      if (max_of(r) >= low) {
        float v[V];
        values(r, v);
        f(v, q * V - mis);
      }
    });
  }
};

// The cluster that works on one row.
struct Team {
  cg::cluster_group cluster;
  int size, rank;
  __device__ __forceinline__ Team() : cluster(cg::this_cluster()) {
    size = (int)cluster.num_blocks();
    rank = (int)cluster.block_rank();
  }
  __device__ __forceinline__ void sync() const {
    if (size > 1)
      cluster.sync();
    else
      __syncthreads();
  }
  template <typename X> __device__ __forceinline__ X* of(X* p, int r) const {
    return size > 1 ? cluster.map_shared_rank(p, r) : p;
  }
  // f(the value of *p in block k, k) for all blocks, read at once
  template <typename X, typename F> __device__ __forceinline__ void over(X* p, F f) const {
    X v[kMaxCluster];
#pragma unroll
    for (int k = 0; k < kMaxCluster; ++k)
      if (k < size) v[k] = *of(p, k);
#pragma unroll
    for (int k = 0; k < kMaxCluster; ++k)
      if (k < size) f(v[k], k);
  }
};

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
  return v;
}
__device__ __forceinline__ u64 warp_scan(u64 v) {      // inclusive
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const u64 o = __shfl_up_sync(0xFFFFFFFFu, v, d);
    if ((threadIdx.x & 31) >= d) v += o;
  }
  return v;
}

// Exclusive prefix sum over the block; *total gets the sum.
__device__ u64 block_scan(u64 v, u64* total) {
  Shared& sh = shared();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const u64 inc = warp_scan(v);
  __syncthreads();
  if (lane == 31) sh.red[warp] = inc;
  __syncthreads();
  u64 before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const u64 t = sh.red[w];
    if (w < warp) before += t;
    sum += t;
  }
  *total = sum;
  return before + inc - v;
}

// Sorts the joined list's first `size` keys descending; a power of two, at least 2.
__device__ void sort_list(int size) {
  Shared& sh = shared();
  __syncthreads();
  for (int len = 2; len <= size; len <<= 1) {
    for (int stride = len >> 1; stride > 0; stride >>= 1) {
      for (int i = threadIdx.x; i < size / 2; i += kThreads) {
        const int p = 2 * i - (i & (stride - 1));
        const u64 a = keys()[p], b = keys()[p + stride];
        const bool up = (p & len) != 0;              // ascending stretch
        if (up ? a > b : a < b) {
          keys()[p] = b;
          keys()[p + stride] = a;
        }
      }
      // a warp's pairs of strides <= 32 stay within its own 64 entries
      if (stride > 32 || (stride == 1 && len >= 64))
        __syncthreads();
      else
        __syncwarp();
    }
  }
  __syncthreads();
}

__device__ __forceinline__ int pow2_at_least(int v) {
  int p = 2;
  while (p < v) p <<= 1;
  return p;
}

__device__ __forceinline__ void put(const Team& team, uint32_t at, u64 key) {
  // (a block alone goes on into the joined list)
  if (at < (uint32_t)(team.size > 1 ? kLocal : kOpen)) keys()[at] = key;
}
__device__ __forceinline__ void append(const Team& team, u64 key) {
  put(team, atomicAdd(&shared().listed, 1u), key);
}

// Tokens listed by all blocks of the cluster; more than kOpen when they do not
// fit.  After a sync that follows the gathering; the caller syncs before the
// lists are used again.
__device__ __forceinline__ u64 listed_by_all(const Team& team) {
  Shared& sh = shared();
  if (team.size == 1) return sh.listed;
  u64 total = 0;
  team.over(&sh.listed, [&](uint32_t c, int) {
    total += c <= (uint32_t)kLocal ? (u64)c : (u64)kOpen + 1ull;
  });
  return total;
}

// The first block's joined list gets the other blocks' lists behind its own
// (they fit).
__device__ void join_lists(const Team& team) {
  Shared& sh = shared();
  if (team.rank != 0 || team.size == 1) return;
  const int warp = threadIdx.x >> 5;                   // one warp a block's list
  if (warp > 0 && warp < team.size) {
    uint32_t at = 0, mine = 0;
    team.over(&sh.listed, [&](uint32_t c, int k) {
      if (k < warp) at += c;
      if (k == warp) mine = c;
    });
    const u64* src = team.of(&sh.list[0], warp);
    for (uint32_t i = threadIdx.x & 31; i < mine; i += 32) keys()[at + i] = src[i];
  }
  __syncthreads();
}

// floor(f * s) for 0 < f < 1 and s < 2^52, and whether something is left of it:
// exact in 128 bits (the product has up to 76 significant ones).
__device__ __forceinline__ u64 floor_product(float f, u64 s, bool* rest) {
  const uint32_t b = __float_as_uint(f);
  const int exponent = max((int)(b >> 23), 1);         // f = mantissa * 2^(exponent - 150)
  const u64 mantissa = (b & 0x7FFFFFu) | (b >> 23 ? 0x800000u : 0u);
  const int shift = 150 - exponent;                    // 24 .. 149
  const u64 lo = mantissa * s, hi = __umul64hi(mantissa, s);       // hi < 2^12
  const int high_shift = min(shift - 64, 12);
  *rest = shift < 64 ? (lo << (64 - shift)) != 0ull
                     : lo != 0ull || (hi & ((1ull << high_shift) - 1ull)) != 0ull;
  return shift < 64 ? (hi << (64 - shift)) | (lo >> shift) : hi >> high_shift;
}

// The integer that a nucleus' weights have to reach: those before a kept
// token sum to less than p * sum, so to less than its ceiling (p < 1).
__device__ __forceinline__ u64 nucleus_target(float p, u64 sum) {
  if (!(p > 0.f)) return 1ull;
  bool rest;
  const u64 t = floor_product(p, sum, &rest);
  return max(t + (rest ? 1ull : 0ull), 1ull);
}

__device__ __forceinline__ u64 draw_target(float u, u64 sum) {
  if (!(u > 0.f)) return 0ull;
  if (u >= 1.f) return sum - 1;
  bool rest;
  return floor_product(u, sum, &rest);
}

__device__ __forceinline__ void write_draw(const SampleArgs& a, int row, int id, uint32_t w,
                                           u64 sum) {
  a.ids[row] = id;
  if (a.logp) a.logp[row] = logf(__fdiv_rn((float)w, (float)sum));
}

// Top-k, top-p, min-p and draw among the `len` tokens of the first block's
// joined list, which hold the first top_k by rank (or, fewer, all with a weight).
// Short lists: every token counts the tokens and sums the weights before it,
// by rank and then, among the kept, by index.
__device__ __noinline__ void finish_by_counting(const SampleArgs& a, int row,
                                                const Row& r, int len, int top_k, float top_p,
                                                float u) {
  Shared& sh = shared();
  static_assert(kThreads == 4 * kCountRank, "four lanes a token");
  const int p = threadIdx.x >> 2, part = threadIdx.x & 3;
  u64 key = 0;
  float e = 0.f;
  uint32_t w = 0;
  if (p < len) {
    key = keys()[p];
    e = Row::e(r.depth(rank_logit(key)));
    w = Row::weight(e);
    if (part == 0) weights()[p] = w;
  }
  __syncthreads();
  u64 before = 0;                      // weights before it by rank, and how many tokens
  for (int j = part; j < len; j += 4)
    if (keys()[j] > key) before += ((u64)weights()[j] << 8) | 1u;
  before += __shfl_xor_sync(0xFFFFFFFFu, before, 1);
  before += __shfl_xor_sync(0xFFFFFFFFu, before, 2);
  const bool in_k = p < len && (int)(before & 255u) < top_k;
  before >>= 8;
  u64 sum = ~0ull;
  if (top_p < 1.f) block_scan(in_k && part == 0 ? w : 0u, &sum);
  const bool keep = in_k && (top_p >= 1.f || before < nucleus_target(top_p, sum)) && e >= r.min_p;
  u64 kept;
  block_scan(keep && part == 0 ? w : 0u, &kept);
  if (p < len && !keep && part == 0) weights()[p] = 0u;
  __syncthreads();
  u64 run = 0;                         // kept weights of lower indices
  const uint32_t idx = rank_index(key);
  for (int j = part; j < len; j += 4)
    if (rank_index(keys()[j]) < idx) run += weights()[j];
  run += __shfl_xor_sync(0xFFFFFFFFu, run, 1);
  run += __shfl_xor_sync(0xFFFFFFFFu, run, 2);
  const u64 target = draw_target(u, kept);
  if (keep && part == 0 && run <= target && target < run + w)
    write_draw(a, row, (int)idx, w, kept);
}

// The same for longer lists: sort, prefix sums, sort the kept by index.
__device__ __noinline__ void finish_by_sorting(const SampleArgs& a, int row, const Row& r, int len,
                                  int top_k, float top_p, float u) {
  Shared& sh = shared();
  const int size = pow2_at_least(len);
  for (int i = len + threadIdx.x; i < size; i += kThreads) keys()[i] = 0ull;
  sort_list(size);
  constexpr int kPer = kList / kThreads;
  const int per = (size + kThreads - 1) / kThreads;    // 1..kPer consecutive entries a thread
  float e[kPer];
  uint32_t w[kPer];
  u64 mine = 0;
  const int limit = min(top_k, len);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int p = threadIdx.x * per + i;
    w[i] = 0u;
    e[i] = 0.f;
    if (i < per && p < limit) {
      e[i] = Row::e(r.depth(rank_logit(keys()[p])));
      w[i] = Row::weight(e[i]);
      mine += w[i];
    }
  }
  u64 sum;
  u64 before = block_scan(mine, &sum);
  const u64 reach = top_p < 1.f ? nucleus_target(top_p, sum) : ~0ull;
  // keep a prefix: count it, and its weights
  u64 kept = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int p = threadIdx.x * per + i;
    if (i < per && p < limit && before < reach && e[i] >= r.min_p)
      kept += ((u64)w[i] << 12) | 1u;                  // up to 2^11 weights of 2^31, and a count
    before += w[i];
    if (i < per && p < kList) weights()[p] = w[i];
  }
  u64 kept_total;
  block_scan(kept, &kept_total);
  const int keep = (int)(kept_total & 0xFFFu);
  const u64 kept_sum = kept_total >> 12;
  // the kept tokens by index: (inverted index, rank), descending
  u64 by_index[kPer];
  const int size2 = pow2_at_least(keep);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int p = threadIdx.x + i * kThreads;
    by_index[i] = p < keep ? ((keys()[p] & kIndexMask) << 32) | (u64)p : 0ull;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int p = threadIdx.x + i * kThreads;
    if (p < size2) keys()[p] = by_index[i];
  }
  sort_list(size2);
  const int per2 = (size2 + kThreads - 1) / kThreads;
  mine = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int p = threadIdx.x * per2 + i;
    w[i] = (i < per2 && p < keep) ? weights()[(uint32_t)keys()[p]] : 0u;
    mine += w[i];
  }
  before = block_scan(mine, &sum);
  const u64 target = draw_target(u, kept_sum);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (before <= target && target < before + w[i])
      write_draw(a, row, (int)(~(uint32_t)(keys()[threadIdx.x * per2 + i] >> 32) & kIndexMask),
                 w[i], kept_sum);
    before += w[i];
  }
}

__device__ __forceinline__ void clear_hist() {
  Shared& sh = shared();
  uint32_t* h = &sh.hist.low[0][0];      // low, high, count
  for (int i = threadIdx.x; i < 3 * kBins * kCopies; i += kThreads) h[i] = 0u;
}

// Folds the copies of the histograms into bin_mass and bin_count.
template <bool COUNT, bool MASS> __device__ __forceinline__ void fold_hist() {
  Shared& sh = shared();
  const int copy = threadIdx.x & (kCopies - 1);
  for (int d = threadIdx.x / kCopies; d < kBins; d += kThreads / kCopies) {
    u64 m = MASS ? (u64)sh.hist.low[d][copy] + ((u64)sh.hist.high[d][copy] << 16) : 0ull;
    uint32_t c = COUNT ? sh.hist.count[d][copy] : 0u;
#pragma unroll
    for (int x = kCopies / 2; x > 0; x >>= 1) {
      if (MASS) m += __shfl_xor_sync(0xFFFFFFFFu, m, x);
      if (COUNT) c += __shfl_xor_sync(0xFFFFFFFFu, c, x);
    }
    if (copy == 0) {
      if (MASS) sh.bin_mass[d] = m;
      if (COUNT) sh.bin_count[d] = c;
    }
  }
}

// Additions in shared memory where x is above a limit (an if around
// atomicAdd() becomes a branch per token).
__device__ __forceinline__ void add_above(float x, float limit, uint32_t addr, uint32_t v) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.gt.f32 p, %2, %3;\n\t"
      "@p red.shared.add.u32 [%0], %1;\n\t}" ::"r"(addr),
      "r"(v), "f"(x), "f"(limit)
      : "memory");
}

// Where a row's cut is being looked for.
struct Search {
  u64 target;          // count or weight that the prefix has to reach
  u64 from;            // rank key of the last candidate (0: all)
  u64 before_count = 0, before_mass = 0;     // ahead of the open tokens
  int bin = -1;        // chosen quarter octave
  u64 prefix = 0;      // chosen leading digits of the rank key
  int shift = 8 * 7;   // bits of the rank key (32 + 20) still open
  bool clean = false;  // the histograms are as the kernel's start left them
};

// One round: a histogram of the open tokens, by quarter octave first and then
// by the next seven bits of the rank key, and in it the digit at which the
// running count (COUNT) or weight reaches the target.  For a nucleus the
// target follows from the first histogram, whose total is the sum of all
// weights.  False when the total stays below the target.
template <bool COUNT, typename P>
__device__ __noinline__ bool search_round(const P& pc, int q0, int q1,
                                          const Team& team, const Row& r, float top_p, Search& f) {
  Shared& sh = shared();
  constexpr int V = P::V;
  constexpr int kDigitBits = 7;
  const int copy = threadIdx.x & (kCopies - 1);
  const bool first = f.bin < 0;
  const int dshift = first ? f.shift : f.shift - kDigitBits;
  if (!f.clean) clear_hist();
  f.clean = false;
  if (threadIdx.x == 0) {
    sh.digit = -1;
    sh.listed = 0u;
  }
  __syncthreads();
  constexpr int kHigh = kBins * kCopies, kCount = 2 * kHigh;     // from a low sum to the others
  uint32_t* const hist = &sh.hist.low[0][copy];
  const uint32_t hist_addr = smem_u32(hist);
  if (first && f.from == 0ull) {
    pc.each(q0, q1, [&](const float (&v)[V], int) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float x = r.depth(v[j]);
        uint32_t high, low;
        Row::halves(Row::e(x), &high, &low);
        const uint32_t h = hist_addr + Row::bin_if_weight(x) * (kCopies * 4);
        // no weight from -31 down, no high half from -15 down
        add_above(x, -31.5f, h, low - Row::kOne);
        add_above(x, -15.5f, h + kHigh * 4, high - Row::kOne);
        if (COUNT) add_above(x, -31.5f, h + kCount * 4, (high | low) != Row::kOne ? 1u : 0u);
      }
    });
  } else {
    const float lowest = f.from ? rank_logit(f.from) : __int_as_float(0xFF800000);
    pc.each(q0, q1, [&](const float (&v)[V], int i0) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float l = v[j];
        if (!(l >= lowest)) continue;
        const float x = r.depth(l);
        const u64 key = rank_key(l, (uint32_t)(i0 + j));
        if (key < f.from) continue;
        int d = Row::bin(x);
        if (!first) {
          if (d != f.bin || (key >> f.shift) != f.prefix) continue;
          d = kBins - 1 - (int)((key >> dshift) & (kBins - 1));
        }
        const uint32_t w = Row::weight(Row::e(x));
        if (w == 0u) continue;
        atomicAdd(hist + d * kCopies, w & 0xFFFFu);
        atomicAdd(hist + d * kCopies + kHigh, w >> 16);
        if (COUNT) atomicAdd(hist + d * kCopies + kCount, 1u);
      }
    });
  }
  __syncthreads();
  fold_hist<COUNT, true>();
  team.sync();
  // every block joins the histograms and comes to the same choice
  u64 cnt = 0, mass = 0;
  if (threadIdx.x < kBins) {
    team.over(&sh.bin_mass[threadIdx.x], [&](u64 m, int) { mass += m; });
    if (COUNT) team.over(&sh.bin_count[threadIdx.x], [&](uint32_t c, int) { cnt += c; });
  }
  u64 total, total_count;
  const u64 to_mass = f.before_mass + block_scan(mass, &total);
  const u64 to_count = COUNT ? f.before_count + block_scan(cnt, &total_count) : 0ull;
  if (!COUNT && first) f.target = nucleus_target(top_p, total);
  const u64 lo = COUNT ? to_count : to_mass, hi = lo + (COUNT ? cnt : mass);
  if (lo < f.target && f.target <= hi) {
    sh.digit = (int)threadIdx.x;
    sh.before_count = to_count;
    sh.before_mass = to_mass;
  }
  __syncthreads();
  const int digit = sh.digit;
  if (digit < 0) return false;
  f.before_count = sh.before_count;
  f.before_mass = sh.before_mass;
  if (first) {
    f.bin = digit;
  } else {
    f.prefix = (f.prefix << kDigitBits) | (u64)(kBins - 1 - digit);
    f.shift = dshift;
  }
  return true;
}

// The distance below the maximum that is `bins` quarter octaves (4 * c may be
// above the largest float, for a temperature next to zero).
__device__ __forceinline__ float distance(const Row& r, float bins) {
  return bins * 0.25f / r.c;
}

// Generous bounds of the logits of quarter octave `bin`: no token of it lies
// outside, and none of a lower or higher one beyond the next.
__device__ __forceinline__ float bin_low(const Row& r, int bin) {
  return r.top - distance(r, (float)bin + 0.75f);
}
__device__ __forceinline__ float bin_high(const Row& r, int bin) {
  return r.top - distance(r, (float)bin - 0.75f);
}

// The open tokens, joined and ranked by the first block: the rank key of the
// one at which the target is reached.
template <bool COUNT>
__device__ __noinline__ u64 rank_open(const Team& team, const Row& r, const Search& f,
                                      int len) {
  Shared& sh = shared();
  join_lists(team);
  if (team.rank == 0) {
    if (len <= kCountRank) {
      const int p = threadIdx.x >> 2, part = threadIdx.x & 3;
      u64 key = 0;
      uint32_t w = 0;
      if (p < len) {
        key = keys()[p];
        w = Row::weight(Row::e(r.depth(rank_logit(key))));
        if (part == 0) weights()[p] = w;
      }
      __syncthreads();
      u64 ahead = 0;
      for (int j = part; j < len; j += 4)
        if (keys()[j] > key) ahead += ((u64)weights()[j] << 8) | 1u;
      ahead += __shfl_xor_sync(0xFFFFFFFFu, ahead, 1);
      ahead += __shfl_xor_sync(0xFFFFFFFFu, ahead, 2);
      const u64 mass = f.before_mass + (ahead >> 8);
      const u64 lo = COUNT ? f.before_count + (ahead & 255u) : mass;
      const u64 hi = lo + (COUNT ? 1ull : (u64)w);
      if (p < len && part == 0 && lo < f.target && f.target <= hi) {
        sh.cut = key;
      }
    } else {
      const int size = pow2_at_least(len);
      for (int i = len + threadIdx.x; i < size; i += kThreads) keys()[i] = 0ull;
      sort_list(size);
      const int per = (size + kThreads - 1) / kThreads;    // consecutive entries a thread
      const int p0 = threadIdx.x * per, p1 = min(p0 + per, len);
      u64 mine = 0;
      auto weight_at = [&](int p) {
        return Row::weight(Row::e(r.depth(rank_logit(keys()[p]))));
      };
      for (int p = p0; p < p1; ++p) mine += weight_at(p);
      u64 total;
      u64 mass = f.before_mass + block_scan(mine, &total);
      for (int p = p0; p < p1; ++p) {
        const uint32_t w = weight_at(p);
        const u64 lo = COUNT ? f.before_count + (u64)p : mass;
        const u64 hi = lo + (COUNT ? 1ull : (u64)w);
        if (lo < f.target && f.target <= hi) {
          sh.cut = keys()[p];
        }
        mass += w;
      }
    }
  }
  team.sync();
  return *team.of(&sh.cut, 0);         // (written again only after further syncs)
}

// The rank key of the last token of the shortest prefix that reaches the
// search's target; 0 when all tokens together do not.  `f` may have its first round behind it (`started`).
template <bool COUNT, typename P>
__device__ __noinline__ u64 find_cut(const P& pc, int q0, int q1, const Team& team,
                                     const Row& r, float top_p, Search& f, bool started) {
  Shared& sh = shared();
  constexpr int V = P::V;
  for (;;) {
    if (!started && !search_round<COUNT>(pc, q0, q1, team, r, top_p, f)) {
      team.sync();
      return 0ull;
    }
    if (!started) {
      // gather the open tokens; the bounds are generous, the test is exact
      const float low = bin_low(r, f.bin), high = bin_high(r, f.bin);
      pc.template each_above<2>(q0, q1, low, [&](const float (&v)[V], int i0) {
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (v[j] >= low && v[j] <= high) {
            const float x = r.depth(v[j]);
            const u64 key = rank_key(v[j], (uint32_t)(i0 + j));
            if (Row::weight(Row::e(x)) != 0u && Row::bin(x) == f.bin && key >= f.from &&
                (key >> f.shift) == f.prefix)
              append(team, key);
          }
      });
      team.sync();
      const u64 open = listed_by_all(team);
      if (open <= (u64)kOpen) return rank_open<COUNT>(team, r, f, (int)open);
    }
    started = false;
    team.sync();                       // counted by all before the next round clears
  }
}

// The draw, once every warp's stretches have their sums in sh.seg: `per`
// batches each; among tokens with e >= min_p and (CUT) a rank key >= `cut`.
template <bool CUT, typename P>
__device__ __noinline__ void draw_by_stretch(const SampleArgs& a, int row, const P& pc, int q0,
                                             int q1, int per, const Team& team,
                                             const Row& r, u64 cut, float u) {
  Shared& sh = shared();
  constexpr int V = P::V;
  constexpr int kBatch = 32 * kShares;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float lowest = rank_logit(cut);
  const int segs = per > 0 ? (q1 - q0 + per * kBatch - 1) / (per * kBatch) : 0;
  const u64 warp_total = warp_sum(lane < segs ? sh.seg[warp][lane] : 0ull);
  if (lane == 0) sh.red[warp] = warp_total;
  __syncthreads();
  u64 before = 0, block_total = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sh.red[w];
    block_total += sh.red[w];
  }
  if (threadIdx.x == 0) sh.sum = block_total;
  team.sync();
  u64 sum = 0;
  team.over(&sh.sum, [&](u64 t, int k) {
    if (k < team.rank) before += t;
    sum += t;
  });
  const u64 target = draw_target(u, sum);
  if (!(before <= target && target < before + warp_total)) return;
  // this warp's part holds the draw: find the stretch, then walk it
  int seg = 0;
  while (target >= before + sh.seg[warp][seg]) before += sh.seg[warp][seg++];
  const int e0 = q0 + seg * per * kBatch, e1 = min(q1, e0 + per * kBatch);
  for (int b = e0; b < e1; b += kBatch) {
    uint4 raw[kShares];
    pc.batch(b, e1, raw);
#pragma unroll 1
    for (int s = 0; s < kShares; ++s) {
      const int q = b + s * 32 + lane;
      const uint4 piece = raw[0];
#pragma unroll
      for (int i = 1; i < kShares; ++i) raw[i - 1] = raw[i];
      uint32_t w[V];
      u64 mine = 0;
      float v[V];
      P::values(piece, v);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float e = Row::e(r.depth(v[j]));
        bool kept = q < e1 && e >= r.min_p;
        if (CUT) kept = kept && v[j] >= lowest && rank_key(v[j], (uint32_t)(q * V - pc.mis + j)) >= cut;
        w[j] = kept ? Row::weight(e) : 0u;
        mine += w[j];
      }
      const u64 inc = warp_scan(mine);
      const u64 step = __shfl_sync(0xFFFFFFFFu, inc, 31);
      if (target < before + step) {
        u64 at = before + inc - mine;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          if (at <= target && target < at + w[j])
            write_draw(a, row, q * V - pc.mis + j, w[j], sum);
          at += w[j];
        }
        return;
      }
      before += step;
    }
  }
}

__device__ __forceinline__ int batches_per_stretch(int q0, int q1) {
  constexpr int kBatch = 32 * kShares;
  return ((q1 - q0 + kBatch - 1) / kBatch + kSegs - 1) / kSegs;
}

// Sums of weights' high and low 16 bits.  A stretch has at most 160 tokens of a
// lane, 5120 of a warp: 2^20 logits of 16 bits off a 16-byte boundary are 2^17 + 1
// pieces, of which one of 16 warps gets 8193, 65 batches, five a stretch.  So a
// warp's sums of them stay below 2^29.
struct Sums {
  uint32_t high, low;
};

// f(first piece, one past the last) -> this lane's sums, for every stretch of
// this warp; the warp's sums go to sh.seg.
template <typename F>
__device__ __forceinline__ void sum_stretches(int q0, int q1, int per, F f) {
  Shared& sh = shared();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int step = per * 32 * kShares;
  int seg = 0;
  for (int b = q0; b < q1; b += step, ++seg) {
    const Sums s = f(b, min(q1, b + step));
    const uint32_t high = __reduce_add_sync(0xFFFFFFFFu, s.high);
    const uint32_t low = __reduce_add_sync(0xFFFFFFFFu, s.low);
    if (lane == 0) sh.seg[warp][seg] = ((u64)high << 16) + low;
  }
}

// The draw over the whole row among tokens with e >= min_p (0 without MIN_P)
// and (CUT) a rank key of at least `cut`.
template <bool CUT, bool MIN_P, typename P>
__device__ __noinline__ void draw_in_row(const SampleArgs& a, int row, const P& pc, int q0, int q1,
                                         const Team& team, const Row& r, u64 cut,
                                         float u) {
  Shared& sh = shared();
  constexpr int V = P::V;
  const float lowest = rank_logit(cut);
  const int per = batches_per_stretch(q0, q1);
  sum_stretches(q0, q1, per, [&](int b0, int b1) {
    uint32_t high = 0, low = 0;
    if constexpr (CUT) {
      pc.template each_above<2>(b0, b1, lowest, [&](const float (&v)[V], int i0) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          if (!(v[j] >= lowest) ||
              (v[j] == lowest && rank_key(v[j], (uint32_t)(i0 + j)) < cut))
            continue;
          const float e = Row::e(r.depth(v[j]));
          const uint32_t w = e >= r.min_p ? Row::weight(e) : 0u;
          high += w >> 16;
          low += w & 0xFFFFu;
        }
      });
    } else {
      uint32_t pieces = 0;             // the halves' sums have kOne in them, modulo 2^32
      pc.each(b0, b1, [&](const float (&v)[V], int) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          float e = Row::e(r.depth(v[j]));
          e = MIN_P ? (e >= r.min_p ? e : 0.f) : fmaxf(e, 0.f);      // (a NaN: 0)
          uint32_t h, l;
          Row::halves(e, &h, &l);
          high += h;
          low += l;
        }
        ++pieces;
      });
      const uint32_t ones = pieces * (uint32_t)V * Row::kOne;
      high -= ones;
      low -= ones;
    }
    return Sums{high, low};
  });
  __syncthreads();
  draw_by_stretch<CUT>(a, row, pc, q0, q1, per, team, r, cut, u);
}

// A nucleus (within the tokens of rank key >= from) and the draw in it.
template <typename P>
__device__ __noinline__ void draw_nucleus(const SampleArgs& a, int row, const P& pc, int q0,
                                          int q1, const Team& team, const Row& r,
                                          u64 from, float top_p, float u, bool clean) {
  Shared& sh = shared();
  constexpr int V = P::V;
  Search f;
  f.from = from;
  f.clean = clean;
  // (always found: the largest weight is 2^31)
  search_round<false>(pc, q0, q1, team, r, top_p, f);
  const float low = bin_low(r, f.bin);
  const int per = batches_per_stretch(q0, q1);
  sum_stretches(q0, q1, per, [&](int b0, int b1) {
    uint32_t high_sum = 0, low_sum = 0, pieces = 0;  // of halves, as in draw_in_row()
    pc.template each_above<2>(b0, b1, low, [&](const float (&v)[V], int i0) {
      uint32_t open = 0;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float x = r.depth(v[j]);
        const float e = Row::e(x);
        const int b = (int)Row::bin_if_weight(x);    // (past the bins without a weight)
        uint32_t h, l;                               // above the open ones: kept
        Row::halves(b < f.bin && e >= r.min_p ? e : 0.f, &h, &l);
        high_sum += h;
        low_sum += l;
        open |= (b == f.bin && e >= 0x1p-31f ? 1u : 0u) << j;
      }
      ++pieces;
      if (open != 0u) {                // one addition to the list's length per piece
        uint32_t at = from == 0ull ? atomicAdd(&sh.listed, (uint32_t)__popc(open)) : 0u;
        for (; open != 0u; open &= open - 1u) {
          const int idx = i0 + __ffs((int)open) - 1;
          const u64 key = rank_key(pc.element(idx), (uint32_t)idx);
          if (from != 0ull) {
            if (key >= from) append(team, key);
          } else {
            put(team, at++, key);
          }
        }
      }
    });
    const uint32_t ones = pieces * (uint32_t)V * Row::kOne;
    return Sums{high_sum - ones, low_sum - ones};
  });
  team.sync();
  const u64 open = listed_by_all(team);
  if (open > (u64)kOpen) {
    const u64 cut = find_cut<false>(pc, q0, q1, team, r, top_p, f, true);
    draw_in_row<true, true>(a, row, pc, q0, q1, team, r, cut, u);
    return;
  }
  const u64 cut = rank_open<false>(team, r, f, (int)open);
  // this block's open tokens that are kept join their stretches' sums (the
  // first block's list is the joined one now)
  const int parts = team.size * kWarps;
  const int mine = team.rank == 0 ? (int)open : (int)sh.listed;
  for (int i = threadIdx.x; i < mine; i += kThreads) {
    const u64 key = keys()[i];
    const float e = Row::e(r.depth(rank_logit(key)));
    if (key < cut || !(e >= r.min_p)) continue;
    const int q = ((int)rank_index(key) + pc.mis) / V;
    const int part = pc.part_of(q, parts);
    if (part / kWarps != team.rank) continue;
    const int p0 = pc.first(part, parts), p1 = pc.first(part + 1, parts);
    const int seg = (q - p0) / (batches_per_stretch(p0, p1) * 32 * kShares);
    atomicAdd(&sh.seg[part - team.rank * kWarps][seg], (u64)Row::weight(e));
  }
  __syncthreads();
  draw_by_stretch<true>(a, row, pc, q0, q1, per, team, r, cut, u);
}

// A row whose maximum is +inf: the infinite logits share the draw, a weight
// of 2^31 each, ranked by index.
template <typename P>
__device__ __noinline__ void draw_infinite(const SampleArgs& a, int row, const P& pc,
                                           int q0, int q1, const Team& team, int top_k,
                                           float top_p, float u) {
  Shared& sh = shared();
  constexpr int V = P::V;
  const int lane = threadIdx.x & 31;
  const float inf = __int_as_float(0x7F800000);
  u64 mine = 0;
  pc.each(q0, q1, [&](const float (&v)[V], int) {
#pragma unroll
    for (int j = 0; j < V; ++j) mine += v[j] == inf;
  });
  const u64 warp_total = warp_sum(mine);
  u64 total;
  u64 before = block_scan(lane == 0 ? warp_total : 0ull, &total);   // of lane 0
  before = __shfl_sync(0xFFFFFFFFu, before, 0);
  if (threadIdx.x == 0) sh.sum = total;
  team.sync();
  u64 kept = 0;
  team.over(&sh.sum, [&](u64 t, int k) {
    if (k < team.rank) before += t;
    kept += t;
  });
  if (top_k > 0 && (u64)top_k < kept) kept = (u64)top_k;
  if (top_p < 1.f) kept = (nucleus_target(top_p, kept << 31) + 0x7FFFFFFFull) >> 31;
  const u64 target = draw_target(u, kept << 31) >> 31;
  for (int q = q0 + lane; q - lane < q1; q += 32) {
    float v[V];
    int c = 0;
    if (q < q1) P::values(pc.load(q), v);
#pragma unroll
    for (int j = 0; j < V; ++j) c += q < q1 && v[j] == inf;
    const u64 inc = warp_scan((u64)c);
    u64 at = before + inc - c;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (q < q1 && v[j] == inf && at++ == target)
        write_draw(a, row, q * V - pc.mis + j, 1u << 31, kept << 31);
    before += __shfl_sync(0xFFFFFFFFu, inc, 31);
  }
}

template <typename T, Mode MODE>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs a) {
  Shared& sh = shared();
  using P = Pieces<T, MODE>;
  constexpr bool HELD = P::HELD;
  constexpr int V = P::V;
  const Team team;
  const int row = blockIdx.x / team.size;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  P pc(reinterpret_cast<const T*>(a.logits) + (size_t)row * a.n, a.n);
  // this warp's pieces
  const int parts = team.size * kWarps, part = team.rank * kWarps + warp;
  const int q0 = pc.first(part, parts), q1 = pc.first(part + 1, parts);
  pc.s0 = pc.first(team.rank * kWarps, parts);
  if (threadIdx.x == 0) {
    if constexpr (HELD) {
      for (int c = 0; c < kChunks; ++c) mbar_init(&sh.bars[c], 1);
      mbar_init(&sh.stall, 1);
    }
    sh.failed = 0;
    sh.listed = 0u;
    sh.digit = -1;
    sh.cut = 0ull;
    sh.sum = 0ull;
    if constexpr (HELD) fence_barrier_init();
  }
  clear_hist();
  __syncthreads();
  griddep_launch_dependents();
  griddep_wait();

  if constexpr (HELD) {
    if (threadIdx.x == 0) {
      // whole pieces inside the row; the ends are read one element at a time
      for (int c = 0; c < kChunks; ++c) {
        const int w0 = team.rank * kWarps + c * (kWarps / kChunks);
        const int b0 = max(pc.first(w0, parts), 1);
        const int b1 = min(pc.first(w0 + kWarps / kChunks, parts), pc.pieces - 1);
        const uint32_t bytes = b1 > b0 ? (uint32_t)(b1 - b0) * 16u : 0u;
        mbar_arrive_expect_tx(&sh.bars[c], bytes);
        if (bytes) bulk_load(held_pieces() + (b0 - pc.s0), pc.base + (size_t)b0 * V, bytes, &sh.bars[c]);
      }
    }
    if (lane == 0 && q0 == 0 && q1 > 0) held_pieces()[0 - pc.s0] = pc.load_end(0);
    if (lane == 0 && q0 < pc.pieces && q1 == pc.pieces)
      held_pieces()[pc.pieces - 1 - pc.s0] = pc.load_end(pc.pieces - 1);
    __syncwarp();
  } else if constexpr (MODE == kRagged) {
    if (threadIdx.x < 2) held_pieces()[threadIdx.x] = pc.load_end(threadIdx.x ? pc.pieces - 1 : 0);
    __syncthreads();
  }

  const float t = a.temperature ? a.temperature[row] : 1.f;
  const float u = a.u[row];
  int top_k = a.top_k ? a.top_k[row] : 0;
  if (top_k >= a.n || top_k < 0) top_k = 0;
  float top_p = a.top_p ? a.top_p[row] : 1.f;
  if (!(top_p < 1.f)) top_p = 1.f;
  Row r;
  r.min_p = a.min_p ? a.min_p[row] : 0.f;
  r.min_p = r.min_p > 0.f ? fminf(r.min_p, 1.f) : 0.f;
  r.c = fminf(__fdiv_rn(kLog2e, t), 3.402823466e38f);

  if constexpr (HELD) {
    uint64_t* bar = a.diag_stall ? &sh.stall : &sh.bars[warp / (kWarps / kChunks)];
    if (!mbar_wait(bar, 0u, a.wait_budget)) sh.failed = 1;
    __syncwarp();
  }

  // the maximum
  float share[kShares];
#pragma unroll
  for (int s = 0; s < kShares; ++s) share[s] = __int_as_float(0xFF800000);
  pc.template each_piece<kShares>(q0, q1, [&](const uint4& piece, int, int s) {
    share[s] = fmaxf(share[s], P::max_of(piece));
  });
  float mx = fmaxf(fmaxf(share[0], share[1]), fmaxf(share[2], share[3]));
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, m));
  if (lane == 0) sh.redf[warp] = mx;
  __syncthreads();
  mx = sh.redf[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, sh.redf[w]);
  // (a block whose copies did not come makes the row's maximum a NaN)
  if (threadIdx.x == 0) sh.max = HELD && sh.failed ? __int_as_float(0x7FC00000) : mx;
  team.sync();
  bool failed = false;
  team.over(&sh.max, [&](float m, int) {
    mx = fmaxf(mx, m);
    if constexpr (HELD) failed = failed || m != m;
  });
  r.top = mx;

  if (failed || mx == __int_as_float(0xFF800000)) {    // nothing left
    if (HELD && sh.failed && threadIdx.x == 0) {
      // no copy may be in flight when the block ends: its shared memory goes to
      // the next one (one more budget, for all of them)
      const long long t0 = clock64();
      for (int c = 0; c < kChunks; ++c) mbar_wait_since(&sh.bars[c], 0u, t0);
    }
    if (team.rank == 0 && threadIdx.x == 0) {
      a.ids[row] = failed ? -2 : -1;
      if (a.logp) a.logp[row] = __int_as_float(0x7FC00000);
    }
    team.sync();
    return;
  }
  if (!(t > 0.f)) {                                    // greedy: the first maximum
    int at = 0x7FFFFFFF;
    pc.each(q0, q1, [&](const float (&v)[V], int i0) {
#pragma unroll
      for (int j = V - 1; j >= 0; --j)
        if (v[j] == mx) at = min(at, i0 + j);
    });
    at = __reduce_min_sync(0xFFFFFFFFu, at);
    if (lane == 0) sh.red[warp] = (u64)(uint32_t)at;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) at = min(at, (int)sh.red[w]);
    if (threadIdx.x == 0) sh.sum = (u64)(uint32_t)at;
    team.sync();
    if (team.rank == 0 && threadIdx.x == 0) {
      team.over(&sh.sum, [&](u64 v, int) { at = min(at, (int)v); });
      a.ids[row] = at;
      if (a.logp) a.logp[row] = 0.f;
    }
    team.sync();
    return;
  }
  if (mx == __int_as_float(0x7F800000)) {
    draw_infinite(a, row, pc, q0, q1, team, top_k, top_p, u);
    team.sync();
    return;
  }

  if (top_k > 0 && top_k <= kMaxListK) {
    // the bound: enough share maxima reach it
    const int copy = threadIdx.x & (kCopies - 1);
#pragma unroll
    for (int s = 0; s < kShares; ++s) {
      const float x = r.depth(share[s]);
      if (x > -31.f) atomicAdd(&sh.hist.count[Row::bin(x)][copy], 1u);
    }
    __syncthreads();
    fold_hist<true, false>();
    team.sync();
    u64 cnt = 0;
    if (threadIdx.x < kBins)
      team.over(&sh.bin_count[threadIdx.x], [&](uint32_t c, int) { cnt += c; });
    u64 total;
    const u64 below = block_scan(cnt, &total);
    if (below < (u64)top_k && (u64)top_k <= below + cnt) sh.digit = (int)threadIdx.x;
    __syncthreads();
    const bool all = sh.digit < 0;
    // (a little below the edge, against the rounding here)
    const float bound = all ? __int_as_float(0xFF800000)
                            : r.top - distance(r, (float)sh.digit + 0.5f + 1e-3f);
    pc.template each_above<4>(q0, q1, bound, [&](const float (&v)[V], int i0) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (v[j] >= bound && Row::weight(Row::e(r.depth(v[j]))) != 0u)
          append(team, rank_key(v[j], (uint32_t)(i0 + j)));
    });
    team.sync();
    const u64 listed = listed_by_all(team);
    if (listed <= (u64)kList && (all || listed >= (u64)top_k)) {
      join_lists(team);
      if (team.rank == 0) {
        if (listed <= (u64)kCountRank)
          finish_by_counting(a, row, r, (int)listed, top_k, top_p, u);
        else
          finish_by_sorting(a, row, r, (int)listed, top_k, top_p, u);
      }
      team.sync();
      return;
    }
    team.sync();                                       // counted by all before it is cleared
  }

  u64 cut = 0;
  if (top_k > 0) {
    Search f;
    f.from = 0ull;
    f.target = (u64)top_k;
    cut = find_cut<true>(pc, q0, q1, team, r, 1.f, f, false);
  }
  if (top_p < 1.f)
    draw_nucleus(a, row, pc, q0, q1, team, r, cut, top_p, u, top_k <= 0);
  else if (cut != 0ull)
    draw_in_row<true, true>(a, row, pc, q0, q1, team, r, cut, u);
  else if (r.min_p > 0.f)
    draw_in_row<false, true>(a, row, pc, q0, q1, team, r, cut, u);
  else
    draw_in_row<false, false>(a, row, pc, q0, q1, team, r, cut, u);
  team.sync();
}

// Blocks per row: as many as still give every row its own share of the SMs
// (two blocks fit one), with at least 4096 logits each.  (256 x 151936 bf16
// with four blocks per row, so that shared memory holds them, takes 66 us for
// top-k and 137 us for a nucleus, most of it in the clusters' barriers; with
// one block per row 31 and 100.)
int cluster_size(int m, int n) {
  int c = 1;
  while (c < kMaxCluster && 2ll * c * m <= 2ll * device_sm_count() && n / (2 * c) >= 4096) c *= 2;
  return c;
}

template <typename T, Mode MODE>
cudaError_t launch_h(const SampleArgs& a, int c, cudaStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);
  const int slice = ((a.n + V - 1) / V + 1 + c - 1) / c + 1;     // pieces of a block, at most
  const size_t smem = sizeof(Shared) + (size_t)(MODE == kHeld ? slice : 2) * 16;
  auto kern = sample_kernel<T, MODE>;
  static LargestPerDevice limit;
  cudaError_t e = allow_smem(limit, kern, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.m * c);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)c;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kern, a);
  note_launch();
  return e;
}

template <typename T>
cudaError_t launch_t(const SampleArgs& a, cudaStream_t s) {
  const int c = cluster_size(a.m, a.n);
  if ((size_t)a.n * sizeof(T) / c + 64 <= (size_t)kHeldBytes) return launch_h<T, kHeld>(a, c, s);
  if (a.n % (16 / (int)sizeof(T)) == 0 && reinterpret_cast<uintptr_t>(a.logits) % 16 == 0)
    return launch_h<T, kWhole>(a, c, s);
  return launch_h<T, kRagged>(a, c, s);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, cudaStream_t s) {
  switch (a.dtype) {
    case WQL_F32: return launch_t<float>(a, s);
    case WQL_F16: return launch_t<__half>(a, s);
    default: return launch_t<__nv_bfloat16>(a, s);
  }
}

}  // namespace wql
