// sample.cu -- draw the next token of every row: temperature, top-k, top-p
// and min-p, from a given random number.
//
// Weights are integers, W = floor(2^31 * exp2((l - max) * log2e / t)), so
// every sum is exact and the same in any order; ranks go by logit descending,
// then index ascending.  Each filter keeps a prefix of that order, so a row's
// filters come down to one cut, the rank key of the last kept token:
// (order-preserving bits of the logit, inverted index).
//
// One cluster of 1 to 8 blocks per row, each over a contiguous slice:
//  * the maximum (and those of four shares of each thread's elements);
//  * top-k up to 768: a bound that about k logits reach, from a histogram of
//    the share maxima (k values at least as large exist if k maxima do); one
//    pass gathers the logits above it; the first block ranks that list,
//    applies the filters by prefix sums and draws;
//  * a nucleus, or a larger top-k: a histogram of the weights (counts) over
//    quarter octaves below the maximum finds the one that holds the cut, a
//    second pass gathers its tokens, the first block ranks them; while they do
//    not fit the list, further histograms over seven bits of the rank key at a
//    time narrow them.  The draw then runs over the row by index, as it does
//    when temperature or min-p alone is on: sums per stretch of the row, then
//    a walk through the one stretch that holds the draw.
//
// What bounds it: two passes at least over a row that the second time comes
// from L2, and per weight some ten instructions, among them an exponential
// and a conversion on the slow unit.  The loops over a row are kept short (one
// 16-byte piece a turn, the next three in flight): unrolled by four they were
// bound by instruction fetches (64 x 248320 fp32, temperature alone: 44.7 us).  Histograms keep 32 copies, one per lane, so that a
// warp's additions never meet in a bank; a copy's sums (16 low and 15 high bits
// of the weights apart) stay below 2^32 for 2^20 tokens.
#include <cooperative_groups.h>

#include "mx.cuh"

namespace cg = cooperative_groups;

namespace wql {
namespace {

typedef unsigned long long u64;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kList = 2048;          // tokens the list holds
constexpr int kBins = 128;
constexpr int kShares = 4;           // maxima kept per thread; loads in flight per thread
constexpr int kSegs = 32;            // stretches of a warp's part of the row
constexpr int kMaxCluster = 8;
constexpr int kMaxListK = 768;       // largest top-k that goes by a bound and a list
constexpr int kCountRank = 128;      // lists up to this long are ranked by counting
constexpr int kIndexBits = 20;
constexpr float kLog2e = 1.44269504088896340736f;
static_assert(WQL_SAMPLE_MAX_N == 1 << kIndexBits, "rank keys hold an index");

struct Shared {
  uint32_t low[kBins][32];           // sums of weights' low 16 bits, by lane
  uint32_t high[kBins][32];          // and of the bits above
  uint32_t count[kBins][32];
  u64 list[kList];
  uint32_t weight[kList];
  u64 seg[kWarps][kSegs];
  u64 red[kWarps];
  float redf[kWarps];
  // read by the other blocks of the cluster
  u64 bin_mass[kBins];
  uint32_t bin_count[kBins];
  float max;
  u64 sum;
  uint32_t listed;
  u64 cut;                           // of the first block
  int done;
  // block-wide results
  int digit;
  u64 before_count, before_mass;
};

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
  // log2 of a token's weight over the likeliest's (NaN for a NaN; top is
  // finite here, and so is c)
  __device__ __forceinline__ float depth(float l) const {
    return __fmul_rn(__fsub_rn(l, top), c);
  }
  // 2^x; the same bits as exp2f() from -126 up, and W = 0 below -31 anyway
  static __device__ __forceinline__ float e(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
  }
  // (a NaN converts to 0)
  static __device__ __forceinline__ uint32_t weight(float e) {
    return __float2uint_rz(e * 2147483648.f);
  }
  // quarter octaves below the maximum, rounded to the nearest: never
  // decreasing with the logit's rank, at most 124 for a token with a weight
  static __device__ __forceinline__ int bin(float x) {
    return (int)min(__float_as_uint(fmaf(x, -4.f, 8388608.f)) - 0x4B000000u,
                    (uint32_t)(kBins - 1));
  }
};

// A row of logits in 16-byte pieces on 16-byte addresses: piece q holds
// elements q*V - mis .. + V-1; those outside the row read as -inf.
template <typename T> struct Pieces {
  static constexpr int V = 16 / (int)sizeof(T);
  const T* base;       // 16-byte aligned, mis elements before the row
  int mis, n, pieces;
  __device__ __forceinline__ Pieces(const T* row, int n_) : n(n_) {
    mis = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    base = row - mis;
    pieces = (n + mis + V - 1) / V;
  }
  __device__ __forceinline__ uint4 load(int q) const {
    if (q > 0 && q < pieces - 1) return __ldg(reinterpret_cast<const uint4*>(base) + q);
    return load_end(q);
  }
  // the first or last piece, which may reach outside the row
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
  // This lane's pieces of the batch at b (32 * kShares consecutive pieces).
  __device__ __forceinline__ void batch(int b, int q1, uint4 (&r)[kShares]) const {
#pragma unroll
    for (int u = 0; u < kShares; ++u) {
      const int q = b + u * 32 + (int)(threadIdx.x & 31);
      r[u] = q < q1 ? load(q) : make_uint4(0u, 0u, 0u, 0u);
    }
  }
  // f(values, index of the first) for this warp's pieces q0 .. q1, one a turn
  template <typename F> __device__ __forceinline__ void each(int q0, int q1, F f) const {
    int q = q0 + (int)(threadIdx.x & 31);
    uint4 r0, r1, r2;
    if (q < q1) r0 = load(q);
    if (q + 32 < q1) r1 = load(q + 32);
    if (q + 64 < q1) r2 = load(q + 64);
#pragma unroll 1
    for (; q < q1; q += 32) {
      const uint4 r = r0;
      r0 = r1;
      r1 = r2;
      if (q + 96 < q1) r2 = load(q + 96);
      float v[V];
      values(r, v);
      f(v, q * V - mis);
    }
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
__device__ u64 block_scan(u64 v, Shared& sh, u64* total) {
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

// Sorts sh.list[0 .. size) descending; size a power of two, at least 2.
__device__ void sort_list(Shared& sh, int size) {
  __syncthreads();
  for (int len = 2; len <= size; len <<= 1) {
    for (int stride = len >> 1; stride > 0; stride >>= 1) {
      for (int i = threadIdx.x; i < size / 2; i += kThreads) {
        const int p = 2 * i - (i & (stride - 1));
        const u64 a = sh.list[p], b = sh.list[p + stride];
        const bool up = (p & len) != 0;              // ascending stretch
        if (up ? a > b : a < b) {
          sh.list[p] = b;
          sh.list[p + stride] = a;
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

__device__ __forceinline__ void append(Shared& sh, u64 key) {
  const uint32_t at = atomicAdd(&sh.listed, 1u);
  if (at < (uint32_t)kList) sh.list[at] = key;
}

// Tokens listed by all blocks of the cluster.  After a sync that follows the
// gathering; the caller syncs before the lists are used again.
__device__ __forceinline__ u64 listed_by_all(Shared& sh, const Team& team) {
  u64 total = 0;
  team.over(&sh.listed, [&](uint32_t c, int) { total += c; });
  return total;
}

// The first block's list gets those of the others appended (they fit).
__device__ void join_lists(Shared& sh, const Team& team) {
  if (team.rank != 0) return;
  uint32_t at = sh.listed;
  for (int r = 1; r < team.size; ++r) {
    const uint32_t c = *team.of(&sh.listed, r);
    const u64* src = team.of(&sh.list[0], r);
    for (uint32_t i = threadIdx.x; i < c; i += kThreads) sh.list[at + i] = src[i];
    at += c;
  }
  __syncthreads();
}

// The integer that a nucleus' weights have to reach: those before a kept
// token sum to less than p * sum, so to less than its ceiling.
__device__ __forceinline__ u64 nucleus_target(float p, u64 sum) {
  const double t = ceil((double)p * (double)sum);
  return t < 1.0 ? 1ull : (u64)t;
}

__device__ __forceinline__ u64 draw_target(float u, u64 sum) {
  const double r = (double)u * (double)sum;
  const u64 v = r > 0.0 ? (u64)r : 0ull;
  return v < sum ? v : sum - 1;
}

__device__ __forceinline__ void write_draw(const SampleArgs& a, int row, int id, uint32_t w,
                                           u64 sum) {
  a.ids[row] = id;
  if (a.logp) a.logp[row] = logf(__fdiv_rn((float)w, (float)sum));
}

// Top-k, top-p, min-p and draw among the `len` tokens of the first block's
// list, which hold the first top_k by rank (or, fewer, all with a weight).
// Short lists: every token counts the tokens and sums the weights before it,
// by rank and then, among the kept, by index.
__device__ __noinline__ void finish_by_counting(const SampleArgs& a, int row, Shared& sh,
                                                const Row& r, int len, int top_k, float top_p,
                                                float u) {
  static_assert(kThreads == 4 * kCountRank, "four lanes a token");
  const int p = threadIdx.x >> 2, part = threadIdx.x & 3;
  u64 key = 0;
  float e = 0.f;
  uint32_t w = 0;
  if (p < len) {
    key = sh.list[p];
    e = Row::e(r.depth(rank_logit(key)));
    w = Row::weight(e);
    if (part == 0) sh.weight[p] = w;
  }
  __syncthreads();
  u64 before = 0;                      // weights before it by rank, and how many tokens
  for (int j = part; j < len; j += 4)
    if (sh.list[j] > key) before += ((u64)sh.weight[j] << 8) | 1u;
  before += __shfl_xor_sync(0xFFFFFFFFu, before, 1);
  before += __shfl_xor_sync(0xFFFFFFFFu, before, 2);
  const bool in_k = p < len && (int)(before & 255u) < top_k;
  before >>= 8;
  u64 sum = ~0ull;
  if (top_p < 1.f) block_scan(in_k && part == 0 ? w : 0u, sh, &sum);
  const bool keep = in_k && (top_p >= 1.f || before < nucleus_target(top_p, sum)) && e >= r.min_p;
  u64 kept;
  block_scan(keep && part == 0 ? w : 0u, sh, &kept);
  if (p < len && !keep && part == 0) sh.weight[p] = 0u;
  __syncthreads();
  u64 run = 0;                         // kept weights of lower indices
  const uint32_t idx = rank_index(key);
  for (int j = part; j < len; j += 4)
    if (rank_index(sh.list[j]) < idx) run += sh.weight[j];
  run += __shfl_xor_sync(0xFFFFFFFFu, run, 1);
  run += __shfl_xor_sync(0xFFFFFFFFu, run, 2);
  const u64 target = draw_target(u, kept);
  if (keep && part == 0 && run <= target && target < run + w)
    write_draw(a, row, (int)idx, w, kept);
}

// The same for longer lists: sort, prefix sums, sort the kept by index.
__device__ __noinline__ void finish_by_sorting(const SampleArgs& a, int row, Shared& sh, const Row& r, int len,
                                  int top_k, float top_p, float u) {
  const int size = pow2_at_least(len);
  for (int i = len + threadIdx.x; i < size; i += kThreads) sh.list[i] = 0ull;
  sort_list(sh, size);
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
      e[i] = Row::e(r.depth(rank_logit(sh.list[p])));
      w[i] = Row::weight(e[i]);
      mine += w[i];
    }
  }
  u64 sum;
  u64 before = block_scan(mine, sh, &sum);
  const u64 reach = top_p < 1.f ? nucleus_target(top_p, sum) : ~0ull;
  // keep a prefix: count it, and its weights
  u64 kept = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int p = threadIdx.x * per + i;
    if (i < per && p < limit && before < reach && e[i] >= r.min_p)
      kept += ((u64)w[i] << 12) | 1u;                  // up to 2^11 weights of 2^31, and a count
    before += w[i];
    if (i < per && p < kList) sh.weight[p] = w[i];
  }
  u64 kept_total;
  block_scan(kept, sh, &kept_total);
  const int keep = (int)(kept_total & 0xFFFu);
  const u64 kept_sum = kept_total >> 12;
  // the kept tokens by index: (inverted index, rank), descending
  u64 by_index[kPer];
  const int size2 = pow2_at_least(keep);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int p = threadIdx.x + i * kThreads;
    by_index[i] = p < keep ? ((sh.list[p] & kIndexMask) << 32) | (u64)p : 0ull;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int p = threadIdx.x + i * kThreads;
    if (p < size2) sh.list[p] = by_index[i];
  }
  sort_list(sh, size2);
  const int per2 = (size2 + kThreads - 1) / kThreads;
  mine = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int p = threadIdx.x * per2 + i;
    w[i] = (i < per2 && p < keep) ? sh.weight[(uint32_t)sh.list[p]] : 0u;
    mine += w[i];
  }
  before = block_scan(mine, sh, &sum);
  const u64 target = draw_target(u, kept_sum);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (before <= target && target < before + w[i])
      write_draw(a, row, (int)(~(uint32_t)(sh.list[threadIdx.x * per2 + i] >> 32) & kIndexMask),
                 w[i], kept_sum);
    before += w[i];
  }
}

// The rank key of the last token of the shortest prefix, in rank order among
// the tokens with a weight and a rank key of at least `from`, whose count
// (COUNT) or sum of weights reaches a target; 0 when there is none.  For a
// nucleus the target follows from the first histogram, whose total is the sum
// of all weights.  *mass_out gets the prefix's sum of weights.
template <bool COUNT, typename T>
__device__ __noinline__ u64 find_cut(const Pieces<T>& pc, int q0, int q1, Shared& sh, const Team& team,
                        const Row& r, int top_k, float top_p, u64 from, u64* mass_out) {
  constexpr int V = Pieces<T>::V;
  constexpr int kDigitBits = 7;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  u64 before_count = 0, before_mass = 0, target = (u64)top_k;
  float lowest = from ? rank_logit(from) : __int_as_float(0xFF800000);   // of the open tokens
  int bin = -1;                      // chosen quarter octave
  u64 prefix = 0;                    // chosen leading digits of the rank key
  int shift = 8 * kDigitBits;        // bits of the rank key (32 + 20) still open
  for (;;) {
    const bool first = bin < 0;
    const int dshift = first ? shift : shift - kDigitBits;
    if (threadIdx.x == 0) sh.digit = -1;
    __syncthreads();
    auto add = [&](int d, uint32_t w) {
      if (w != 0u) atomicAdd(&sh.low[d][lane], w & 0xFFFFu);
      if (w > 0xFFFFu) atomicAdd(&sh.high[d][lane], w >> 16);
      if (COUNT && w != 0u) atomicAdd(&sh.count[d][lane], 1u);
    };
    if (first && from == 0ull) {
      pc.each(q0, q1, [&](const float (&v)[V], int) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float x = r.depth(v[j]);
          add(Row::bin(x), Row::weight(Row::e(x)));
        }
      });
    } else {
      pc.each(q0, q1, [&](const float (&v)[V], int i0) {
#pragma unroll 1
        for (int j = 0; j < V; ++j) {
          const float l = v[j];
          if (!(l >= lowest)) continue;
          const float x = r.depth(l);
          const u64 key = rank_key(l, (uint32_t)(i0 + j));
          if (key < from) continue;
          int d = Row::bin(x);
          if (!first) {
            if (d != bin || (key >> shift) != prefix) continue;
            d = kBins - 1 - (int)((key >> dshift) & (kBins - 1));
          }
          add(d, Row::weight(Row::e(x)));
        }
      });
    }
    __syncthreads();
    // fold the lanes' copies, and clear them for the next time
    for (int d = warp; d < kBins; d += kWarps) {
      const u64 m = warp_sum((u64)sh.low[d][lane] + ((u64)sh.high[d][lane] << 16));
      sh.low[d][lane] = 0u;
      sh.high[d][lane] = 0u;
      uint32_t c = 0;
      if (COUNT) {
        c = __reduce_add_sync(0xFFFFFFFFu, sh.count[d][lane]);
        sh.count[d][lane] = 0u;
      }
      if (lane == 0) {
        sh.bin_mass[d] = m;
        sh.bin_count[d] = c;
      }
    }
    team.sync();
    // every block joins the histograms and comes to the same choice
    u64 cnt = 0, mass = 0;
    if (threadIdx.x < kBins) {
      team.over(&sh.bin_mass[threadIdx.x], [&](u64 m, int) { mass += m; });
      if (COUNT) team.over(&sh.bin_count[threadIdx.x], [&](uint32_t c, int) { cnt += c; });
    }
    u64 total_mass, total_count;
    const u64 to_mass = before_mass + block_scan(mass, sh, &total_mass);
    const u64 to_count = COUNT ? before_count + block_scan(cnt, sh, &total_count) : 0ull;
    if (!COUNT && first) target = nucleus_target(top_p, total_mass);
    const u64 lo = COUNT ? to_count : to_mass, hi = lo + (COUNT ? cnt : mass);
    if (lo < target && target <= hi) {
      sh.digit = (int)threadIdx.x;
      sh.before_count = to_count;
      sh.before_mass = to_mass;
    }
    if (threadIdx.x == 0) sh.listed = 0u;
    __syncthreads();
    const int digit = sh.digit;
    if (digit < 0) {                 // (top-k only: fewer tokens than that have a weight)
      *mass_out = total_mass;
      team.sync();
      return 0ull;
    }
    before_count = sh.before_count;
    before_mass = sh.before_mass;
    if (first) {
      bin = digit;
    } else {
      prefix = (prefix << kDigitBits) | (u64)(kBins - 1 - digit);
      shift = dshift;
    }
    // gather the open tokens; the bounds are generous, the test is exact
    const float low_b = r.top - ((float)bin + 0.75f) / (4.f * r.c);
    const float high_b = r.top - ((float)bin - 0.75f) / (4.f * r.c);
    if (low_b > lowest) lowest = low_b;
    pc.each(q0, q1, [&](const float (&v)[V], int i0) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (v[j] >= lowest && v[j] <= high_b) {
          const float x = r.depth(v[j]);
          const u64 key = rank_key(v[j], (uint32_t)(i0 + j));
          if (Row::weight(Row::e(x)) != 0u && Row::bin(x) == bin && key >= from &&
              (key >> shift) == prefix)
            append(sh, key);
        }
    });
    team.sync();
    const u64 open = listed_by_all(sh, team);
    if (open <= (u64)kList) break;
    team.sync();                     // counted by all before the next round clears
  }
  // the first block ranks the open tokens and finds the cut
  const int len = (int)listed_by_all(sh, team);
  join_lists(sh, team);
  if (team.rank == 0) {
    if (len <= kCountRank) {
      const int p = threadIdx.x >> 2, part = threadIdx.x & 3;
      u64 key = 0;
      uint32_t w = 0;
      if (p < len) {
        key = sh.list[p];
        w = Row::weight(Row::e(r.depth(rank_logit(key))));
        if (part == 0) sh.weight[p] = w;
      }
      __syncthreads();
      u64 ahead = 0;
      for (int j = part; j < len; j += 4)
        if (sh.list[j] > key) ahead += ((u64)sh.weight[j] << 8) | 1u;
      ahead += __shfl_xor_sync(0xFFFFFFFFu, ahead, 1);
      ahead += __shfl_xor_sync(0xFFFFFFFFu, ahead, 2);
      const u64 mass = before_mass + (ahead >> 8);
      const u64 lo = COUNT ? before_count + (ahead & 255u) : mass;
      const u64 hi = lo + (COUNT ? 1ull : (u64)w);
      if (p < len && part == 0 && lo < target && target <= hi) {
        sh.cut = key;
        sh.sum = mass + w;
      }
    } else {
      const int size = pow2_at_least(len);
      for (int i = len + threadIdx.x; i < size; i += kThreads) sh.list[i] = 0ull;
      sort_list(sh, size);
      constexpr int kPer = kList / kThreads;
      const int per = (size + kThreads - 1) / kThreads;
      uint32_t w[kPer];
      u64 mine = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int p = threadIdx.x * per + i;
        w[i] = (i < per && p < len) ? Row::weight(Row::e(r.depth(rank_logit(sh.list[p])))) : 0u;
        mine += w[i];
      }
      u64 total;
      u64 mass = before_mass + block_scan(mine, sh, &total);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int p = threadIdx.x * per + i;
        if (i < per && p < len) {
          const u64 lo = COUNT ? before_count + (u64)p : mass;
          const u64 hi = lo + (COUNT ? 1ull : (u64)w[i]);
          if (lo < target && target <= hi) {
            sh.cut = sh.list[p];
            sh.sum = mass + w[i];
          }
        }
        mass += w[i];
      }
    }
  }
  team.sync();
  const u64 cut = *team.of(&sh.cut, 0);
  *mass_out = *team.of(&sh.sum, 0);
  team.sync();
  return cut;
}

// The draw over the whole row, by index, among tokens with e >= min_p and
// (CUT) a rank key of at least `cut`.
template <bool CUT, typename T>
__device__ __noinline__ void draw_in_row(const SampleArgs& a, int row, const Pieces<T>& pc, int q0, int q1,
                            Shared& sh, const Team& team, const Row& r, u64 cut, float u) {
  constexpr int V = Pieces<T>::V;
  constexpr int kBatch = 32 * kShares;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float lowest = rank_logit(cut);
  auto kept = [&](float l, int idx) -> uint32_t {
    const float e = Row::e(r.depth(l));
    const uint32_t w = Row::weight(e);
    if constexpr (CUT) {
      if (l == lowest && rank_key(l, (uint32_t)idx) < cut) return 0u;
    }
    return e >= r.min_p ? w : 0u;
  };
  const int per = ((q1 - q0 + kBatch - 1) / kBatch + kSegs - 1) / kSegs;   // batches a stretch
  u64 warp_total = 0;
  int seg = 0;
  for (int b0 = q0; b0 < q1; b0 += per * kBatch, ++seg) {
    const int b1 = min(q1, b0 + per * kBatch);
    u64 mine = 0;
    pc.each(b0, b1, [&](const float (&v)[V], int i0) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (!CUT || v[j] >= lowest) mine += kept(v[j], i0 + j);
    });
    mine = warp_sum(mine);
    if (lane == 0) sh.seg[warp][seg] = mine;
    warp_total += mine;
  }
  __syncthreads();
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
  if (before <= target && target < before + warp_total) {
    // this warp's part holds the draw: find the stretch, then walk it
    seg = 0;
    while (target >= before + sh.seg[warp][seg]) before += sh.seg[warp][seg++];
    const int e0 = q0 + seg * per * kBatch, e1 = min(q1, e0 + per * kBatch);
    bool found = false;
    for (int b = e0; b < e1 && !found; b += kBatch) {
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
        Pieces<T>::values(piece, v);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          w[j] = q < e1 && (!CUT || v[j] >= lowest) ? kept(v[j], q * V - pc.mis + j) : 0u;
          mine += w[j];
        }
        const u64 inc = warp_scan(mine);
        const u64 step = __shfl_sync(0xFFFFFFFFu, inc, 31);
        if (!found && target < before + step) {
          u64 at = before + inc - mine;
#pragma unroll
          for (int j = 0; j < V; ++j) {
            if (at <= target && target < at + w[j])
              write_draw(a, row, q * V - pc.mis + j, w[j], sum);
            at += w[j];
          }
          found = true;
        }
        before += step;
      }
    }
  }
}

// A row whose maximum is +inf: the infinite logits share the draw, a weight
// of 2^31 each, ranked by index.
template <typename T>
__device__ __noinline__ void draw_infinite(const SampleArgs& a, int row, const Pieces<T>& pc,
                                           int q0, int q1, Shared& sh, const Team& team, int top_k,
                                           float top_p, float u) {
  constexpr int V = Pieces<T>::V;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float inf = __int_as_float(0x7F800000);
  u64 mine = 0;
  pc.each(q0, q1, [&](const float (&v)[V], int) {
#pragma unroll
    for (int j = 0; j < V; ++j) mine += v[j] == inf;
  });
  const u64 warp_total = warp_sum(mine);
  u64 total;
  u64 before = block_scan(lane == 0 ? warp_total : 0ull, sh, &total);   // of lane 0
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
    if (q < q1) Pieces<T>::values(pc.load(q), v);
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

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  constexpr int V = Pieces<T>::V;
  const Team team;
  const int row = blockIdx.x / team.size;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < kBins * 32; i += kThreads) {
    (&sh.low[0][0])[i] = 0u;
    (&sh.high[0][0])[i] = 0u;
    (&sh.count[0][0])[i] = 0u;
  }
  griddep_launch_dependents();
  griddep_wait();
  const Pieces<T> pc(reinterpret_cast<const T*>(a.logits) + (size_t)row * a.n, a.n);
  // this warp's pieces
  const int part = team.rank * kWarps + warp, parts = team.size * kWarps;
  const int q0 = (int)((long long)pc.pieces * part / parts);
  const int q1 = (int)((long long)pc.pieces * (part + 1) / parts);

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

  // the maximum
  float share[kShares];
#pragma unroll
  for (int s = 0; s < kShares; ++s) share[s] = __int_as_float(0xFF800000);
#pragma unroll 1
  for (int b = q0; b < q1; b += 32 * kShares) {
    uint4 raw[kShares];
    pc.batch(b, q1, raw);
#pragma unroll
    for (int s = 0; s < kShares; ++s) {
      float v[V];
      Pieces<T>::values(raw[s], v);
      float m = v[0];
#pragma unroll
      for (int j = 1; j < V; ++j) m = fmaxf(m, v[j]);
      if (b + s * 32 + lane < q1) share[s] = fmaxf(share[s], m);
    }
  }
  float mx = fmaxf(fmaxf(share[0], share[1]), fmaxf(share[2], share[3]));
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, m));
  if (lane == 0) sh.redf[warp] = mx;
  __syncthreads();
  mx = sh.redf[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, sh.redf[w]);
  if (threadIdx.x == 0) {
    sh.max = mx;
    sh.listed = 0u;
    sh.digit = -1;
    sh.cut = 0ull;
    sh.sum = 0ull;
  }
  team.sync();
  team.over(&sh.max, [&](float m, int) { mx = fmaxf(mx, m); });
  r.top = mx;

  if (mx == __int_as_float(0xFF800000)) {              // nothing left
    if (team.rank == 0 && threadIdx.x == 0) {
      a.ids[row] = -1;
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
    draw_infinite(a, row, pc, q0, q1, sh, team, top_k, top_p, u);
    team.sync();
    return;
  }

  if (top_k > 0 && top_k <= kMaxListK) {
    // the bound: enough share maxima reach it
#pragma unroll
    for (int s = 0; s < kShares; ++s) {
      const float x = r.depth(share[s]);
      if (x > -31.f) atomicAdd(&sh.count[Row::bin(x)][lane], 1u);
    }
    __syncthreads();
    for (int d = warp; d < kBins; d += kWarps) {
      const uint32_t c = __reduce_add_sync(0xFFFFFFFFu, sh.count[d][lane]);
      sh.count[d][lane] = 0u;
      if (lane == 0) sh.bin_count[d] = c;
    }
    team.sync();
    u64 cnt = 0;
    if (threadIdx.x < kBins)
      team.over(&sh.bin_count[threadIdx.x], [&](uint32_t c, int) { cnt += c; });
    u64 total;
    const u64 below = block_scan(cnt, sh, &total);
    if (below < (u64)top_k && (u64)top_k <= below + cnt) sh.digit = (int)threadIdx.x;
    __syncthreads();
    const bool all = sh.digit < 0;
    // (a little below the edge, against the rounding here)
    const float bound = all ? __int_as_float(0xFF800000)
                            : r.top - ((float)sh.digit + 0.5f + 1e-3f) / (4.f * r.c);
    pc.each(q0, q1, [&](const float (&v)[V], int i0) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (v[j] >= bound && Row::weight(Row::e(r.depth(v[j]))) != 0u)
          append(sh, rank_key(v[j], (uint32_t)(i0 + j)));
    });
    team.sync();
    const u64 listed = listed_by_all(sh, team);
    if (listed <= (u64)kList && (all || listed >= (u64)top_k)) {
      join_lists(sh, team);
      if (team.rank == 0) {
        if (listed <= (u64)kCountRank)
          finish_by_counting(a, row, sh, r, (int)listed, top_k, top_p, u);
        else
          finish_by_sorting(a, row, sh, r, (int)listed, top_k, top_p, u);
      }
      team.sync();
      return;
    }
    team.sync();                                       // counted by all before it is cleared
  }

  u64 cut = 0, sum = 0;
  if (top_k > 0) cut = find_cut<true>(pc, q0, q1, sh, team, r, top_k, 1.f, 0ull, &sum);
  if (top_p < 1.f) cut = find_cut<false>(pc, q0, q1, sh, team, r, 0, top_p, cut, &sum);
  if (cut != 0ull)
    draw_in_row<true>(a, row, pc, q0, q1, sh, team, r, cut, u);
  else
    draw_in_row<false>(a, row, pc, q0, q1, sh, team, r, cut, u);
  team.sync();
}

// Blocks per row: as many as still give every row its own share of the SMs
// (two blocks fit one), with at least 4096 logits each.
int cluster_size(int m, int n) {
  int c = 1;
  while (c < kMaxCluster && 2ll * c * m <= 2ll * device_sm_count() && n / (2 * c) >= 4096) c *= 2;
  return c;
}

template <typename T>
cudaError_t launch_t(const SampleArgs& a, cudaStream_t s) {
  const int c = cluster_size(a.m, a.n);
  auto kern = sample_kernel<T>;
  static bool configured = false;
  if (!configured) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)sizeof(Shared));
    if (e != cudaSuccess) return e;
    configured = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.m * c);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Shared);
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
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a);
  note_launch();
  return e;
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
