// sample.cu -- draw the next token of every row: temperature, top-k, top-p
// and min-p, from a given random number.
//
// Weights are integers, W = floor(2^31 * exp2((l - max) * log2e / t)), so
// every sum is exact and the same in any order; ranks go by logit descending,
// then index ascending.  Each filter keeps a prefix of that order, so a row's
// filters come down to one cut, the 64-bit rank key of the last kept token:
// (order-preserving bits of the logit, inverted index).
//
// One cluster of 1 to 8 blocks per row, each over a contiguous slice:
//  1. maximum (and the maxima of four shares of each thread's elements);
//  2. a bound that about K logits reach, from a histogram of those maxima: K
//     values at least as large exist if K maxima do;
//  3. one pass that gathers the logits above the bound into a list (and sums
//     all weights when a nucleus needs them);
//  4. the first block sorts the list and applies the filters by a prefix sum,
//     then sorts the kept tokens by index and draws.
// Rows whose cut lies outside the list (large top-k, a wide nucleus) find it
// by a descent over histograms of counts and weights: 256 steps of an eighth
// of an octave below the maximum, then the bytes of the rank key, until the
// undecided tokens fit the list.  The draw then runs over the whole row by
// index, as it does when temperature or min-p alone is on.
#include <cooperative_groups.h>

#include "mx.cuh"

namespace cg = cooperative_groups;

namespace wql {
namespace {

typedef unsigned long long u64;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kList = 2048;          // tokens the list holds
constexpr int kBins = 256;
constexpr int kShares = 4;           // maxima kept per thread; loads in flight per thread
constexpr int kMaxCluster = 8;
constexpr int kNucleusBound = 768;   // tokens the bound aims at for a nucleus
constexpr float kLog2e = 1.44269504088896340736f;

struct Shared {
  u64 list[kList];
  uint32_t weight[kList];
  u64 mass[kBins];
  uint32_t count[kBins];
  u64 red[kWarps];
  float redf[kWarps];
  // read by the other blocks of the cluster
  float max;
  u64 sum;
  uint32_t listed;
  u64 cut;                           // of the first block
  int done;
  // block-wide results
  int digit;
  u64 digit_count, before_count, before_mass;
};

__device__ __forceinline__ uint32_t logit_key(float l) {
  const uint32_t b = __float_as_uint(l + 0.f);        // -0 ranks as +0
  return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ __forceinline__ u64 rank_key(float l, uint32_t idx) {
  return ((u64)logit_key(l) << 32) | (uint32_t)~idx;
}

// What a row is drawn with.
struct Row {
  float top;       // largest logit
  float c;         // log2e / temperature
  float min_p;     // 0: off
  __device__ __forceinline__ float e(float l) const {
    return l == top ? 1.f : exp2f(__fmul_rn(__fsub_rn(l, top), c));
  }
  // (a NaN converts to 0)
  static __device__ __forceinline__ uint32_t weight(float e) {
    return __float2uint_rz(e * 2147483648.f);
  }
  // eighths of an octave below the maximum; 255 and below it, negligible
  __device__ __forceinline__ int bin(float l) const {
    const float f = l == top ? 0.f : __fmul_rn(__fmul_rn(__fsub_rn(top, l), c), 8.f);
    return f < 255.f ? (int)f : 255;                  // NaN: 255
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
    const int i0 = q * V - mis;
    if (i0 >= 0 && i0 + V <= n) return __ldg(reinterpret_cast<const uint4*>(base) + q);
    uint4 r;
    T* h = reinterpret_cast<T*>(&r);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int i = i0 + j;
      if (i >= 0 && i < n)
        h[j] = base[(size_t)q * V + j];
      else if constexpr (sizeof(T) == 4)
        h[j] = __int_as_float(0xFF800000);
      else
        h[j] = from_f32<T>(__int_as_float(0xFF800000));
    }
    return r;
  }
  static __device__ __forceinline__ void values(const uint4& r, float (&v)[V]) {
    const T* h = reinterpret_cast<const T*>(&r);
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = to_f32(h[j]);
  }
  // f(values, index of the first, share) for this warp's pieces q0 .. q1
  template <typename F> __device__ __forceinline__ void each(int q0, int q1, F f) const {
    const int lane = threadIdx.x & 31;
    for (int b = q0; b < q1; b += 32 * kShares) {
      uint4 r[kShares];
#pragma unroll
      for (int u = 0; u < kShares; ++u) {
        const int q = b + u * 32 + lane;
        if (q < q1) r[u] = load(q);
      }
#pragma unroll
      for (int u = 0; u < kShares; ++u) {
        const int q = b + u * 32 + lane;
        if (q < q1) {
          float v[V];
          values(r[u], v);
          f(v, q * V - mis, u);
        }
      }
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
};

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
  return v;
}

// Exclusive prefix sum over the block; *total gets the sum.
__device__ u64 block_scan(u64 v, Shared& sh, u64* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  u64 inc = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const u64 o = __shfl_up_sync(0xFFFFFFFFu, inc, d);
    if (lane >= d) inc += o;
  }
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

// The lists of all blocks of the cluster, joined in the first block's list;
// returns the length there, or -1 when they do not fit.  Call on all blocks
// after a sync that follows the gathering; only the first block's result and
// list are meaningful.
__device__ int join_lists(Shared& sh, const Team& team) {
  int total = 0;
  if (team.rank != 0) return 0;
  for (int r = 0; r < team.size; ++r) {
    const uint32_t c = *team.of(&sh.listed, r);
    if (c > (uint32_t)kList || total + (int)c > kList) return -1;
    if (r > 0) {
      const u64* src = team.of(&sh.list[0], r);
      for (int i = threadIdx.x; i < (int)c; i += kThreads) sh.list[total + i] = src[i];
    }
    total += (int)c;
  }
  __syncthreads();
  return total;
}

__device__ __forceinline__ void append(Shared& sh, u64 key) {
  const uint32_t at = atomicAdd(&sh.listed, 1u);
  if (at < (uint32_t)kList) sh.list[at] = key;
}

// Sum of `v` over the cluster.  Ends with a sync.
__device__ u64 team_sum(u64 v, Shared& sh, const Team& team) {
  u64 total;
  block_scan(v, sh, &total);
  if (threadIdx.x == 0) sh.sum = total;
  team.sync();
  u64 s = 0;
  for (int r = 0; r < team.size; ++r) s += *team.of(&sh.sum, r);
  team.sync();
  return s;
}

// The integer that a nucleus' weights have to reach: those before a kept
// token sum to less than p * sum, so to less than its ceiling.
__device__ __forceinline__ u64 nucleus_target(float p, u64 sum) {
  const double t = ceil((double)p * (double)sum);
  return t < 1.0 ? 1ull : (u64)t;
}

__device__ __forceinline__ u64 draw_target(float u, u64 sum) {
  const double r = (double)u * (double)sum;
  u64 v = r > 0.0 ? (u64)r : 0ull;
  return v < sum ? v : sum - 1;
}

__device__ __forceinline__ void write_draw(const SampleArgs& a, int row, int id, uint32_t w,
                                           u64 sum) {
  a.ids[row] = id;
  if (a.logp) a.logp[row] = logf(__fdiv_rn((float)w, (float)sum));
}

// Filters and draw within the list of the first block (`len` tokens, all that
// reach some bound; `all`: no other token has a weight).  False when the cut
// may lie outside it.
__device__ bool finish_in_list(const SampleArgs& a, int row, Shared& sh, const Row& r, int len,
                               bool all, int top_k, float top_p, float u, u64 sum) {
  if (len <= 0) return false;
  if (top_k > len && !all) return false;
  const int size = pow2_at_least(len);
  for (int i = len + threadIdx.x; i < size; i += kThreads) sh.list[i] = 0ull;
  sort_list(sh, size);
  constexpr int kPer = kList / kThreads;
  const int per = (size + kThreads - 1) / kThreads;    // 1..kPer consecutive entries a thread
  float e[kPer];
  uint32_t w[kPer];
  u64 mine = 0;
  const int limit = top_k > 0 ? min(top_k, len) : len;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int p = threadIdx.x * per + i;
    w[i] = 0u;
    e[i] = 0.f;
    if (i < per && p < limit) {
      e[i] = r.e(key_logit((uint32_t)(sh.list[p] >> 32)));
      w[i] = Row::weight(e[i]);
      mine += w[i];
    }
  }
  u64 total;
  u64 before = block_scan(mine, sh, &total);
  const u64 reach = top_p < 1.f ? nucleus_target(top_p, top_k > 0 ? total : sum) : ~0ull;
  if (top_k <= 0 && total < reach && total != sum) return false;
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
    by_index[i] = p < keep ? ((sh.list[p] & 0xFFFFFFFFull) << 32) | (u64)p : 0ull;
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
  before = block_scan(mine, sh, &total);
  const u64 target = draw_target(u, kept_sum);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (before <= target && target < before + w[i])
      write_draw(a, row, (int)~(uint32_t)(sh.list[threadIdx.x * per2 + i] >> 32), w[i], kept_sum);
    before += w[i];
  }
  return true;
}

// The rank key of the last token of the shortest prefix, in rank order among
// the tokens with a weight and a rank key of at least `from`, whose count (or
// sum of weights) reaches `target`; 0 when there is none.  *mass_out (when
// wanted) gets the prefix's sum of weights.
template <typename T>
__device__ u64 find_cut(const Pieces<T>& pc, int q0, int q1, Shared& sh, const Team& team,
                        const Row& r, bool by_count, u64 target, u64 from, u64* mass_out) {
  constexpr int V = Pieces<T>::V;
  u64 before_count = 0, before_mass = 0;
  int bin = -1;                      // chosen eighth of an octave
  u64 prefix = 0;                    // chosen leading bytes of the rank key
  int shift = 64;                    // bits of the rank key still open
  for (;;) {
    const bool first = bin < 0;
    const int dshift = first ? 0 : shift - 8;
    for (int i = threadIdx.x; i < kBins; i += kThreads) {
      sh.count[i] = 0u;
      sh.mass[i] = 0ull;
    }
    if (threadIdx.x == 0) sh.digit = -1;
    __syncthreads();
    pc.each(q0, q1, [&](const float (&v)[V], int i0, int) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const uint32_t w = Row::weight(r.e(v[j]));
        if (w == 0u) continue;
        const u64 key = rank_key(v[j], (uint32_t)(i0 + j));
        if (key < from) continue;
        const int b = r.bin(v[j]);
        int d = b;
        if (!first) {
          if (b != bin || (shift < 64 && (key >> shift) != prefix)) continue;
          d = 255 - (int)((key >> dshift) & 255u);
        }
        atomicAdd(&sh.count[d], 1u);
        atomicAdd(&sh.mass[d], (u64)w);
      }
    });
    team.sync();
    // every block joins the histograms and comes to the same choice
    u64 cnt = 0, mass = 0;
    if (threadIdx.x < kBins)
      for (int k = 0; k < team.size; ++k) {
        cnt += *team.of(&sh.count[threadIdx.x], k);
        mass += *team.of(&sh.mass[threadIdx.x], k);
      }
    u64 total_count, total_mass;
    const u64 pc_count = before_count + block_scan(cnt, sh, &total_count);
    const u64 pc_mass = before_mass + block_scan(mass, sh, &total_mass);
    const u64 lo = by_count ? pc_count : pc_mass, hi = lo + (by_count ? cnt : mass);
    if (lo < target && target <= hi) {
      sh.digit = (int)threadIdx.x;
      sh.digit_count = cnt;
      sh.before_count = pc_count;
      sh.before_mass = pc_mass;
    }
    team.sync();
    if (sh.digit < 0) {
      if (mass_out) *mass_out = before_mass + total_mass;
      return 0ull;
    }
    before_count = sh.before_count;
    before_mass = sh.before_mass;
    const u64 open = sh.digit_count;
    if (first) {
      bin = sh.digit;
    } else {
      prefix = (prefix << 8) | (u64)(255 - sh.digit);
      shift = dshift;
    }
    __syncthreads();                 // the choice is read before the next round clears it
    if (open <= (u64)kList) break;
  }
  // the open tokens fit the list: the first block sorts them and finds the cut
  if (threadIdx.x == 0) sh.listed = 0u;
  __syncthreads();
  pc.each(q0, q1, [&](const float (&v)[V], int i0, int) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (Row::weight(r.e(v[j])) == 0u || r.bin(v[j]) != bin) continue;
      const u64 key = rank_key(v[j], (uint32_t)(i0 + j));
      if (key < from || (shift < 64 && (key >> shift) != prefix)) continue;
      append(sh, key);
    }
  });
  team.sync();
  const int len = join_lists(sh, team);
  if (team.rank == 0) {
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
      w[i] = (i < per && p < len) ? Row::weight(r.e(key_logit((uint32_t)(sh.list[p] >> 32)))) : 0u;
      mine += w[i];
    }
    u64 total;
    u64 mass = before_mass + block_scan(mine, sh, &total);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int p = threadIdx.x * per + i;
      if (i < per && p < len) {
        const u64 lo = by_count ? before_count + (u64)p : mass;
        const u64 hi = lo + (by_count ? 1ull : (u64)w[i]);
        if (lo < target && target <= hi) {
          sh.cut = sh.list[p];
          sh.sum = mass + w[i];
        }
      }
      mass += w[i];
    }
  }
  team.sync();
  const u64 cut = *team.of(&sh.cut, 0);
  if (mass_out) *mass_out = *team.of(&sh.sum, 0);
  team.sync();
  return cut;
}

// The draw over the whole row, by index, among tokens with a rank key of at
// least `cut` and e >= min_p.
template <typename T>
__device__ void draw_in_row(const SampleArgs& a, int row, const Pieces<T>& pc, int q0, int q1,
                            Shared& sh, const Team& team, const Row& r, u64 cut, float u) {
  constexpr int V = Pieces<T>::V;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto kept = [&](float l, int idx) -> uint32_t {
    const float e = r.e(l);
    if (!(e >= r.min_p) || (cut != 0ull && rank_key(l, (uint32_t)idx) < cut)) return 0u;
    return Row::weight(e);
  };
  u64 mine = 0;
  pc.each(q0, q1, [&](const float (&v)[V], int i0, int) {
#pragma unroll
    for (int j = 0; j < V; ++j) mine += kept(v[j], i0 + j);
  });
  const u64 warp_total = warp_sum(mine);
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
  for (int k = 0; k < team.size; ++k) {
    const u64 t = *team.of(&sh.sum, k);
    if (k < team.rank) before += t;
    sum += t;
  }
  const u64 target = draw_target(u, sum);
  if (before <= target && target < before + warp_total) {
    // this warp's stretch holds the draw: walk it, 32 pieces at a time
    for (int b = q0; b < q1; b += 32) {
      const int q = b + lane;
      uint32_t w[V];
      u64 s = 0;
#pragma unroll
      for (int j = 0; j < V; ++j) w[j] = 0u;
      if (q < q1) {
        float v[V];
        Pieces<T>::values(pc.load(q), v);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          w[j] = kept(v[j], q * V - pc.mis + j);
          s += w[j];
        }
      }
      u64 inc = s;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const u64 o = __shfl_up_sync(0xFFFFFFFFu, inc, d);
        if (lane >= d) inc += o;
      }
      const u64 step = __shfl_sync(0xFFFFFFFFu, inc, 31);
      if (target < before + step) {
        u64 at = before + inc - s;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          if (at <= target && target < at + w[j])
            write_draw(a, row, q * V - pc.mis + j, w[j], sum);
          at += w[j];
        }
        break;
      }
      before += step;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs a) {
  __shared__ Shared sh;
  constexpr int V = Pieces<T>::V;
  griddep_launch_dependents();
  griddep_wait();
  const Team team;
  const int row = blockIdx.x / team.size;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
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
  r.c = __fdiv_rn(kLog2e, t);

  // 1. maxima
  float share[kShares];
#pragma unroll
  for (int s = 0; s < kShares; ++s) share[s] = __int_as_float(0xFF800000);
  pc.each(q0, q1, [&](const float (&v)[V], int, int s) {
#pragma unroll
    for (int j = 0; j < V; ++j) share[s] = fmaxf(share[s], v[j]);
  });
  float mx = fmaxf(fmaxf(share[0], share[1]), fmaxf(share[2], share[3]));
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, m));
  if (lane == 0) sh.redf[warp] = mx;
  for (int i = threadIdx.x; i < kBins; i += kThreads) sh.count[i] = 0u;
  __syncthreads();
  mx = sh.redf[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, sh.redf[w]);
  if (threadIdx.x == 0) {
    sh.max = mx;
    sh.listed = 0u;
    sh.done = 0;
    sh.cut = 0ull;
  }
  team.sync();
  for (int k = 0; k < team.size; ++k) mx = fmaxf(mx, *team.of(&sh.max, k));
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
    pc.each(q0, q1, [&](const float (&v)[V], int i0, int) {
#pragma unroll
      for (int j = V - 1; j >= 0; --j)
        if (v[j] == mx) at = min(at, i0 + j);
    });
    at = __reduce_min_sync(0xFFFFFFFFu, at);
    __syncthreads();
    if (lane == 0) sh.red[warp] = (u64)(uint32_t)at;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) at = min(at, (int)sh.red[w]);
    if (threadIdx.x == 0) sh.sum = (u64)(uint32_t)at;
    team.sync();
    if (team.rank == 0 && threadIdx.x == 0) {
      for (int k = 0; k < team.size; ++k) at = min(at, (int)*team.of(&sh.sum, k));
      a.ids[row] = at;
      if (a.logp) a.logp[row] = 0.f;
    }
    team.sync();
    return;
  }

  u64 cut = 0;
  if (top_k > 0 || top_p < 1.f) {
    u64 sum = 0;                                       // of all weights, for a nucleus
    const bool need_sum = top_k <= 0;
    bool listed = false;
    if (top_k <= kNucleusBound) {
      // 2. the bound
#pragma unroll
      for (int s = 0; s < kShares; ++s) {
        const int b = r.bin(share[s]);
        if (b < 255) atomicAdd(&sh.count[b], 1u);
      }
      if (threadIdx.x == 0) sh.digit = -1;
      team.sync();
      u64 cnt = 0;
      if (threadIdx.x < kBins)
        for (int k = 0; k < team.size; ++k) cnt += *team.of(&sh.count[threadIdx.x], k);
      u64 total;
      const u64 below = block_scan(cnt, sh, &total);
      const u64 want = top_k > 0 ? (u64)top_k : (u64)kNucleusBound;
      if (below < want && want <= below + cnt) sh.digit = (int)threadIdx.x;
      __syncthreads();
      const float bound = sh.digit < 0 ? __int_as_float(0xFF800000)
                                       : r.top - (float)(sh.digit + 1) / (8.f * r.c);
      // 3. the list
      u64 mine = 0;
      pc.each(q0, q1, [&](const float (&v)[V], int i0, int) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          if (need_sum) mine += Row::weight(r.e(v[j]));
          if (v[j] >= bound && Row::weight(r.e(v[j])) != 0u)
            append(sh, rank_key(v[j], (uint32_t)(i0 + j)));
        }
      });
      if (need_sum)
        sum = team_sum(mine, sh, team);
      else
        team.sync();
      // 4. filters and draw
      const int len = join_lists(sh, team);
      if (team.rank == 0) {
        const bool ok = finish_in_list(a, row, sh, r, len, bound == __int_as_float(0xFF800000),
                                       top_k, top_p, u, sum);
        if (threadIdx.x == 0) sh.done = ok ? 1 : 0;
      }
      team.sync();
      listed = *team.of(&sh.done, 0) != 0;
      team.sync();
    }
    if (listed) return;
    if (top_k > 0) {
      cut = find_cut(pc, q0, q1, sh, team, r, true, (u64)top_k, 0ull, &sum);
    }
    if (top_p < 1.f) {
      const u64 c2 = find_cut(pc, q0, q1, sh, team, r, false, nucleus_target(top_p, sum), cut,
                              nullptr);
      if (c2 != 0ull) cut = c2;
    }
  }
  draw_in_row(a, row, pc, q0, q1, sh, team, r, cut, u);
  team.sync();
}

// Blocks per row: as many as still give every row its own share of the SMs
// (two blocks fit one), with at least 4096 logits each.
int cluster_size(int m, int n) {
  int c = 1;
  while (c < kMaxCluster && 2 * c * m <= 2 * device_sm_count() && n / (2 * c) >= 4096) c *= 2;
  return c;
}

template <typename T>
cudaError_t launch_t(const SampleArgs& a, cudaStream_t s) {
  const int c = cluster_size(a.m, a.n);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.m * c);
  cfg.blockDim = dim3(kThreads);
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
  const cudaError_t e = cudaLaunchKernelEx(&cfg, sample_kernel<T>, a);
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
