// beam_select.cu -- one step of beam search: the best `beams` continuations of
// a sequence's beams * n by s[w, v] = scores[w] + l[w, v] - log sum exp l[w, :].
//
// Two launches.  beam_part_kernel reads the logits once, a block per part of a
// row that stays in registers: the part's maximum, its sum of exponentials and
// its best `beams` continuations.  beam_join_kernel, a block per sequence, joins
// the sums, takes the best of each row's lists, and the best of those.
//
// Inside a row the order of the scores is that of the logits, so lists hold
// (logit, token) keys and no score; scores exist in binary64 for beams * beams
// keys only.  Every order is total (ties by token, then by beam), hence results
// do not depend on the order in which lists were filled.
#include "requests.cuh"

namespace wql {
namespace {

using u64 = unsigned long long;
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kGroups = kThreads / 8;    // of 8 lanes, whose maxima give a part's threshold
constexpr int kList = 256;               // continuations that pass it
constexpr int kSmall = 8 * kThreads;     // elements of a part, few rows
constexpr int kLarge = 32 * kThreads;    // many rows
constexpr int kLanes = 6;                // lists a lane looks after when a row is joined
static_assert(kGroups >= WQL_MAX_BEAMS, "a group for each of the best");
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kMinusInf = -__builtin_huge_valf();

// Floats in the order of their bits (no NaN), and back.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t o) {
  return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
// Larger logit first, then the lower token (-0 is 0); 0 is below every key.
__device__ __forceinline__ u64 make_key(float v, uint32_t token) {
  return (u64)ordered(v + 0.f) << 32 | (0xFFFFFFFFu - token);
}
__device__ __forceinline__ uint32_t key_token(u64 k) { return 0xFFFFFFFFu - (uint32_t)k; }
__device__ __forceinline__ float key_logit(u64 k) { return from_ordered((uint32_t)(k >> 32)); }

__device__ __forceinline__ u64 warp_max(u64 k) {
  const uint32_t hi = __reduce_max_sync(0xFFFFFFFFu, (uint32_t)(k >> 32));
  const uint32_t lo = __reduce_max_sync(0xFFFFFFFFu, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
  return (u64)hi << 32 | lo;
}

__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// The 16 bytes of a group of elements as they are held: NaN and what lies
// outside the row as -inf.
template <typename T> struct Group;
template <> struct Group<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ uint4 clean(uint4 v) {
    uint32_t* p = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      p[i] = __float_as_uint(fmaxf(__uint_as_float(p[i]), kMinusInf));
    return v;
  }
  static __device__ __forceinline__ float at(const uint4& v, int i) {
    return __uint_as_float(reinterpret_cast<const uint32_t*>(&v)[i]);
  }
  static __device__ __forceinline__ float max(const uint4& v) {
    return fmaxf(fmaxf(at(v, 0), at(v, 1)), fmaxf(at(v, 2), at(v, 3)));
  }
  static __device__ __forceinline__ void erase(uint4& v, int i) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j == i) reinterpret_cast<uint32_t*>(&v)[j] = 0xFF800000u;
  }
};
template <typename T, typename T2, uint32_t MINUS_INF> struct Group16 {
  static constexpr int kN = 8;
  static __device__ __forceinline__ T2 pair(uint32_t v) { return *reinterpret_cast<T2*>(&v); }
  static __device__ __forceinline__ uint4 clean(uint4 v) {
    uint32_t* p = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const T2 m = __hmax2(pair(p[i]), pair(MINUS_INF));
      p[i] = *reinterpret_cast<const uint32_t*>(&m);
    }
    return v;
  }
  static __device__ __forceinline__ float at(const uint4& v, int i) {
    const uint32_t w = reinterpret_cast<const uint32_t*>(&v)[i >> 1];
    const uint16_t h = (uint16_t)(w >> (16 * (i & 1)));
    return to_f32(*reinterpret_cast<const T*>(&h));
  }
  static __device__ __forceinline__ float max(const uint4& v) {
    const T2 m = __hmax2(__hmax2(pair(v.x), pair(v.y)), __hmax2(pair(v.z), pair(v.w)));
    return fmaxf(to_f32(m.x), to_f32(m.y));
  }
  static __device__ __forceinline__ void erase(uint4& v, int i) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j == i) {
        uint32_t& w = reinterpret_cast<uint32_t*>(&v)[j >> 1];
        w = j & 1 ? (w & 0x0000FFFFu) | (MINUS_INF & 0xFFFF0000u)
                  : (w & 0xFFFF0000u) | (MINUS_INF & 0x0000FFFFu);
      }
  }
};
template <> struct Group<__half> : Group16<__half, __half2, 0xFC00FC00u> {};
template <> struct Group<__nv_bfloat16> : Group16<__nv_bfloat16, __nv_bfloat162, 0xFF80FF80u> {};

// Elements [e, e + kN) of a row of n that starts at `row`; `row + e` lies on a
// 16-byte address, e may be negative.  -inf outside the row.
template <typename T>
__device__ __forceinline__ uint4 load_group(const T* row, int e, int n) {
  constexpr int kN = Group<T>::kN;
  if (e >= 0 && e + kN <= n) return __ldg(reinterpret_cast<const uint4*>(row + e));
  alignas(16) T tmp[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i)
    tmp[i] = e + i >= 0 && e + i < n ? row[e + i] : from_f32<T>(kMinusInf);
  return *reinterpret_cast<const uint4*>(tmp);
}

// The 16 bytes that start `mis` elements into a, b.
template <typename T> __device__ __forceinline__ uint4 shifted(uint4 a, uint4 b, int mis) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  const int words = sizeof(T) == 4 ? mis : mis >> 1;
#pragma unroll
  for (int i = 0; i < 6; ++i) w[i] = words & 2 ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) w[i] = words & 1 ? w[i + 1] : w[i];
  if (sizeof(T) == 2 && (mis & 1)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// ---------------------------------------------------------------------------
// One part of a row: VECS groups of 16 bytes a thread, group j * 256 + thread
// of the part.  Which tokens a thread has does not depend on where the row
// starts, so that equal rows give equal sums and their ties go to the lower
// beam; a row off a 16-byte boundary is read in aligned groups, two of which
// make one (ALIGNED: no row is).
// stats[row][part] = (maximum, sum of exp(l - maximum)), (-inf, 0) without any;
// keys[row][part][0 .. beams) = the best continuations but eos, 0 past them.
// ---------------------------------------------------------------------------
template <typename T, int VECS, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) beam_part_kernel(const BeamSelectArgs a) {
  using G = Group<T>;
  constexpr int kN = G::kN;
  __shared__ float group_max[kGroups];
  __shared__ float eos_logit;
  __shared__ float warp_sum[kWarps];
  __shared__ u64 list[kList];
  __shared__ int listed;
  __shared__ u64 best_of[2][kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_launch_dependents();
  griddep_wait();
  const int row = blockIdx.x / a.parts, part = blockIdx.x % a.parts;
  const T* logits = static_cast<const T*>(a.logits) + (size_t)row * a.n;
  const int first = (part * (VECS * kThreads) + tid) * kN;   // this thread's first token
  const int eos = a.eos;

  uint4 v[VECS];
  if constexpr (ALIGNED) {
#pragma unroll
    for (int j = 0; j < VECS; ++j) v[j] = load_group(logits, first + j * kThreads * kN, a.n);
  } else {
    const int mis = (int)(reinterpret_cast<uintptr_t>(logits) / sizeof(T)) & (kN - 1);
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
      const int e = first + j * kThreads * kN - mis;
      const uint4 lo = load_group(logits, e, a.n);
      v[j] = mis ? shifted<T>(lo, load_group(logits, e + kN, a.n), mis) : lo;
    }
  }
  if (tid == 0) {
    listed = 0;
    eos_logit = kMinusInf;
  }
  float top = kMinusInf;
#pragma unroll
  for (int j = 0; j < VECS; ++j) v[j] = G::clean(v[j]);
  __syncthreads();
  // the end token counts in the sum, not among the continuations
  float end = kMinusInf;
  if (eos >= 0) {
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
      const int e = first + j * kThreads * kN;
      if (eos >= e && eos < e + kN) {
#pragma unroll
        for (int i = 0; i < kN; ++i)
          if (i == eos - e) end = G::at(v[j], i);
        G::erase(v[j], eos - e);
        eos_logit = end;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < VECS; ++j) top = fmaxf(top, G::max(v[j]));
  float m8 = top;
#pragma unroll
  for (int d = 1; d < 8; d *= 2) m8 = fmaxf(m8, __shfl_xor_sync(0xFFFFFFFFu, m8, d));
  if ((lane & 7) == 0) group_max[tid >> 3] = m8;
  __syncthreads();
  // the block's maximum, and a bound that `beams` continuations reach: the
  // beams-th largest of the groups' maxima
  uint32_t o = ordered(group_max[lane]);
  const float best = from_ordered(__reduce_max_sync(0xFFFFFFFFu, o));
  const float ref = fmaxf(best, eos_logit);
  u64* keys = reinterpret_cast<u64*>(a.keys) + (size_t)blockIdx.x * a.beams;
  if (ref == kMinusInf) {
    for (int i = tid; i < a.beams; i += kThreads) keys[i] = 0ull;
    if (tid == 0) a.stats[blockIdx.x] = make_float2(kMinusInf, 0.f);
    return;
  }
  float bound = kMinusInf;
  for (int left = a.beams; left > 0;) {
    const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, o);
    bound = from_ordered(m);
    left -= __popc(__ballot_sync(0xFFFFFFFFu, o == m));
    if (o == m) o = 0u;
  }
  // (groups run out only when all are counted: 32 of them, beams <= 32)

  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < VECS; ++j)
#pragma unroll
    for (int i = 0; i < kN; ++i) sum += ex2((G::at(v[j], i) - ref) * kLog2e);
  if (end > kMinusInf) sum += ex2((end - ref) * kLog2e);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
  if (lane == 0) warp_sum[warp] = sum;

  if (top >= bound && top > kMinusInf) {
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
      if (G::max(v[j]) < bound) continue;
      const int e = first + j * kThreads * kN;
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const float l = G::at(v[j], i);
        if (l >= bound && l > kMinusInf) {
          const int at = atomicAdd(&listed, 1);
          if (at < kList) list[at] = make_key(l, (uint32_t)(e + i));
        }
      }
    }
  }
  __syncthreads();
  if (tid == 0) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += warp_sum[w];
    a.stats[blockIdx.x] = make_float2(ref, ref == -kMinusInf ? 1.f : s);
  }
  const int count = listed;
  if (count <= kList) {
    if (tid < count) {
      const u64 mine = list[tid];
      int rank = 0;
      for (int i = 0; i < count; ++i) rank += list[i] > mine;
      if (rank < a.beams) keys[rank] = mine;
    }
    for (int i = count + tid; i < a.beams; i += kThreads) keys[i] = 0ull;
    return;
  }
  // many equal logits: the best of all threads, one after another; the thread
  // that gave one looks for its next
  auto below = [&](u64 limit) {
    u64 k = 0ull;
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
      const int e = first + j * kThreads * kN;
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const float l = G::at(v[j], i);
        const u64 c = l > kMinusInf ? make_key(l, (uint32_t)(e + i)) : 0ull;
        if (c < limit && c > k) k = c;
      }
    }
    return k;
  };
  u64 mine = below(~0ull);
  for (int r = 0; r < a.beams; ++r) {
    const u64 w = warp_max(mine);
    if (lane == 0) best_of[r & 1][warp] = w;
    __syncthreads();
    const u64 b = warp_max(best_of[r & 1][lane & (kWarps - 1)]);
    if (tid == 0) keys[r] = b;
    if (b != 0ull && mine == b) mine = below(b);
  }
}

// ---------------------------------------------------------------------------
// One sequence.
// ---------------------------------------------------------------------------
// log(t) for t in [1, 2^31): exponent and mantissa apart, so that the error is
// fp32's of a value below 1.
__device__ __forceinline__ double log_of_sum(double t) {
  const u64 bits = (u64)__double_as_longlong(t);
  const int e = (int)(bits >> 52) - 1023;
  const double m = __longlong_as_double((long long)((bits & 0xFFFFFFFFFFFFFull) | 0x3FF0000000000000ull));
  const float mf = (float)m;
  const float rest = (float)(m - (double)mf) / mf;          // log(m) = log(mf) + log(1 + rest)
  return (double)e * 0.69314718055994530942 + ((double)logf(mf) + (double)rest);
}

__device__ __forceinline__ u64 ordered64(double v) {
  const u64 b = (u64)__double_as_longlong(v);
  return b ^ ((u64)((long long)b >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double from_ordered64(u64 o) {
  return __longlong_as_double((long long)(o ^ ((o >> 63) ? 0x8000000000000000ull : ~0ull)));
}

struct RowStats {
  double log_sum;            // of exp(l - top)
  float top;
  float score;               // of the beam
};

// The ordered score of a logit in a row, 0 where it does not continue the beam.
__device__ __forceinline__ u64 score_of(const RowStats& r, float l) {
  if (!(fabsf(r.score) <= 3.4028235e38f) || !(l > kMinusInf)) return 0ull;
  if (r.top == -kMinusInf) return l == r.top ? ordered64((double)r.score) : 0ull;
  return ordered64((double)r.score + ((double)l - (double)r.top - r.log_sum));
}

template <typename T>
__global__ void __launch_bounds__(kThreads) beam_join_kernel(const BeamSelectArgs a) {
  __shared__ RowStats stats[WQL_MAX_BEAMS];
  __shared__ u64 score[WQL_MAX_BEAMS][WQL_MAX_BEAMS];       // [beam][rank in the beam]
  __shared__ uint32_t token[WQL_MAX_BEAMS][WQL_MAX_BEAMS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_launch_dependents();
  griddep_wait();
  const int beams = a.beams, parts = a.parts, row0 = blockIdx.x * beams;
  for (int w = warp; w < beams; w += kWarps) {
    const float2* st = a.stats + (size_t)(row0 + w) * parts;
    float2 mine[kLanes];
    float top = kMinusInf;
#pragma unroll
    for (int q = 0; q < kLanes; ++q) {
      const int p = lane + 32 * q;
      mine[q] = p < parts ? st[p] : make_float2(kMinusInf, 0.f);
      top = fmaxf(top, mine[q].x);
    }
    top = from_ordered(__reduce_max_sync(0xFFFFFFFFu, ordered(top)));
    double sum = 0.;
#pragma unroll
    for (int q = 0; q < kLanes; ++q)
      if (mine[q].x > kMinusInf && top < -kMinusInf)
        sum += (double)mine[q].y * (double)ex2((mine[q].x - top) * kLog2e);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
    RowStats r;
    r.top = top;
    r.score = a.scores[row0 + w];
    r.log_sum = sum >= 1. ? log_of_sum(sum) : 0.;
    if (lane == 0) stats[w] = r;
    // the row's best `beams`: every lane holds the heads of its parts' lists
    const u64* keys = reinterpret_cast<const u64*>(a.keys) + (size_t)(row0 + w) * parts * beams;
    u64 head[kLanes];
    int at[kLanes];
#pragma unroll
    for (int q = 0; q < kLanes; ++q) {
      const int p = lane + 32 * q;
      head[q] = p < parts ? keys[(size_t)p * beams] : 0ull;
      at[q] = 0;
    }
    for (int i = 0; i < beams; ++i) {
      u64 k = head[0];
#pragma unroll
      for (int q = 1; q < kLanes; ++q) k = head[q] > k ? head[q] : k;
      const u64 b = warp_max(k);
      if (lane == 0) {
        score[w][i] = b ? score_of(r, key_logit(b)) : 0ull;
        token[w][i] = key_token(b);
      }
      if (b == 0ull) continue;
#pragma unroll
      for (int q = 0; q < kLanes; ++q)
        if (head[q] == b)
          head[q] = ++at[q] < beams ? keys[(size_t)(lane + 32 * q) * beams + at[q]] : 0ull;
    }
  }
  __syncthreads();
  if (warp != 0) return;
  // lane w: beam w's list, best first
  const bool in = lane < beams;
  u64 end = 0ull;
  if (a.ended && in && a.eos >= 0)
    end = score_of(stats[lane], fmaxf(to_f32(static_cast<const T*>(a.logits)[(size_t)(row0 + lane) * a.n + a.eos]), kMinusInf));
  int at = 0, slot_beam = -1;                              // lane i: the i-th best
  u64 head = in ? score[lane][0] : 0ull, slot_score = 0ull;
  uint32_t slot_token = 0u;
  int larger = 0;                                          // continuations that beat this beam's end
  for (int i = 0; i < beams; ++i) {
    const u64 b = warp_max(head);
    if (b == 0ull) break;
    larger += b > end;
    const int w = __ffs(__ballot_sync(0xFFFFFFFFu, head == b)) - 1;
    const int j = __shfl_sync(0xFFFFFFFFu, at, w);
    if (lane == i) {
      slot_beam = w;
      slot_score = b;
      slot_token = token[w][j];
    }
    if (lane == w) head = ++at < beams ? score[w][at] : 0ull;
  }
  if (a.ended) {
    for (int i = 0; i < beams; ++i) larger += __shfl_sync(0xFFFFFFFFu, end, i) > end;
    if (in)
      a.ended[row0 + lane] = end != 0ull && larger < beams ? (float)from_ordered64(end) : kMinusInf;
  }
  int slot = lane;
  if (a.order == WQL_BEAM_ANCHORED) {
    // lanes of one beam: the lowest takes its slot, the others the free ones
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, slot_beam);
    const bool stays = slot_beam >= 0 && __ffs(same) - 1 == lane;
    const uint32_t taken = __reduce_or_sync(0xFFFFFFFFu, stays ? 1u << slot_beam : 0u);
    const uint32_t moves = __ballot_sync(0xFFFFFFFFu, !stays);
    uint32_t open = ~taken;                                // lanes past the beams go past them
    for (int i = __popc(moves & ((1u << lane) - 1u)); i > 0; --i) open &= open - 1u;
    slot = stays ? slot_beam : __ffs(open) - 1;
  }
  if (in) {
    const int to = row0 + slot;
    a.tokens[to] = slot_beam >= 0 ? (int32_t)slot_token : -1;
    a.parents[to] = slot_beam;
    a.scores_out[to] = slot_beam >= 0 ? (float)from_ordered64(slot_score) : kMinusInf;
  }
}

template <typename T, int VECS> cudaError_t launch_v(const BeamSelectArgs& a, cudaStream_t s) {
  const bool aligned = a.n % Group<T>::kN == 0 && reinterpret_cast<uintptr_t>(a.logits) % 16 == 0;
  cudaError_t e = launch_pdl(aligned ? beam_part_kernel<T, VECS, true> : beam_part_kernel<T, VECS, false>,
                             dim3((unsigned)(a.batch * a.beams) * (unsigned)a.parts),
                             dim3(kThreads), 0, s, a);
  if (e != cudaSuccess) return e;
  note_launch();
  e = launch_pdl(beam_join_kernel<T>, dim3((unsigned)a.batch), dim3(kThreads), 0, s, a);
  if (e == cudaSuccess) note_launch();
  return e;
}

template <typename T> cudaError_t launch_t(const BeamSelectArgs& a, cudaStream_t s) {
  constexpr int kN = Group<T>::kN;
  return beam_part_elements((int64_t)a.batch * a.beams, a.n) == kSmall
             ? launch_v<T, kSmall / kThreads / kN>(a, s) : launch_v<T, kLarge / kThreads / kN>(a, s);
}

int parts_of(int64_t n, int elements) { return (int)((n + elements - 1) / elements); }

}  // namespace

// Small parts where the large ones would not give every SM two blocks, and the
// lists of a row still fit the lanes that join them.
int beam_part_elements(int64_t rows, int64_t n) {
  return rows * parts_of(n, kLarge) < 304 && parts_of(n, kSmall) <= 32 * kLanes ? kSmall : kLarge;
}
int beam_parts(int64_t rows, int64_t n) { return parts_of(n, beam_part_elements(rows, n)); }
static_assert((WQL_BEAM_MAX_N + kLarge - 1) / kLarge <= 32 * kLanes, "lists of a row");

cudaError_t launch_beam_select(const BeamSelectArgs& a, cudaStream_t s) {
  switch (a.dtype) {
    case WQL_F32: return launch_t<float>(a, s);
    case WQL_F16: return launch_t<__half>(a, s);
    default: return launch_t<__nv_bfloat16>(a, s);
  }
}

}  // namespace wql
