// beam_select.cu -- one step of beam search: the best `beams` continuations of
// a sequence's beams * n by s[w, v] = scores[w] + l[w, v] - log sum exp l[w, :].
//
// Two launches.  beam_part_kernel reads the logits once, a block per part of a
// row: the part's maximum, its sum of exponentials and its best `beams`
// continuations.  beam_join_kernel, a block per sequence, joins the sums, takes
// the best of each row's lists, and the best of those.
//
// Inside a row the order of the scores is that of the logits, so lists hold
// (logit, token) keys and no score; scores exist for beams * beams keys only.
// Every order is total (ties by token, then by beam), hence results do not
// depend on the order in which lists were filled.
//
// HBM-bound, where there are logits enough: 16 sequences x 16 beams x 248320 fp32
// 54.7 us (68 % of the copy rate), 64 x 4 x 151936 bf16 24.6 us (47 %): its logits
// arrive in 11 to 14 us, at the copy rate; 3.5 us follow for the ends of the
// parts, 1 for the second launch and 3 for the joining.  1 x 4 x 151936 bf16 7.6
// us, 7 x 5 x 50303 fp16 10.0 us, of which the two launches and their dependent
// steps are all.  All but a thousandth masked by -1e9 or -inf costs nothing more; by a
// value beyond -1.4e9, whose exponentials take the slower form, 64 x 4 x 151936 38.5.
#include "requests.cuh"
#include "sm100.cuh"

namespace wql {
namespace {

using u64 = unsigned long long;
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kResident = 4;             // blocks on an SM
constexpr int kVecs = 4;                 // 16-byte groups a lane takes of a chunk
constexpr int kStages = 2;               // chunks on their way to a warp
constexpr int kSlot = 32 * kVecs + 1;    // 16-byte groups of one
constexpr size_t kRing = (size_t)kWarps * kStages * kSlot * 16;
constexpr int kBlocks = 152 * kResident; // at a time on 152 SMs
constexpr int kTops = 16;                // chunks whose maxima are held
constexpr int kList = 64;                // a warp's list: the best and 32 more
constexpr int kStaged = 4096;            // keys of a sequence that are joined in shared memory
constexpr int kMaxLists = 8;             // lists a lane looks after when a row is joined
constexpr int kGroups = kWarps * kList * 2;  // groups looked at once more
static_assert(kThreads >= kWarps * WQL_MAX_BEAMS && WQL_MAX_BEAMS < 64, "a thread for every list's keys");
static_assert(kList >= WQL_MAX_BEAMS + 32, "room for one from every lane");
static_assert(WQL_BEAM_MAX_N / (32 * kVecs * 4 * kWarps) <= 32 * kMaxLists, "of one chunk a warp");
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kMinusInf = -__builtin_huge_valf();
constexpr float kLargest = 3.4028235e38f;

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

// Exponentials are taken as 2^(l * log2 e - base(m)) over a maximum m: one
// fused multiply-add, whose base is an fp32 number, so that its rounding is
// none of the sum's (as long as all take the same one: a product that the compiler
// fuses into a difference of two bases is not rounded).  At l = m the exponent is that
// rounding, up to half a unit in base's last place, not 0.  Below 2^31 it is at most 64,
// so that sums of 2^20 terms stay in fp32's range (and where it is more than 10, logits
// lie more than 14 apart); from there on, which takes masks of large finite values,
// exponentials are 2^((l - m) * log2 e).  m alone decides.
constexpr float kPlain = 2147483648.f;
__device__ __forceinline__ bool plain_base(float b) { return fabsf(b) < kPlain; }
__device__ __forceinline__ float base(float m) { return __fmul_rn(m, kLog2e); }
__device__ __forceinline__ bool plain(float m) { return plain_base(base(m)); }
__device__ __forceinline__ double base64(float m) {
  return plain(m) ? (double)base(m) : (double)m * (double)kLog2e;
}
// What a sum over `from` is multiplied with to be one over `to`, from <= to.
__device__ __forceinline__ float rescale(float from, float to) {
  if (from == to) return 1.f;
  const float a = base(from), b = base(to);
  const bool p = plain_base(a), q = plain_base(b);
  // each less what it is held over
  return ex2(fmaf((p ? 0.f : from) - (q ? 0.f : to), kLog2e, (p ? a : 0.f) - (q ? b : 0.f)));
}

// Two floats in one register pair.
__device__ __forceinline__ u64 pair2(float a, float b) {
  u64 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair2(u64 v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ u64 fma2(u64 a, u64 b, u64 c) {
  u64 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ u64 add2(u64 a, u64 b) {
  u64 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// The 16 bytes of a group of elements as they are held.
template <typename T> struct Group;
template <> struct Group<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ float at(const uint4& v, int i) {
    return __uint_as_float(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w);
  }
  // The largest of all (a NaN is not larger than anything); -inf at least.
  template <int N> static __device__ __forceinline__ float max(const uint4 (&v)[N]) {
    float m = kMinusInf;
#pragma unroll
    for (int j = 0; j < N; ++j) m = fmaxf(fmaxf(m, fmaxf(at(v[j], 0), at(v[j], 1))), fmaxf(at(v[j], 2), at(v[j], 3)));
    return m;
  }
};
template <typename T, typename T2> struct Group16 {
  static constexpr int kN = 8;
  static __device__ __forceinline__ float at(const uint4& v, int i) {
    const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    const uint16_t h = (uint16_t)(w >> (16 * (i & 1)));
    return to_f32(*reinterpret_cast<const T*>(&h));
  }
  static __device__ __forceinline__ T2 two(const uint32_t& v) { return *reinterpret_cast<const T2*>(&v); }
  template <int N> static __device__ __forceinline__ float max(const uint4 (&v)[N]) {
    T2 m = two(v[0].x);
#pragma unroll
    for (int j = 0; j < N; ++j)
      m = __hmax2(__hmax2(m, __hmax2(two(v[j].x), two(v[j].y))), __hmax2(two(v[j].z), two(v[j].w)));
    return fmaxf(fmaxf(kMinusInf, to_f32(m.x)), to_f32(m.y));
  }
};
template <> struct Group<__half> : Group16<__half, __half2> {};
template <> struct Group<__nv_bfloat16> : Group16<__nv_bfloat16, __nv_bfloat162> {};

// Elements [e, e + kN) of a row of n that starts at `row`, one by one; -inf
// outside the row.
template <typename T> __device__ __noinline__ uint4 edge_group(const T* row, int e, int n) {
  constexpr int kN = Group<T>::kN;
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kN == 4) {
      w[i] = e + i >= 0 && e + i < n ? __float_as_uint(row[e + i]) : 0xFF800000u;
    } else {
      const T none = from_f32<T>(kMinusInf);
      const int k = e + 2 * i;
      const T lo = k >= 0 && k < n ? row[k] : none, hi = k + 1 >= 0 && k + 1 < n ? row[k + 1] : none;
      w[i] = (uint32_t)*reinterpret_cast<const uint16_t*>(&lo) |
             (uint32_t)*reinterpret_cast<const uint16_t*>(&hi) << 16;
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// The same where `row + e` lies on a 16-byte address; e may be negative.
template <typename T> __device__ __forceinline__ uint4 load_group(const T* row, int e, int n) {
  if (e >= 0 && e + Group<T>::kN <= n) return __ldg(reinterpret_cast<const uint4*>(row + e));
  return edge_group(row, e, n);
}
// 16 bytes to shared memory, on their way when it returns.
__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
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

// Ranks a list by counting and keeps the best `beams`, in order; the last of
// those, or 0 where there are fewer.  (A call: inlined, its copies push the
// loop around it out of the instruction cache.)
__device__ __noinline__ u64 settle(u64* list, int count, int beams, int lane) {
  const u64 e0 = lane < count ? list[lane] : 0ull, e1 = lane + 32 < count ? list[lane + 32] : 0ull;
  int r0 = 0, r1 = 0;
  for (int k = 0; k < count; ++k) {
    const u64 x = list[k];
    r0 += x > e0;
    r1 += x > e1;
  }
  __syncwarp();
  if (lane < count && r0 < beams) list[r0] = e0;
  if (lane + 32 < count && r1 < beams) list[r1] = e1;
  __syncwarp();
  return count >= beams ? list[beams - 1] : 0ull;
}

// A warp's best continuations so far, in shared memory.
struct Best {
  u64* list;
  int count;
  u64 limit;                  // the beams-th best, or 0 while there are fewer

  __device__ __forceinline__ void keep_best(int beams, int lane) {
    limit = settle(list, count, beams, lane);
    count = min(count, beams);
  }

  // The whole warp; a key of each lane that has one.
  __device__ __forceinline__ void add(u64 key, bool in, int beams, int lane) {
    uint32_t who = __ballot_sync(0xFFFFFFFFu, in);
    if (count + __popc(who) > kList) {
      keep_best(beams, lane);
      in = in && key > limit;
      who = __ballot_sync(0xFFFFFFFFu, in);
    }
    if (in) list[count + __popc(who & ((1u << lane) - 1u))] = key;
    count += __popc(who);
    __syncwarp();
  }
};

// ---------------------------------------------------------------------------
// One part of a row, a block's: chunks of kVecs groups of 16 bytes a lane, dealt
// to the warps in turn and copied ahead into each warp's own ring.  Every lane
// keeps its own maximum and sum, and the maximum of its group of each chunk.
// The loop over the logits looks for nothing else: at its end the beams-th
// largest of the maxima of 64 columns of lanes bounds the best continuations from
// below, and the few groups that reach it are read once more.  (Appending to
// lists inside the loop cost more than the sums: 64 x 4 x 151936 bf16 44 us for
// the call.)  Blocks stay and take a part after another; their copies run on into
// the next part while this one's end is worked on.
// Which tokens a lane has does not depend on where the row starts, so that
// equal rows give equal sums and their ties go to the lower beam; a row off a
// 16-byte boundary is read in aligned groups, two of which make one (ALIGNED:
// no row is).
// stats[row][part] = (maximum, sum), (-inf, 0) without any;
// keys[row][part][0 .. beams) = the best continuations but eos, 0 past them.
// ---------------------------------------------------------------------------
template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, kResident) beam_part_kernel(const BeamSelectArgs a) {
  using G = Group<T>;
  constexpr int kN = G::kN, kChunk = 32 * kVecs * kN;
  extern __shared__ uint4 ring[];                        // [warp][stage][kSlot]
  __shared__ u64 lists[kWarps][kList];
  __shared__ float tops[kWarps][kTops * 32];
  __shared__ float peaks[kWarps][32];
  __shared__ float2 sums[kWarps];
  __shared__ float bound_of_all;
  __shared__ int counts[kWarps];
  __shared__ u64 all[kThreads];
  __shared__ int grouped, listed;
  int* group = reinterpret_cast<int*>(lists);            // (one or the other is in use)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  griddep_launch_dependents();
  griddep_wait();
  const int jobs = a.batch * a.beams * a.parts, beams = a.beams;
  constexpr int kStep = kWarps * kChunk;                 // from a warp's chunk to its next
  // The warp's chunks of a job, a part of a row.
  struct Job {
    const T* logits;                                     // the row
    int mis, first, end;
  };
  auto job_of = [&](int job) {
    const int row = job / a.parts, part = job - row * a.parts;
    Job j;
    j.logits = static_cast<const T*>(a.logits) + (size_t)row * a.n;
    j.mis = ALIGNED ? 0 : (int)(reinterpret_cast<uintptr_t>(j.logits) / sizeof(T)) & (kN - 1);
    j.first = (part * a.part_chunks + warp) * kChunk;
    j.end = min((part + 1) * a.part_chunks * kChunk, a.n);
    return j;
  };

  // Copies run kStages chunks ahead, into the next job where one ends.
  int ahead = blockIdx.x;
  Job next = job_of(ahead);
  auto copy = [&](uint32_t to) {
    while (ahead < jobs && next.first >= next.end) {
      ahead += gridDim.x;
      if (ahead < jobs) next = job_of(ahead);
    }
    if (ahead < jobs) {
      const int c = next.first;
      next.first += kStep;
      // groups on 16-byte addresses, and the one behind them, which the last of
      // a row off the boundary reaches into
      if (c - next.mis >= 0 && c + kChunk + (ALIGNED ? 0 : kN) <= a.n) {     // all inside the row
        const T* from = next.logits + (c - next.mis + lane * kN);
#pragma unroll
        for (int j = 0; j < kVecs; ++j) copy16(to + (uint32_t)(j * 32 + lane) * 16, from + j * 32 * kN);
        if (!ALIGNED && lane == 0) copy16(to + kVecs * 32 * 16, from + kChunk);
      } else {
        uint4* at = reinterpret_cast<uint4*>(__cvta_shared_to_generic(to));
        for (int j = lane; j < kVecs * 32 + (ALIGNED ? 0 : 1); j += 32)
          at[j] = load_group(next.logits, c + j * kN - next.mis, a.n);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  float* top_of = tops[warp] + lane;
  const uint32_t slot = (uint32_t)__cvta_generic_to_shared(ring + warp * kStages * kSlot);
  int stage = 0;
#pragma unroll
  for (int i = 0; i < kStages; ++i) copy(slot + i * kSlot * 16);
  for (int job = blockIdx.x; job < jobs; job += gridDim.x) {
    const Job now = job_of(job);
    const int first = now.first, end = now.end, mis = now.mis;
    float m = kMinusInf, sum = 0.f;                        // this lane's
    int held = 0;
    for (int c = first; c < end; c += kStep, ++held) {
      uint4 v[kVecs];
      const uint32_t here = slot + (uint32_t)stage * (kSlot * 16);
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      __syncwarp();                                        // the other lanes' copies too
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        v[j] = lds128(here + (uint32_t)(j * 32 + lane) * 16);
        if (!ALIGNED && mis) v[j] = shifted<T>(v[j], lds128(here + (uint32_t)(j * 32 + lane + 1) * 16), mis);
      }
      __syncwarp();                                        // before they are overwritten
      copy(here);
      stage = stage + 1 == kStages ? 0 : stage + 1;
      const float top = G::max(v);
      top_of[32 * held] = top;
      if (top > m) {
        sum = m == kMinusInf ? 0.f : sum * rescale(m, top);
        m = top;
      }
      // (a lane that has seen -inf alone: over 0)
      const float over = m == kMinusInf ? 0.f : base(m);
      const u64 slope = pair2(kLog2e, kLog2e), shift = pair2(-over, -over);
      u64 part0 = 0ull, part1 = 0ull;
#pragma unroll
      for (int j = 0; j < kVecs; ++j)
#pragma unroll
        for (int i = 0; i < kN; i += 4) {
          float e0, e1, e2, e3;
          unpair2(fma2(pair2(G::at(v[j], i), G::at(v[j], i + 1)), slope, shift), e0, e1);
          unpair2(fma2(pair2(G::at(v[j], i + 2), G::at(v[j], i + 3)), slope, shift), e2, e3);
          part0 = add2(part0, pair2(ex2(e0), ex2(e1)));
          part1 = add2(part1, pair2(ex2(e2), ex2(e3)));
        }
      float p0, p1;
      unpair2(add2(part0, part1), p0, p1);
      float more = p0 + p1;
      if (!(more <= kLargest && plain_base(over))) {       // NaN among them, or m is far from zero
        more = 0.f;
#pragma unroll
        for (int j = 0; j < kVecs; ++j)
#pragma unroll
          for (int i = 0; i < kN; ++i) {
            const float l = G::at(v[j], i);
            if (l > kMinusInf) more += plain(m) ? ex2(fmaf(l, kLog2e, -over)) : ex2((l - m) * kLog2e);
          }
      }
      sum += more;
    }

    peaks[warp][lane] = m;
    const float top = from_ordered(__reduce_max_sync(0xFFFFFFFFu, ordered(m)));
    sum = m == kMinusInf || top == -kMinusInf ? 0.f : sum * rescale(m, top);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
    if (lane == 0) sums[warp] = make_float2(top, sum);
    __syncthreads();
    if (warp == 0) {
      // An element of each of so many columns, 64 of them, reaches this (one may
      // be eos).
      float even = peaks[0][lane], odd = peaks[1][lane];
#pragma unroll
      for (int w = 2; w < kWarps; w += 2) {
        even = fmaxf(even, peaks[w][lane]);
        odd = fmaxf(odd, peaks[w + 1][lane]);
      }
      uint32_t o0 = ordered(even), o1 = ordered(odd), w = 0u;
      for (int left = beams + (a.eos >= 0); left > 0;) {
        w = __reduce_max_sync(0xFFFFFFFFu, max(o0, o1));
        left -= __popc(__ballot_sync(0xFFFFFFFFu, o0 == w)) + __popc(__ballot_sync(0xFFFFFFFFu, o1 == w));
        o0 = o0 == w ? 0u : o0;
        o1 = o1 == w ? 0u : o1;
      }
      if (lane == 0) {
        bound_of_all = from_ordered(w);
        grouped = listed = 0;
      }
    } else if (warp == 1) {
      const float2 mine = lane < kWarps ? sums[lane] : make_float2(kMinusInf, 0.f);
      const float all = from_ordered(__reduce_max_sync(0xFFFFFFFFu, ordered(mine.x)));
      float s = mine.x == kMinusInf || all == -kMinusInf ? 0.f : mine.y * rescale(mine.x, all);
#pragma unroll
      for (int d = 4; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
      if (lane == 0) a.stats[job] = make_float2(all, s);
    }
    __syncthreads();
    const float bound = bound_of_all;
    const int t = threadIdx.x;
    // the groups that reach it, one of each lane and chunk
    if (m >= bound && m > kMinusInf)
      for (int q = 0; q < held; ++q)
        if (top_of[32 * q] >= bound) {
          const int at = atomicAdd(&grouped, 1);
          if (at < kGroups) group[at] = first + q * kStep + lane * kN;     // its first token
        }
    __syncthreads();
    // once more, 16 bytes a thread, for the elements that do
    if (grouped <= kGroups)
      for (int i = t; i < grouped * kVecs; i += kThreads) {
        const int token = group[i / kVecs] + i % kVecs * 32 * kN, e = token - mis;
        uint4 g = load_group(now.logits, e, a.n);
        if (!ALIGNED && mis) g = shifted<T>(g, load_group(now.logits, e + kN, a.n), mis);
#pragma unroll
        for (int k = 0; k < kN; ++k) {
          const float l = G::at(g, k);
          if (l >= bound && l > kMinusInf && token + k != a.eos) {
            const int at = atomicAdd(&listed, 1);
            if (at < kThreads) all[at] = make_key(l, (uint32_t)(token + k));
          }
        }
      }
    __syncthreads();
    int total = listed;
    if (grouped > kGroups || total > kThreads) {
      // Many equal ones: every warp's own best, then those together.
      Best best{lists[warp], 0, 0ull};
      for (int q = 0; q < held; ++q) {
        const int c = first + q * kStep;
        const float peak = top_of[32 * q];
        const bool look = peak >= bound && peak > kMinusInf && make_key(peak, (uint32_t)(c + lane * kN)) > best.limit;
        if (!__any_sync(0xFFFFFFFFu, look)) continue;
        for (int j = 0; j < kVecs; ++j) {
          const int token = c + (j * 32 + lane) * kN, e = token - mis;
          uint4 g = load_group(now.logits, e, a.n);
          if (!ALIGNED && mis) g = shifted<T>(g, load_group(now.logits, e + kN, a.n), mis);
#pragma unroll 1
          for (int k = 0; k < kN; ++k) {
            const float l = G::at(g, k);
            const u64 key = make_key(l, (uint32_t)(token + k));
            best.add(key, look && l >= bound && l > kMinusInf && token + k != a.eos && key > best.limit,
                     beams, lane);
          }
        }
      }
      best.keep_best(beams, lane);
      if (lane == 0) counts[warp] = best.count;
      __syncthreads();
      int before = 0;
      total = 0;
      for (int w = 0; w < kWarps; ++w) {
        before += w < warp ? counts[w] : 0;
        total += counts[w];
      }
      if (lane < best.count) all[before + lane] = best.list[lane];
      __syncthreads();
    }
    // ranked by counting, one key a thread
    u64* keys = reinterpret_cast<u64*>(a.keys) + (size_t)job * beams;
    if (t < total) {
      const u64 mine = all[t];
      int rank = 0;
      for (int i = 0; i < total; ++i) rank += all[i] > mine;
      if (rank < beams) keys[rank] = mine;
    }
    if (t >= total && t < beams) keys[t] = 0ull;
  }
}

// ---------------------------------------------------------------------------
// One sequence.
// ---------------------------------------------------------------------------
// Sums and scores are held in two fp32 parts, hi the nearest fp32 number and lo
// the rest: some 46 bits, which keep the logits' order and their distances; the parts'
// sums and the logarithm of the row's are fp32's.  (In binary64 a sequence of 16 beams
// took 4 us more: the SM does two such operations a cycle.)
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Two normal(float hi, float lo) {            // |lo| <= |hi|
  const float s = __fadd_rn(hi, lo);
  return {s, __fsub_rn(lo, __fsub_rn(s, hi))};
}
__device__ __forceinline__ Two add(Two a, Two b) {
  const Two s = two_sum(a.hi, b.hi);
  return normal(s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)));
}
__device__ __forceinline__ Two split(double v) {
  const float hi = (float)v;
  return {hi, (float)(v - (double)hi)};
}

// log2(t) for a normal t: the exponent and the logarithm of what is left, which lies
// in [0, 1].
__device__ __forceinline__ Two log2_of(Two t) {
  const int e = (int)(__float_as_uint(t.hi) >> 23) - 127;
  const float m = __uint_as_float((__float_as_uint(t.hi) & 0x007FFFFFu) | 0x3F800000u);
  const Two whole = two_sum((float)e, log2f(m));
  return normal(whole.hi, fmaf(t.lo / t.hi, kLog2e, whole.lo));
}

struct RowStats {
  Two over;                  // log2 of the sum of 2^(l log2 e - base(top))
  float top;
  float score;               // of the beam
  float end;                 // the end token's logit, or -inf
};

// log2 e is fp32's in the sums and here, and scores are divided by the same: of l - top
// nothing is lost, and the logarithm of the sum is off by 1.3e-8 of the mean of top - l.
constexpr double kPerLog2 = 1.0 / (double)kLog2e;

// The score of a logit in a row as a key (larger scores have larger keys), 0
// where it does not continue the beam.
__device__ __forceinline__ u64 score_of(const RowStats& r, float l) {
  if (!(fabsf(r.score) <= kLargest) || !(l > kMinusInf)) return 0ull;
  Two s{r.score, 0.f};
  if (r.top == -kMinusInf) {
    if (l != r.top) return 0ull;
  } else if (fabsf(l) < 1e38f && plain(r.top)) {
    const float p = __fmul_rn(l, kLog2e);
    const Two d = add(add({p, fmaf(l, kLog2e, -p)}, {-base(r.top), 0.f}), {-r.over.hi, -r.over.lo});
    constexpr float kPer = (float)kPerLog2, kPerRest = (float)(kPerLog2 - (double)kPer);
    const float q = __fmul_rn(d.hi, kPer);
    s = add(s, normal(q, fmaf(d.lo, kPer, fmaf(d.hi, kPerRest, fmaf(d.hi, kPer, -q)))));
  } else {                   // a row of masks, or a masked token of the lowest values
    // (the maximum first: the logarithm of the sum would be lost beside it)
    const double d = ((double)l * (double)kLog2e - base64(r.top)) - ((double)r.over.hi + (double)r.over.lo);
    s = split((double)r.score + d * kPerLog2);
  }
  if (!(s.hi >= -kLargest)) return 0ull;                     // below fp32's range, or NaN of its sums
  return (u64)ordered(s.hi + 0.f) << 32 | ordered(s.lo + 0.f);
}
__device__ __forceinline__ float key_score(u64 k) { return from_ordered((uint32_t)(k >> 32)); }

// A warp per beam, LISTS lists a lane.  Latency alone, and fetching its own
// instructions is a part of it: so it goes through them once before the parts are
// there, over made-up lists (half a microsecond less).
template <typename T, int LISTS>
__global__ void __launch_bounds__(32 * WQL_MAX_BEAMS) beam_join_kernel(const BeamSelectArgs a) {
  __shared__ RowStats stats[WQL_MAX_BEAMS];
  __shared__ u64 score[WQL_MAX_BEAMS][WQL_MAX_BEAMS];       // [beam][rank in the beam]
  __shared__ uint32_t token[WQL_MAX_BEAMS][WQL_MAX_BEAMS];
  __shared__ int place[WQL_MAX_BEAMS];                      // beam * 32 + rank in it, of the i-th best
  extern __shared__ u64 staged_keys[];                      // [beam][part][beams]
  const bool staged = a.beams * a.parts * a.beams <= kStaged;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  griddep_launch_dependents();
  const int beams = a.beams, row0 = blockIdx.x * beams;
  for (int pass = 0; pass < 2; ++pass) {
    if (pass != 0) griddep_wait();
    const int parts = pass != 0 ? a.parts : 0;
    {
      const int w = warp;
      const float2* st = a.stats + (size_t)(row0 + w) * parts;
      const u64* keys = reinterpret_cast<const u64*>(a.keys) + (size_t)(row0 + w) * parts * beams;
      // all loads that wait for nothing but the parts
      float2 mine[LISTS];
#pragma unroll
      for (int q = 0; q < LISTS; ++q) {
        const int p = lane + 32 * q;
        mine[q] = make_float2(0.f, 1.f);
        if (pass != 0) mine[q] = p < parts ? st[p] : make_float2(kMinusInf, 0.f);
      }
      RowStats r;
      r.score = pass != 0 ? a.scores[row0 + w] : 0.f;
      r.end = kMinusInf;
      if (a.ended && a.eos >= 0 && pass != 0)
        r.end = fmaxf(to_f32(static_cast<const T*>(a.logits)[(size_t)(row0 + w) * a.n + a.eos]), kMinusInf);
      if (staged) {
        // the row's lists in shared memory: a list's next key is a step of every
        // round below
        u64* own = staged_keys + w * a.parts * beams;
        for (int i = lane; i < parts * beams; i += 32) own[i] = keys[i];
        keys = own;
        __syncwarp();
      }
      u64 head[LISTS];
      int at[LISTS];
      float top = kMinusInf;
#pragma unroll
      for (int q = 0; q < LISTS; ++q) {
        const int p = lane + 32 * q;
        head[q] = make_key((float)lane, 1u);
        if (pass != 0) head[q] = p < parts ? keys[p * beams] : 0ull;
        at[q] = 0;
      }
#pragma unroll
      for (int q = 0; q < LISTS; ++q) top = fmaxf(top, mine[q].x);
      top = from_ordered(__reduce_max_sync(0xFFFFFFFFu, ordered(top)));
      Two sum{0.f, 0.f};
#pragma unroll
      for (int q = 0; q < LISTS; ++q)
        if (mine[q].x > kMinusInf && top < -kMinusInf)
          sum = add(sum, {mine[q].y * rescale(mine[q].x, top), 0.f});
#pragma unroll
      for (int d = 16; d > 0; d >>= 1)
        sum = add(sum, {__shfl_xor_sync(0xFFFFFFFFu, sum.hi, d), __shfl_xor_sync(0xFFFFFFFFu, sum.lo, d)});
      r.top = top;
      r.over = sum.hi > 0.f ? log2_of(sum) : Two{0.f, 0.f};
      if (lane == 0) stats[w] = r;
      // the row's best `beams`, one after another: lane i gets the i-th
      u64 key = 0ull;
      for (int i = 0; i < beams; ++i) {
        u64 k = head[0];
#pragma unroll
        for (int q = 1; q < LISTS; ++q) k = head[q] > k ? head[q] : k;
        const u64 b = warp_max(k);
        if (b == 0ull) break;
        if (lane == i) key = b;
#pragma unroll
        for (int q = 0; q < LISTS; ++q)
          if (head[q] == b)
            head[q] = ++at[q] < beams && pass != 0 ? keys[(lane + 32 * q) * beams + at[q]] : 0ull;
      }
      score[w][lane] = key ? score_of(r, key_logit(key)) : 0ull;
      token[w][lane] = key_token(key);
    }
    __syncthreads();
    if (warp == 0) {
      // lane w: beam w's list, best first
      const bool in = lane < beams;
      const u64 end = in ? score_of(stats[lane], stats[lane].end) : 0ull;
      int at = 0, larger = 0;                                  // larger: continuations that beat this beam's end
      u64 head = in ? score[lane][0] : 0ull, slot_score = 0ull;
      int found = 0;
      for (; found < beams; ++found) {
        const u64 b = warp_max(head);
        if (b == 0ull) break;
        larger += b > end;
        if (lane == found) slot_score = b;
        // of equal ones the lowest beam
        if (lane == __ffs(__ballot_sync(0xFFFFFFFFu, head == b)) - 1) {
          place[found] = lane * 32 + at;
          head = ++at < beams ? score[lane][at] : 0ull;
        }
      }
      __syncwarp();
      const int slot_beam = lane < found ? place[lane] >> 5 : -1;
      const uint32_t slot_token = lane < found ? token[slot_beam][place[lane] & 31] : 0u;
      if (a.ended) {
        for (int i = 0; i < beams; ++i) larger += __shfl_sync(0xFFFFFFFFu, end, i) > end;
        if (in && pass != 0)
          a.ended[row0 + lane] = end != 0ull && larger < beams ? key_score(end) : kMinusInf;
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
      if (in && pass != 0) {
        const int to = row0 + slot;
        a.tokens[to] = slot_beam >= 0 ? (int32_t)slot_token : -1;
        a.parents[to] = slot_beam;
        a.scores_out[to] = slot_beam >= 0 ? key_score(slot_score) : kMinusInf;
      }
    }
    __syncthreads();
  }
}

template <typename T> cudaError_t launch_t(const BeamSelectArgs& a, cudaStream_t s) {
  const bool aligned = a.n % Group<T>::kN == 0 && reinterpret_cast<uintptr_t>(a.logits) % 16 == 0;
  auto part = aligned ? beam_part_kernel<T, true> : beam_part_kernel<T, false>;
  static LargestPerDevice limits[2];
  cudaError_t e = allow_smem(limits[aligned], part, kRing);
  if (e != cudaSuccess) return e;
  const int jobs = a.batch * a.beams * a.parts;
  e = launch_pdl(part, dim3((unsigned)(jobs < kBlocks ? jobs : kBlocks)), dim3(kThreads), kRing, s, a);
  if (e != cudaSuccess) return e;
  note_launch();
  const size_t lists = (size_t)a.beams * a.parts * a.beams;
  e = launch_pdl(a.parts <= 32   ? beam_join_kernel<T, 1>
                 : a.parts <= 64 ? beam_join_kernel<T, 2> : beam_join_kernel<T, kMaxLists>,
                 dim3((unsigned)a.batch), dim3(32u * (unsigned)a.beams), lists <= kStaged ? lists * 8 : 0,
                 s, a);
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace

// Parts of at most kTops chunks a warp.  A block's time is that of its chunks and
// of each part's end, which costs about two chunks; of the ways to cut rows the
// one is taken whose longest block is done first.
BeamParts beam_parts(int64_t rows, int64_t n, int dtype) {
  const int64_t chunk = 32 * kVecs * (dtype == WQL_F32 ? 4 : 8), steps = ((n + chunk - 1) / chunk + kWarps - 1) / kWarps;
  int64_t best = 0, best_cost = 0;
  for (int64_t parts = (steps + kTops - 1) / kTops; parts <= steps && parts <= 32 * kMaxLists; ++parts) {
    const int64_t each = (steps + parts - 1) / parts;
    const int64_t cost = (rows * parts + kBlocks - 1) / kBlocks * (each + 2);
    if (best == 0 || cost < best_cost) best = parts, best_cost = cost;
  }
  const int64_t each = (steps + best - 1) / best;
  return {(int)((steps + each - 1) / each), (int)each * kWarps};
}

cudaError_t launch_beam_select(const BeamSelectArgs& a, cudaStream_t s) {
  switch (a.dtype) {
    case WQL_F32: return launch_t<float>(a, s);
    case WQL_F16: return launch_t<__half>(a, s);
    default: return launch_t<__nv_bfloat16>(a, s);
  }
}

}  // namespace wql
