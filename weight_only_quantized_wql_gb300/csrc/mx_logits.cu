// mx_logits.cu -- logits of a microscaled head: X (e4m3 or e2m1) times W^T
// (e2m1), both in blocks of 32 columns with power-of-two scales.
//
// The block-scaled tensor-core instructions take codes and scales as they are
// stored, so nothing is dequantised: the kernel is a stream of the weight
// through shared memory, bound by HBM (n*k*17/32 bytes of weight, 2*m*n of
// logits) up to several hundred tokens.
//
// Design (sm_103a, one persistent CTA per SM):
//  * Swap AB: a 128-row vocab tile is the MMA M dimension, the tokens (padded
//    to a multiple of 16, at most 256 at a time, 128 for e4m3) are N; fp32
//    accumulators in tensor memory, two when they fit, so a tile's epilogue
//    overlaps the next tile's products.
//  * A stage holds 256 columns of a vocab tile and of the tokens, and both sets
//    of scales.  e2m1 x e2m1 (kind::mxf4, 64 columns per instruction): all of
//    it as stored.  e2m1 x e4m3 (kind::mxf8f6f4, 32 columns): the tensor core
//    wants 16 e2m1 codes (8 bytes) at the start of each 16-byte unit; TMA
//    spreads them so when rows are whole 128-column blocks, else four warps
//    copy 8-byte pieces into that layout with cp.async.  (Stages of 128
//    columns would free their slots sooner, but took 168 us where 256 took
//    119, now 108, one e4m3 token on the 248320 x 5120 head: more copies to
//    issue.)
//  * One warp issues: tcgen05.cp spreads a stage's scales over tensor memory
//    (the stored tiles are in the order it wants), then the stage's products;
//    both run in issue order.
//  * Eight warps read the accumulators, add the bias, round, and store through
//    shared memory by TMA, whole 256-byte runs of a token's logits: 32.0 us
//    for 256 tokens on 151936 x 1024, 48 us straight from registers (which few
//    tokens, and rows that are not 16-byte aligned, still do).
//  * More than 128 tokens, when 128 of them fit shared memory next to a ring
//    of 64 KB of weight: they stay there for the whole launch, and CTAs take
//    slices of 128 in turn over the same vocab tiles, so the weight comes from
//    HBM about once (256 tokens, 151936 x 1024, e2m1: 32.0 us, 38.8 us with
//    256 tokens re-read per tile).  Longer rows re-read the tokens from L2 for
//    every tile, up to 256 (e4m3: 128) at a time.
//  * The weight and the tokens have a producing thread each: one thread for
//    both was the limit where a stage takes more copies.
//  * While the kernel before it still runs, the weight's first stages are
//    prefetched into L2 (one token on 151936 x 1024, e2m1: 18.0 us, 18.6
//    without; more than four stages ahead crowd the first real copies).
//  * Measured, the tokens' quantisation included (as in the figures above):
//    one token 12.2 us of bytes in 18.1 us on 151936 x 1024 (17.1 us alone), 90 to
//    94 % of the measured copy rate on 248320 x 5120 up to 32 tokens, 2490 TFLOP/s
//    at 256 tokens (e2m1, K = 1024) and 4080 TFLOP/s (K = 5120).
//  * Every wait is bounded; on a timeout the CTA records it, drains its own
//    copies and products, frees its tensor memory and returns.
#include "mx.cuh"
#include "ring.cuh"
#include "sm100.cuh"

namespace wql {
namespace {

constexpr int kTileRows = 128;
constexpr int kBlockBytes = kTileRows * 128;       // 128 rows x 128 bytes, 128B-swizzled
constexpr int kCols = 256;                         // columns of a stage
constexpr int kTiles = kCols / 128;                // scale tiles along them
constexpr int kScaleBytes = kTiles * kMxTileBytes;
constexpr int kCodeBytes = kTileRows * kCols / 2;  // of the weight, in HBM
constexpr int kProducerWarp = 0, kMmaWarp = 1, kEpilogueWarp0 = 2, kEpilogueWarps = 8;
constexpr int kTokenWarp = kEpilogueWarp0 + kEpilogueWarps;
constexpr int kCopyWarp0 = kTokenWarp + 1, kCopyWarps = 4;
constexpr int kAheadStages = 4;                    // of the weight, prefetched into L2
constexpr int kMaxResident = 24;                   // stages' worth of tokens that may stay
constexpr int kMaxCopyDepth = 3;                   // stages of copies in flight per copying thread
constexpr int kMaxStages = 12, kMinStages = 2;
constexpr int kResidentBytes = 64 * 1024;          // a ring for that much weight, or the tokens do not stay
constexpr int kOutTokens = 16;                     // tokens of one store
constexpr int kOutBytes = kOutTokens * kTileRows * 2;
constexpr uint32_t kBarBytes = 512;
constexpr uint32_t kErrWait = 8u;                  // error word: a wait ran out

// COPY: the weight by cp.async (e2m1 x e4m3 only), else by TMA.
template <int XFMT, bool COPY> struct Kind {
  static constexpr bool kFp8 = XFMT == WQL_MX_FP8;
  static constexpr bool kCopy = COPY;
  static constexpr int kBlocks = kFp8 ? 2 : 1;          // 128-byte blocks per row and stage
  static constexpr int kMmaCols = kFp8 ? 32 : 64;
  static constexpr int kMmas = kCols / kMmaCols;        // products of a stage
  static constexpr int kWarps = kCopyWarp0 + (COPY ? kCopyWarps : 0);
};

struct MxParams {
  MxLogitsArgs a;
  int tiles;            // ceil(n / 128)
  int tile_cols;        // scale tiles along k
  int stages_k;         // stages per vocab tile
  int slices;           // token slices
  int slice;            // tokens of a slice (the last may have fewer): at most 256; a multiple
                        // of 128, a scale tile, when there are several
  int x_resident;       // the slice's tokens stay in shared memory for the whole launch
  int tma_store;        // logits rows are 16-byte aligned: stored by TMA
  int npad;             // tokens of the largest slice, padded to 16
  int xtiles;           // scale tiles of a slice's tokens: 1 or 2
  int acc_bufs;
  int ring;             // stages in shared memory
  int copy_depth;       // 1..kMaxCopyDepth, below ring: a stage's copies are handed on that
                        // many stages later, and its slot cannot be reused before
  uint32_t tmem_cols;
  uint32_t stage_bytes, off_x, off_ws, off_xs, off_bar;
  uint32_t off_res, res_bytes;     // resident tokens: stages_k parts of res_bytes
  uint32_t off_out;                // staging of the stores
  int out_bufs;                    // buffers of each epilogue group
  long long wait_budget;
  int diag_stall;                  // diagnostics: the issuing warp first waits on a barrier
                                   // nothing arrives on (the timeout path runs)
};

// 3-D tiled TMA load of one box.
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

// The same boxes, and a stretch of bytes, into L2 only.
__device__ __forceinline__ void prefetch_3d(const CUtensorMap* map, int x, int y, int z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(map),
               "r"(x), "r"(y), "r"(z)
               : "memory");
}
__device__ __forceinline__ void prefetch_2d(const CUtensorMap* map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(map),
               "r"(x), "r"(y)
               : "memory");
}
__device__ __forceinline__ void prefetch_bytes(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr) {
  // K-major rows of 128 bytes, 8-row groups 1024 bytes apart, 128-byte swizzle
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)1u << 16) |
         ((uint64_t)(1024u >> 4) << 32) | ((uint64_t)1u << 46) | ((uint64_t)2u << 61);
}
__device__ __forceinline__ uint64_t desc_scales(uint32_t addr) {
  // 32 rows of 16 bytes, 8-row groups 128 bytes apart, no swizzle
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(128u >> 4) << 32) | ((uint64_t)1u << 46);
}

// One 512-byte scale tile to four tensor-memory columns, in all four lane quarters.
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc)
               : "memory");
}

// Instruction descriptor: A = W e2m1, B = X, fp32 accumulator, M = 128, scales
// e8m0; both operands' scale byte in its 32-bit word is added as a multiple of
// kIdescScale.
constexpr uint32_t kIdescScale = (1u << 4) | (1u << 29);
template <int XFMT> __device__ __forceinline__ uint32_t idesc(int n) {
  const uint32_t atype = XFMT == WQL_MX_FP8 ? 5u : 1u, btype = XFMT == WQL_MX_FP8 ? 0u : 1u;
  return (atype << 7) | (btype << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) |
         ((uint32_t)(kTileRows >> 7) << 27);
}

template <int XFMT>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t sa,
                                    uint32_t sb, uint32_t accumulate) {
  if constexpr (XFMT == WQL_MX_FP8) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, "
        "[%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, "
        "[%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
  }
}

__device__ __forceinline__ bool elect_one() {
  uint32_t pred;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(pred));
  return pred != 0u;
}
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tmem_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_load16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// Barrier of an epilogue group's four warps, and whether any thread says yes.
__device__ __forceinline__ void group_sync(int group) {
  asm volatile("bar.sync %0, 128;" ::"r"(group + 1) : "memory");
}
__device__ __forceinline__ bool group_any(int group, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(group + 1), "r"((uint32_t)v)
      : "memory");
  return r != 0u;
}

__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;"); }
template <int N> __device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int XFMT, bool COPY, typename OT>
__global__ void __launch_bounds__(Kind<XFMT, COPY>::kWarps * 32, 1)
    mx_logits_kernel(const __grid_constant__ CUtensorMap tw, const __grid_constant__ CUtensorMap tx,
                     const __grid_constant__ CUtensorMap to, const MxParams p) {
  using K = Kind<XFMT, COPY>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base - raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + p.off_bar);
  uint64_t* empty = full + kMaxStages;
  uint64_t* acc_full = empty + kMaxStages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* x_full = acc_empty + 2;
  uint64_t* drain = x_full + kMaxResident;
  uint64_t* stall = drain + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(stall + 1);
  unsigned int* failed = tmem_slot + 1;

  const MxLogitsArgs& a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int slice = blockIdx.x % p.slices;
  const int team = blockIdx.x / p.slices, teams = gridDim.x / p.slices;
  const int t0 = (int)((long long)p.tiles * team / teams);
  const int t1 = (int)((long long)p.tiles * (team + 1) / teams);
  const int tokens = min(p.slice, a.m - slice * p.slice);
  const int ntok = (tokens + 15) & ~15;              // this slice's N
  const int steps = (t1 - t0) * p.stages_k;          // ring fills of this CTA

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.ring; ++s) {
      mbar_init(&full[s], (p.x_resident ? 1 : 2) + (COPY ? kCopyWarps : 0));
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&acc_full[s], 1);
      mbar_init(&acc_empty[s], kEpilogueWarps);
    }
    for (int c = 0; c < kMaxResident; ++c) mbar_init(&x_full[c], 1);
    mbar_init(drain, 1);
    mbar_init(stall, 1);
    *failed = 0u;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(p.tmem_cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // The kernel before this one (it may be writing X) is still running: bring
  // the weight's first stages into L2 meanwhile, where a write of it would
  // still be seen.
  if (!COPY && warp == kProducerWarp && lane == 0) {
    prefetch_tmap(&tw);
    for (int i = 0; i < min(steps, kAheadStages); ++i) {
      const int t = t0 + i / p.stages_k, c = i % p.stages_k;
      if constexpr (K::kFp8)
        prefetch_3d(&tw, 0, t * kTileRows, c * K::kBlocks);
      else
        prefetch_2d(&tw, c * 32, t * kTileRows);
      prefetch_bytes(reinterpret_cast<const uint8_t*>(a.w_scales) +
                         ((size_t)t * p.tile_cols + c * kTiles) * kMxTileBytes,
                     (uint32_t)(min(kTiles, p.tile_cols - c * kTiles) * kMxTileBytes));
    }
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  griddep_launch_dependents();
  griddep_wait();
  const uint32_t tmem = *tmem_slot;
  bool bad = false;
  // Every copy that a thread has issued lands before the CTA can finish.  Each
  // producing thread waits for its own: when one of them gives up the other may
  // get further, and nobody else waits for those copies.  (The arrivals of a
  // role that gave up are missing, and this runs out too: one budget in all.)
  auto drain_fills = [&](int fills) {
    const long long since = clock64();
    return drain_ring(fills, p.ring, [&](int s, uint32_t parity) {
      return mbar_wait_since(&full[s], parity, since);
    });
  };

  if (warp == kProducerWarp) {
    // ---------------- TMA: the weight and its scales ----------------
    if (lane == 0) {
      const uint8_t* wsc = reinterpret_cast<const uint8_t*>(a.w_scales);
      int fills = 0, slot = 0;
      uint32_t phase = 0;
      for (int t = t0; t < t1 && !bad; ++t)
        for (int c = 0; c < p.stages_k && !bad; ++c) {
          if (fills >= p.ring) bad = !mbar_wait(&empty[slot], phase ^ 1u, p.wait_budget);
          if (bad) break;
          uint8_t* st = sm + slot * p.stage_bytes;
          const uint32_t sbytes = (uint32_t)(min(kTiles, p.tile_cols - c * kTiles) * kMxTileBytes);
          mbar_arrive_expect_tx(&full[slot], sbytes + (COPY ? 0u : (uint32_t)kCodeBytes));
          if constexpr (!COPY) {
            if constexpr (K::kFp8)
              tma_load_3d(st, &tw, 0, t * kTileRows, c * K::kBlocks, &full[slot]);
            else
              tma_load_2d(st, &tw, c * 32, t * kTileRows, &full[slot]);
          }
          bulk_load(st + p.off_ws, wsc + ((size_t)t * p.tile_cols + c * kTiles) * kMxTileBytes,
                    sbytes, &full[slot]);
          ++fills;
          if (++slot == p.ring) { slot = 0; phase ^= 1u; }
        }
      bad = !drain_fills(fills) || bad;
    }
  } else if (warp == kTokenWarp) {
    // ---------------- TMA: the tokens and their scales ----------------
    if (lane == 0) {
      prefetch_tmap(&tx);
      const uint8_t* xsc = reinterpret_cast<const uint8_t*>(a.x_scales);
      const int xt = (tokens + 127) / 128;           // this slice's token scale tiles
      const uint32_t x_bytes = (uint32_t)(K::kBlocks * p.npad * 128);
      auto load = [&](int c, uint8_t* codes, uint8_t* scales, uint64_t* bar) {
        const uint32_t sbytes = (uint32_t)(min(kTiles, p.tile_cols - c * kTiles) * kMxTileBytes);
        mbar_arrive_expect_tx(bar, x_bytes + sbytes * xt);
        if constexpr (K::kFp8 && !COPY) {
          tma_load_3d(codes, &tx, 0, slice * p.slice, c * K::kBlocks, bar);
        } else {
          for (int b = 0; b < K::kBlocks; ++b)
            tma_load_2d(codes + b * p.npad * 128, &tx, (c * K::kBlocks + b) * 32, slice * p.slice,
                        bar);
        }
        for (int x = 0; x < xt; ++x)
          bulk_load(scales + x * kScaleBytes,
                    xsc + ((size_t)(slice * (p.slice / 128) + x) * p.tile_cols + c * kTiles) *
                              kMxTileBytes,
                    sbytes, bar);
      };
      if (p.x_resident) {
        for (int c = 0; c < p.stages_k && steps > 0; ++c) {
          uint8_t* part = sm + p.off_res + c * p.res_bytes;
          load(c, part, part + x_bytes, &x_full[c]);
        }
        for (int c = 0; c < p.stages_k && steps > 0; ++c)
          if (!mbar_wait(&x_full[c], 0u)) bad = true;
      } else {
        int slot = 0, c = 0, fills = 0;
        uint32_t phase = 0;
        for (; fills < steps; ++fills) {
          if (fills >= p.ring) bad = !mbar_wait(&empty[slot], phase ^ 1u, p.wait_budget);
          if (bad) break;
          uint8_t* st = sm + slot * p.stage_bytes;
          load(c, st + p.off_x, st + p.off_xs, &full[slot]);
          if (++slot == p.ring) { slot = 0; phase ^= 1u; }
          if (++c == p.stages_k) c = 0;
        }
        bad = !drain_fills(fills) || bad;
      }
    }
  } else if (warp == kMmaWarp) {
    // ---------------- tensor cores ----------------
    // The whole warp runs the loop, so that descriptors and addresses are
    // warp-uniform values, made from their first ones by additions (the
    // start-address fields count 16-byte units and never carry); one elected
    // lane issues.  Computed by that lane alone, they took 6 % more time for
    // one token on the 248320 x 5120 head.
    const bool leader = elect_one();
    const uint32_t sf0 = tmem + (uint32_t)(p.acc_bufs * p.npad);
    const uint32_t xcols = 4u * (uint32_t)p.xtiles;          // columns of a scale tile of X
    const uint32_t sf_set = (uint32_t)kTiles * (4u + xcols);
    const uint32_t id0 = idesc<XFMT>(ntok);
    const uint32_t x0 = base + (p.x_resident ? p.off_res : p.off_x);
    const uint32_t x_block = (uint32_t)p.npad * 128u;
    const uint32_t xs0 = base + (p.x_resident ? p.off_res + K::kBlocks * x_block : p.off_xs);
    const uint64_t aw0 = desc_sw128(base), bx0 = desc_sw128(x0);
    const uint64_t sw0 = desc_scales(base + p.off_ws), sx0 = desc_scales(xs0);
    const uint32_t stage16 = p.stage_bytes >> 4, res16 = p.res_bytes >> 4;
    const int last_cols = a.k - (p.stages_k - 1) * kCols;
    const int last_mmas = (last_cols + K::kMmaCols - 1) / K::kMmaCols;
    int slot = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0, set = 0;
    bool issued = false;
    if (p.diag_stall) bad = !mbar_wait(stall, 0u, p.wait_budget);
    for (int t = t0; t < t1; ++t) {
      if (!bad && t - t0 >= p.acc_bufs) bad = !mbar_wait(&acc_empty[acc], acc_phase ^ 1u, p.wait_budget);
      if (__any_sync(0xFFFFFFFFu, bad)) { bad = true; break; }
      tmem_fence_after();
      const uint32_t d = tmem + (uint32_t)(acc * p.npad);
      for (int c = 0; c < p.stages_k; ++c) {
        if (p.x_resident && t == t0) bad = !mbar_wait(&x_full[c], 0u, p.wait_budget);
        bad = bad || !mbar_wait(&full[slot], phase, p.wait_budget);
        if (__any_sync(0xFFFFFFFFu, bad)) { bad = true; break; }
        tmem_fence_after();
        const uint32_t at = (uint32_t)slot * stage16;
        const uint32_t xat = p.x_resident ? (uint32_t)c * res16 : at;
        const uint64_t aw = aw0 + at, bx = bx0 + xat, sw = sw0 + at, sx = sx0 + xat;
        const uint32_t sfw = sf0 + set, sfx = sfw + 4u * kTiles;
        const int mmas = c + 1 < p.stages_k ? K::kMmas : last_mmas;
        const uint32_t more = c != 0 ? 1u : 0u;
        if (leader) {
          // (a scale tile past the row's end is copied too, and not used)
#pragma unroll
          for (int kt = 0; kt < kTiles; ++kt) {
            copy_scales(sfw + 4u * kt, sw + (uint64_t)(kt * (kMxTileBytes >> 4)));
            copy_scales(sfx + xcols * kt, sx + (uint64_t)(kt * (kMxTileBytes >> 4)));
            if (p.xtiles > 1)
              copy_scales(sfx + xcols * kt + 4u,
                          sx + (uint64_t)((kScaleBytes + kt * kMxTileBytes) >> 4));
          }
#pragma unroll
          for (int j = 0; j < K::kMmas; ++j) {
            constexpr int kPerTile = K::kMmas / kTiles;
            const int kt = j / kPerTile, in = j % kPerTile;
            const uint64_t ao = K::kFp8 ? (uint64_t)(kt * (kBlockBytes >> 4) + in * 2) : j * 2u;
            const uint64_t bo = K::kFp8 ? (uint64_t)(kt * (x_block >> 4) + in * 2u) : j * 2u;
            if (j < mmas)
              mma<XFMT>(d, aw + ao, bx + bo,
                        id0 + (uint32_t)(K::kFp8 ? in : in * 2) * kIdescScale, sfw + 4u * kt,
                        sfx + xcols * kt, j == 0 ? more : 1u);
          }
          commit(&empty[slot]);
        }
        issued = true;
        __syncwarp();
        set = sf_set - set;
        if (++slot == p.ring) { slot = 0; phase ^= 1u; }
      }
      if (bad) break;
      if (leader) commit(&acc_full[acc]);
      __syncwarp();
      if (++acc == p.acc_bufs) { acc = 0; acc_phase ^= 1u; }
    }
    if (bad && issued) {
      // the products already issued finish before tensor memory is freed
      if (leader) commit(drain);
      __syncwarp();
      mbar_wait(drain, 0u);
    }
  } else if (warp < kTokenWarp) {
    // ---------------- epilogue: lanes are vocab rows, columns tokens ----------------
    // Two groups of four warps (one per lane quarter) take 16 tokens in turn.
    const int quarter = warp & 3, group = (warp - kEpilogueWarp0) >> 2;
    const int r = quarter * 32 + lane;                // row of the tile
    uint8_t* staging = sm + p.off_out + group * p.out_bufs * kOutBytes;
    int buf = 0;
    int acc = 0;
    uint32_t acc_phase = 0;
    OT* out = reinterpret_cast<OT*>(a.out) + (size_t)slice * p.slice * a.n;
    for (int t = t0; t < t1; ++t) {
      // (a group's warps give up together, so that none waits at the barriers below)
      bad = !mbar_wait(&acc_full[acc], acc_phase, p.wait_budget);
      if (p.tma_store) {
        bad = group_any(group, bad);
      } else {
        bad = __any_sync(0xFFFFFFFFu, bad);
      }
      if (bad) break;
      tmem_fence_after();
      const int row = t * kTileRows + r;
      const float b = (a.bias && row < a.n) ? to_f32(reinterpret_cast<const OT*>(a.bias)[row]) : 0.f;
      const uint32_t src = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc * p.npad);
      for (int c = group * kOutTokens; c < ntok; c += 2 * kOutTokens) {
        uint32_t v[16];
        tmem_load16(src + (uint32_t)c, v);
        if (c + 2 * kOutTokens >= ntok) {             // this warp's last columns of the tile
          tmem_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&acc_empty[acc]);
        }
        if (p.tma_store) {
          // [16 tokens][128 rows] through shared memory, whole 256-byte runs out
          OT* st = reinterpret_cast<OT*>(staging + buf * kOutBytes);
          if (quarter == 0 && lane == 0) {            // this buffer is free again
            if (p.out_bufs == 2)
              asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
            else
              asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          }
          group_sync(group);
#pragma unroll
          for (int j = 0; j < 16; ++j)
            st[j * kTileRows + r] = from_f32<OT>(__uint_as_float(v[j]) + b);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          group_sync(group);
          if (quarter == 0 && lane == 0) {
            asm volatile(
                "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::
                    "l"(&to),
                "r"(t * kTileRows), "r"(slice * p.slice + c), "r"(smem_u32(st))
                : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          }
          buf = p.out_bufs - 1 - buf;
        } else if (row < a.n) {
          OT* dst = out + (size_t)c * a.n + row;
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (c + j < tokens) dst[(size_t)j * a.n] = from_f32<OT>(__uint_as_float(v[j]) + b);
        }
      }
      if (group * kOutTokens >= ntok) {               // no columns for this group
        if (lane == 0) mbar_arrive(&acc_empty[acc]);
      }
      if (++acc == p.acc_bufs) { acc = 0; acc_phase ^= 1u; }
    }
    if (p.tma_store && quarter == 0 && lane == 0)
      asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  } else if constexpr (COPY) {
    // ---------------- the weight's codes, 8 bytes to each 16-byte unit ----------------
    const int id = (warp - kCopyWarp0) * 32 + lane;          // 0..127
    const int piece = id & 15, r0 = id >> 4;                 // 16 pieces of 16 codes; rows r0 + 8 i
    const uint32_t unit = (uint32_t)((piece >> 3) * kBlockBytes + r0 * 128 +
                                     (((piece & 7) ^ (r0 & 7)) * 16));
    const size_t pitch = (size_t)a.k / 2;
    const uint8_t* w = reinterpret_cast<const uint8_t*>(a.w_codes);
    int slot = 0, handed_slot = 0, issued = 0, handed = 0;
    uint32_t phase = 0;
    auto hand_on = [&] {
      // the tensor core reads through the async proxy
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[handed_slot]);
      if (++handed_slot == p.ring) handed_slot = 0;
      ++handed;
    };
    int t = t0, c = 0;
    for (; issued < steps; ++issued) {
      if (issued >= p.ring) bad = !mbar_wait(&empty[slot], phase ^ 1u, p.wait_budget);
      bad = __any_sync(0xFFFFFFFFu, bad);
      if (bad) break;
      const int col = c * kCols + piece * 16;
      if (col < a.k) {
        const uint32_t dst = base + (uint32_t)slot * p.stage_bytes + unit;
        const uint8_t* src = w + col / 2;
#pragma unroll
        for (int r = 0; r < kTileRows; r += 8)
          // rows past the last repeat it; their logits are not stored
          cp_async8(dst + r * 128, src + (size_t)min(t * kTileRows + r0 + r, a.n - 1) * pitch);
      }
      cp_async_commit();
      if (++slot == p.ring) { slot = 0; phase ^= 1u; }
      if (++c == p.stages_k) { c = 0; ++t; }
      if (issued >= p.copy_depth) {
        if (p.copy_depth == 3)
          cp_async_wait<3>();
        else if (p.copy_depth == 2)
          cp_async_wait<2>();
        else
          cp_async_wait<1>();
        hand_on();
      }
    }
    cp_async_wait<0>();
    while (handed < issued) hand_on();
  }

  if (bad) atomicOr(failed, 1u);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(p.tmem_cols)
                 : "memory");
  if (threadIdx.x == 0 && *failed != 0u && a.err) atomicOr(a.err, kErrWait);
}

constexpr uint32_t rup1k(uint32_t v) { return (v + 1023u) & ~1023u; }

// Lays out a launch with slices of at most `most` tokens; false when fewer
// than kMinStages stages fit.
template <typename K> bool plan(MxParams& p, int most) {
  const int m = p.a.m;
  // cp.async fetches through the L1 that shares the SM's memory: with 227 KB
  // taken, 64 tokens on a 151936 x 992 head took 43.0 us, with 192 KB 30.9
  const uint32_t room = (K::kCopy ? 192u : 227u) * 1024u - 1024u - kBarBytes -
                        (uint32_t)(2 * p.out_bufs * kOutBytes);
  auto lay = [&](int slice, bool resident) {
    p.slice = slice;
    p.slices = (m + slice - 1) / slice;
    p.npad = ((m < slice ? m : slice) + 15) / 16 * 16;
    p.xtiles = (p.npad + 127) / 128;
    p.x_resident = resident;
    const uint32_t x_bytes = (uint32_t)(K::kBlocks * p.npad * 128);
    const uint32_t xs_bytes = rup1k((uint32_t)(p.xtiles * kScaleBytes));
    // a stage: weight, tokens, their scales; every part a multiple of 1024 bytes
    p.off_x = K::kBlocks * kBlockBytes;
    p.off_ws = p.off_x + (resident ? 0u : x_bytes);
    p.off_xs = p.off_ws + kScaleBytes;
    p.stage_bytes = rup1k(p.off_xs + (resident ? 0u : (uint32_t)(p.xtiles * kScaleBytes)));
    p.res_bytes = x_bytes + xs_bytes;
    const uint64_t held = resident ? (uint64_t)p.stages_k * p.res_bytes : 0u;
    if (held >= room || (resident && p.stages_k > kMaxResident)) return 0;
    const int fit = (int)((room - (uint32_t)held) / p.stage_bytes);
    return fit < kMaxStages ? fit : kMaxStages;
  };
  p.ring = 0;
  if (m > 128) p.ring = lay(128, true);
  if (p.ring < kResidentBytes / kCodeBytes) p.ring = lay(most, false);
  if (p.ring < kMinStages) return false;
  const uint32_t scale_cols = 2u * (uint32_t)kTiles * (4u + 4u * (uint32_t)p.xtiles);
  p.acc_bufs = 2u * (uint32_t)p.npad + scale_cols <= 512u ? 2 : 1;
  p.tmem_cols = 32;
  while (p.tmem_cols < (uint32_t)(p.acc_bufs * p.npad) + scale_cols) p.tmem_cols <<= 1;
  p.copy_depth = p.ring - 1 < kMaxCopyDepth ? p.ring - 1 : kMaxCopyDepth;
  p.off_res = (uint32_t)p.ring * p.stage_bytes;
  p.off_out = p.off_res + (p.x_resident ? (uint32_t)p.stages_k * p.res_bytes : 0u);
  p.off_bar = p.off_out + (uint32_t)(2 * p.out_bufs * kOutBytes);
  return true;
}

template <int XFMT, bool COPY, typename OT>
cudaError_t launch_t(const MxLogitsArgs& a, cudaStream_t s) {
  using K = Kind<XFMT, COPY>;
  MxParams p{};
  p.a = a;
  p.wait_budget = diag_wait_budget();
  p.diag_stall = diag_stall_mma();
  p.tiles = (a.n + kTileRows - 1) / kTileRows;
  p.tile_cols = (int)mx_tile_cols(a.k);
  p.stages_k = (a.k + kCols - 1) / kCols;
  // few tokens: 64-byte stores straight from registers (copying the weight, they
  // leave room for a fifth stage); up to two groups of 16, one block per group
  // and tile, need one buffer each
  p.tma_store = a.m > (COPY ? 32 : 8) && a.n % 8 == 0 && reinterpret_cast<uintptr_t>(a.out) % 16 == 0;
  p.out_bufs = !p.tma_store ? 0 : a.m <= 2 * kOutTokens ? 1 : 2;
  if (!plan<K>(p, K::kFp8 ? 128 : 256)) return cudaErrorInvalidConfiguration;
  const size_t smem = p.off_bar + kBarBytes + 1024;

  CUtensorMap tw, tx, to;
  const uint64_t wrow = (uint64_t)a.k / 2, xrow = K::kFp8 ? (uint64_t)a.k : (uint64_t)a.k / 2;
  cudaError_t e;
  if (K::kFp8 && !COPY) {
    e = make_tmap_blocks(&tw, true, a.w_codes, wrow, (uint64_t)a.n, kTileRows, K::kBlocks);
    if (e != cudaSuccess) return e;
    e = make_tmap_blocks(&tx, false, a.x_codes, xrow, (uint64_t)a.m, (uint32_t)p.npad, K::kBlocks);
  } else {
    e = make_tmap_2d(&tw, a.w_codes, 4, wrow / 4, (uint64_t)a.n, wrow, 32, kTileRows,
                     Swizzle::k128B);
    if (e != cudaSuccess) return e;
    e = make_tmap_2d(&tx, a.x_codes, 4, xrow / 4, (uint64_t)a.m, xrow, 32, (uint32_t)p.npad,
                     Swizzle::k128B);
  }
  if (e != cudaSuccess) return e;
  to = tx;
  if (p.tma_store) {
    e = make_tmap_2d(&to, a.out, 2, (uint64_t)a.n, (uint64_t)a.m, (uint64_t)a.n * 2, kTileRows,
                     kOutTokens, Swizzle::kNone);
    if (e != cudaSuccess) return e;
  }
  auto kern = mx_logits_kernel<XFMT, COPY, OT>;
  static LargestPerDevice limit;
  e = allow_smem(limit, kern, smem);
  if (e != cudaSuccess) return e;
  int teams = device_sm_count() / p.slices;
  if (teams < 1) teams = 1;
  if (teams > p.tiles) teams = p.tiles;
  e = launch_pdl(kern, dim3((unsigned)(teams * p.slices)), dim3(K::kWarps * 32), smem, s, tw, tx, to, p);
  note_launch();
  return e;
}

}  // namespace

cudaError_t launch_mx_logits(const MxLogitsArgs& a, cudaStream_t s) {
  const bool f16 = a.out_dtype == WQL_F16;
  if (a.x_format == WQL_MX_FP4)
    return f16 ? launch_t<WQL_MX_FP4, false, __half>(a, s)
               : launch_t<WQL_MX_FP4, false, __nv_bfloat16>(a, s);
  // TMA spreads e2m1 codes over 16-byte units itself, for whole 128-column
  // blocks and 32-byte aligned codes: 32 tokens on the 248320 x 5120 head take
  // 113 us so, 190 us with cp.async
  if (a.k % 128 == 0 && reinterpret_cast<uintptr_t>(a.w_codes) % 32 == 0)
    return f16 ? launch_t<WQL_MX_FP8, false, __half>(a, s)
               : launch_t<WQL_MX_FP8, false, __nv_bfloat16>(a, s);
  return f16 ? launch_t<WQL_MX_FP8, true, __half>(a, s)
             : launch_t<WQL_MX_FP8, true, __nv_bfloat16>(a, s);
}

}  // namespace wql
