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
//    to a multiple of 16, at most 256 at a time, 128 for e4m3) are N; fp32 accumulators in
//    tensor memory, two when they fit, so a tile's epilogue overlaps the next
//    tile's products.
//  * A stage holds 256 columns of a vocab tile, of the tokens, and both sets
//    of scales.  e2m1 x e2m1 (kind::mxf4, 64 columns per instruction): all of
//    it comes by TMA.  e2m1 x e4m3 (kind::mxf8f6f4, 32 columns): the tensor
//    core wants 16 e2m1 codes (8 bytes) at the start of each 16-byte unit, so
//    four warps copy the weight's 8-byte pieces with cp.async straight into
//    that layout; X and the scales come by TMA.
//  * One warp issues: tcgen05.cp spreads a stage's scales over tensor memory
//    (the stored tiles are in the order it wants), then the stage's products;
//    both run in issue order.
//  * Eight warps read the accumulators, add the bias, round and store.
//  * More tokens: CTAs take slices of them in turn and run the
//    same vocab tiles side by side, so the weight is read from HBM about once.
//  * Every wait is bounded; on a timeout the CTA records it, drains its own
//    copies and products, frees its tensor memory and returns.
#include "mx.cuh"
#include "sm100.cuh"

namespace wql {
namespace {

constexpr int kTileRows = 128;
constexpr int kStageCols = 256;
constexpr int kBlockBytes = kTileRows * 128;       // 128 rows x 128 bytes, 128B-swizzled
constexpr int kProducerWarp = 0, kMmaWarp = 1, kEpilogueWarp0 = 2, kEpilogueWarps = 8;
constexpr int kCopyWarp0 = kEpilogueWarp0 + kEpilogueWarps, kCopyWarps = 4;
constexpr int kMaxCopyDepth = 3;                   // stages of copies in flight per copying thread
constexpr int kMaxStages = 8, kMinStages = 2;
constexpr uint32_t kErrWait = 8u;                  // error word: a wait ran out

// COPY: the weight by cp.async (e2m1 x e4m3 only), else by TMA.
template <int XFMT, bool COPY> struct Kind {
  static constexpr bool kFp8 = XFMT == WQL_MX_FP8;
  static constexpr int kBlocks = kFp8 ? 2 : 1;          // 128-byte blocks per row and stage
  static constexpr int kMmaCols = kFp8 ? 32 : 64;
  static constexpr int kMmaPerStage = kStageCols / kMmaCols;
  static constexpr int kMmaPerTile = 128 / kMmaCols;    // per scale tile of 128 columns
  static constexpr int kSlice = kFp8 ? 128 : 256;       // most tokens at a time
  // bytes a 128-row block of the weight counts on a barrier: the codes themselves
  static constexpr int kWeightTx = kFp8 ? kTileRows * 64 : kBlockBytes;
  static constexpr int kWarps = kCopyWarp0 + (COPY ? kCopyWarps : 0);
};

struct MxParams {
  MxLogitsArgs a;
  int tiles;            // ceil(n / 128)
  int tile_cols;        // scale tiles along k
  int stages_k;         // stages per vocab tile
  int slices;           // token slices
  int npad;             // tokens of the largest slice, padded to 16
  int xtiles;           // scale tiles of a slice's tokens: 1 or 2
  int acc_bufs;
  int ring;             // stages in shared memory
  int copy_depth;       // 1..kMaxCopyDepth, below ring: a stage's copies are handed on that
                        // many stages later, and its slot cannot be reused before
  uint32_t tmem_cols;
  uint32_t stage_bytes, off_x, off_ws, off_xs, off_bar;
  long long wait_budget;
};

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
// e8m0, `id` the scale's byte in its 32-bit word.
template <int XFMT> __device__ __forceinline__ uint32_t idesc(int n, uint32_t id) {
  const uint32_t atype = XFMT == WQL_MX_FP8 ? 5u : 1u, btype = XFMT == WQL_MX_FP8 ? 0u : 1u;
  return (id << 4) | (atype << 7) | (btype << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) |
         ((uint32_t)(kTileRows >> 7) << 27) | (id << 29);
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
                     const MxParams p) {
  using K = Kind<XFMT, COPY>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base - raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + p.off_bar);
  uint64_t* empty = full + kMaxStages;
  uint64_t* acc_full = empty + kMaxStages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  unsigned int* failed = tmem_slot + 1;

  const MxLogitsArgs& a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int slice = blockIdx.x % p.slices;
  const int team = blockIdx.x / p.slices, teams = gridDim.x / p.slices;
  const int t0 = (int)((long long)p.tiles * team / teams);
  const int t1 = (int)((long long)p.tiles * (team + 1) / teams);
  const int tokens = min(K::kSlice, a.m - slice * K::kSlice);
  const int ntok = (tokens + 15) & ~15;              // this slice's N
  const int steps = (t1 - t0) * p.stages_k;          // ring fills of this CTA

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.ring; ++s) {
      mbar_init(&full[s], 1 + (COPY ? kCopyWarps : 0));
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&acc_full[s], 1);
      mbar_init(&acc_empty[s], kEpilogueWarps);
    }
    mbar_init(drain, 1);
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
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  griddep_launch_dependents();
  griddep_wait();
  const uint32_t tmem = *tmem_slot;
  bool bad = false;

  if (warp == kProducerWarp) {
    // ---------------- TMA: X, scales, and (e2m1 x e2m1) the weight ----------------
    if (lane == 0) {
      prefetch_tmap(&tx);
      if (!COPY) prefetch_tmap(&tw);
      const uint8_t* wsc = reinterpret_cast<const uint8_t*>(a.w_scales);
      const uint8_t* xsc = reinterpret_cast<const uint8_t*>(a.x_scales);
      const int xt = (tokens + 127) / 128;           // this slice's token scale tiles
      int fills = 0, slot = 0;
      uint32_t phase = 0;
      for (int t = t0; t < t1 && !bad; ++t)
        for (int c = 0; c < p.stages_k && !bad; ++c) {
          if (fills >= p.ring) bad = !mbar_wait(&empty[slot], phase ^ 1u, p.wait_budget);
          if (bad) break;
          uint8_t* st = sm + slot * p.stage_bytes;
          const int kt = c * 2, nkt = min(2, p.tile_cols - kt);    // scale tiles of this stage
          const uint32_t sbytes = (uint32_t)(nkt * kMxTileBytes);
          const uint32_t bytes = (uint32_t)(K::kBlocks * p.npad * 128) + sbytes * (1 + xt) +
                                 (COPY ? 0u : (uint32_t)(K::kBlocks * K::kWeightTx));
          mbar_arrive_expect_tx(&full[slot], bytes);
          if (!COPY)
            for (int b = 0; b < K::kBlocks; ++b)      // x in map elements: words, or codes
              tma_load_2d(st + b * kBlockBytes, &tw, (c * K::kBlocks + b) * (K::kFp8 ? 128 : 32),
                          t * kTileRows, &full[slot]);
          for (int b = 0; b < K::kBlocks; ++b)
            tma_load_2d(st + p.off_x + b * p.npad * 128, &tx, (c * K::kBlocks + b) * 32,
                        slice * K::kSlice, &full[slot]);
          bulk_load(st + p.off_ws, wsc + ((size_t)t * p.tile_cols + kt) * kMxTileBytes, sbytes,
                    &full[slot]);
          for (int x = 0; x < xt; ++x)
            bulk_load(st + p.off_xs + x * 2 * kMxTileBytes,
                      xsc + ((size_t)(slice * (K::kSlice / 128) + x) * p.tile_cols + kt) * kMxTileBytes, sbytes,
                      &full[slot]);
          ++fills;
          if (++slot == p.ring) { slot = 0; phase ^= 1u; }
        }
      // every copy issued lands before the CTA can finish; when the copying
      // warps gave up their arrivals are missing, so this can run out too
      for (int s = 0; s < p.ring && s < fills; ++s)
        if (!mbar_wait(&full[s], (uint32_t)(((fills - 1 - s) / p.ring) & 1))) bad = true;
    }
  } else if (warp == kMmaWarp) {
    // ---------------- tensor cores ----------------
    const bool leader = elect_one();
    const uint32_t sf0 = tmem + (uint32_t)(p.acc_bufs * p.npad);
    const uint32_t sf_set = 8u + 8u * (uint32_t)p.xtiles;    // columns: W 2 x 4, X 2 x 4 x xtiles
    const uint32_t xcols = 4u * (uint32_t)p.xtiles;
    int slot = 0, acc = 0, step = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool issued = false;
    for (int t = t0; t < t1; ++t) {
      if (t - t0 >= p.acc_bufs) bad = !mbar_wait(&acc_empty[acc], acc_phase ^ 1u, p.wait_budget);
      if (__any_sync(0xFFFFFFFFu, bad)) { bad = true; break; }
      tmem_fence_after();
      const uint32_t d = tmem + (uint32_t)(acc * p.npad);
      for (int c = 0; c < p.stages_k; ++c, ++step) {
        bad = !mbar_wait(&full[slot], phase, p.wait_budget);
        if (__any_sync(0xFFFFFFFFu, bad)) { bad = true; break; }
        tmem_fence_after();
        if (leader) {
          const uint32_t st = base + (uint32_t)slot * p.stage_bytes;
          const uint32_t sfw = sf0 + (uint32_t)(step & 1) * sf_set, sfx = sfw + 8u;
          const int cols = min(kStageCols, a.k - c * kStageCols);
          const int nkt = (cols + 127) / 128;
          for (int kt = 0; kt < nkt; ++kt) {
            copy_scales(sfw + 4u * kt, desc_scales(st + p.off_ws + kt * kMxTileBytes));
            for (int x = 0; x < p.xtiles; ++x)
              copy_scales(sfx + xcols * kt + 4u * x,
                          desc_scales(st + p.off_xs + (x * 2 + kt) * kMxTileBytes));
          }
          const int products = (cols + K::kMmaCols - 1) / K::kMmaCols;
          const uint64_t aw = desc_sw128(st), bx = desc_sw128(st + p.off_x);
#pragma unroll
          for (int j = 0; j < K::kMmaPerStage; ++j) {
            if (j >= products) break;
            const int kt = j / K::kMmaPerTile, in = j % K::kMmaPerTile;
            const uint64_t ao = K::kFp8 ? (uint64_t)(kt * (kBlockBytes >> 4) + in * 2)
                                        : (uint64_t)(j * 2);
            const uint64_t bo = K::kFp8 ? (uint64_t)(kt * ((p.npad * 128) >> 4) + in * 2)
                                        : (uint64_t)(j * 2);
            mma<XFMT>(d, aw + ao, bx + bo, idesc<XFMT>(ntok, K::kFp8 ? in : in * 2), sfw + 4u * kt,
                      sfx + xcols * kt, (c | j) != 0 ? 1u : 0u);
          }
          commit(&empty[slot]);
        }
        issued = true;
        __syncwarp();
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
  } else if (warp < kCopyWarp0) {
    // ---------------- epilogue: lanes are vocab rows, columns tokens ----------------
    const int quarter = warp & 3, half = (warp - kEpilogueWarp0) >> 2;
    // this warp's token columns: every other group of 16
    int acc = 0;
    uint32_t acc_phase = 0;
    OT* out = reinterpret_cast<OT*>(a.out) + (size_t)slice * K::kSlice * a.n;
    for (int t = t0; t < t1; ++t) {
      bad = bad || !mbar_wait(&acc_full[acc], acc_phase, p.wait_budget);
      bad = __any_sync(0xFFFFFFFFu, bad);
      if (bad) break;
      tmem_fence_after();
      const int row = t * kTileRows + quarter * 32 + lane;
      const float b = (a.bias && row < a.n) ? to_f32(reinterpret_cast<const OT*>(a.bias)[row]) : 0.f;
      const uint32_t src = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc * p.npad);
      for (int c = half * 16; c < ntok; c += 32) {
        uint32_t v[16];
        tmem_load16(src + (uint32_t)c, v);
        if (row < a.n) {
          OT* dst = out + (size_t)c * a.n + row;
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (c + j < tokens) dst[(size_t)j * a.n] = from_f32<OT>(__uint_as_float(v[j]) + b);
        }
      }
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[acc]);
      if (++acc == p.acc_bufs) { acc = 0; acc_phase ^= 1u; }
    }
  } else if constexpr (COPY) {
    // ---------------- the weight's codes, 8 bytes to each 16-byte unit ----------------
    const int id = (warp - kCopyWarp0) * 32 + lane;          // 0..127
    const int piece = id & 15, r0 = id >> 4;                 // 16 pieces of 16 codes; rows r0 + 8 i
    const uint32_t unit = (uint32_t)((piece >> 3) * kBlockBytes + r0 * 128 +
                                     (((piece & 7) ^ (r0 & 7)) * 16));
    const size_t pitch = (size_t)a.k / 2;
    const uint8_t* w = reinterpret_cast<const uint8_t*>(a.w_codes);
    int slot = 0, done_slot = 0;
    uint32_t phase = 0;
    int t = t0, c = 0;
    for (int i = 0; i < steps + p.copy_depth; ++i) {
      if (i < steps) {
        if (i >= p.ring) bad = bad || !mbar_wait(&empty[slot], phase ^ 1u, p.wait_budget);
        bad = __any_sync(0xFFFFFFFFu, bad);
        if (bad) break;
        const int col = c * kStageCols + piece * 16;
        if (col < a.k) {
          const uint32_t dst = base + (uint32_t)slot * p.stage_bytes + unit;
          const uint8_t* src = w + col / 2;
#pragma unroll
          for (int r = 0; r < kTileRows; r += 8)
            // rows past the last repeat it; their logits are not stored
            cp_async8(dst + r * 128, src + (size_t)min(t * kTileRows + r0 + r, a.n - 1) * pitch);
        }
        if (++slot == p.ring) { slot = 0; phase ^= 1u; }
        if (++c == p.stages_k) { c = 0; ++t; }
      }
      cp_async_commit();
      if (i >= p.copy_depth) {
        if (p.copy_depth == 3)
          cp_async_wait<3>();
        else if (p.copy_depth == 2)
          cp_async_wait<2>();
        else
          cp_async_wait<1>();
        // the tensor core reads through the async proxy
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[done_slot]);
        if (++done_slot == p.ring) done_slot = 0;
      }
    }
    cp_async_wait<0>();
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

template <int XFMT, bool COPY, typename OT>
cudaError_t launch_t(const MxLogitsArgs& a, cudaStream_t s) {
  using K = Kind<XFMT, COPY>;
  MxParams p{};
  p.a = a;
  p.wait_budget = diag_wait_budget();
  p.tiles = (a.n + kTileRows - 1) / kTileRows;
  p.tile_cols = (int)mx_tile_cols(a.k);
  p.stages_k = (a.k + kStageCols - 1) / kStageCols;
  p.slices = (a.m + K::kSlice - 1) / K::kSlice;
  p.npad = ((a.m < K::kSlice ? a.m : K::kSlice) + 15) / 16 * 16;
  p.xtiles = (p.npad + 127) / 128;
  const uint32_t scale_cols = 2u * (8u + 8u * (uint32_t)p.xtiles);
  p.acc_bufs = 2u * (uint32_t)p.npad + scale_cols <= 512u ? 2 : 1;
  p.tmem_cols = 32;
  while (p.tmem_cols < (uint32_t)(p.acc_bufs * p.npad) + scale_cols) p.tmem_cols <<= 1;
  // a stage: weight, tokens, their scales; every part a multiple of 1024 bytes
  p.off_x = K::kBlocks * kBlockBytes;
  p.off_ws = p.off_x + (uint32_t)(K::kBlocks * p.npad * 128);
  p.off_xs = p.off_ws + 2 * kMxTileBytes;
  p.stage_bytes = p.off_xs + (uint32_t)p.xtiles * 2 * kMxTileBytes;
  const uint32_t room = 227u * 1024u - 1024u - 256u;
  p.ring = (int)(room / p.stage_bytes);
  if (p.ring > kMaxStages) p.ring = kMaxStages;
  if (p.ring < kMinStages) return cudaErrorInvalidConfiguration;
  p.copy_depth = p.ring - 1 < kMaxCopyDepth ? p.ring - 1 : kMaxCopyDepth;
  p.off_bar = (uint32_t)p.ring * p.stage_bytes;
  const size_t smem = p.off_bar + 256 + 1024;

  CUtensorMap tw, tx;
  const uint64_t wrow = (uint64_t)a.k / 2, xrow = K::kFp8 ? (uint64_t)a.k : (uint64_t)a.k / 2;
  cudaError_t e = cudaSuccess;
  if (K::kFp8 && !COPY)
    e = make_tmap_e2m1_spread(&tw, a.w_codes, (uint64_t)a.k, (uint64_t)a.n, kTileRows);
  else
    e = make_tmap_2d(&tw, a.w_codes, 4, wrow / 4, (uint64_t)a.n, wrow, 32, kTileRows,
                     Swizzle::k128B);
  if (e != cudaSuccess) return e;
  e = make_tmap_2d(&tx, a.x_codes, 4, xrow / 4, (uint64_t)a.m, xrow, 32, (uint32_t)p.npad,
                   Swizzle::k128B);
  if (e != cudaSuccess) return e;
  auto kern = mx_logits_kernel<XFMT, COPY, OT>;
  static size_t configured = 0;
  if (smem > configured) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    configured = smem;
  }
  int teams = device_sm_count() / p.slices;
  if (teams < 1) teams = 1;
  if (teams > p.tiles) teams = p.tiles;
  e = launch_pdl(kern, dim3((unsigned)(teams * p.slices)), dim3(K::kWarps * 32), smem, s, tw, tx, p);
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
  // blocks of 32-byte aligned rows
  if (a.k % 128 == 0 && reinterpret_cast<uintptr_t>(a.w_codes) % 32 == 0)
    return f16 ? launch_t<WQL_MX_FP8, false, __half>(a, s)
               : launch_t<WQL_MX_FP8, false, __nv_bfloat16>(a, s);
  return f16 ? launch_t<WQL_MX_FP8, true, __half>(a, s)
             : launch_t<WQL_MX_FP8, true, __nv_bfloat16>(a, s);
}

}  // namespace wql
