// beam_reorder.cu -- the states of beams follow a selection, in place: row
// b * beams + j of every state becomes what row b * beams + parents[b, j] was.
//
// HBM-bound: what has to move is one read of every parent of a moved beam and
// one write of every moved beam.  A thread takes the same 16 bytes of all rows of
// a sequence: it loads them from the parents and then stores them to the
// children, and no other thread touches these bytes, so no copy of a state and no
// barrier is needed.  Where there is enough to move, the pieces wait in shared
// memory instead of registers (16 sequences of 4 beams, 32 states: 141 us, 190
// through registers), which also reads a parent of several children once.
// Measured: that case, ranked, 88 % of the copy rate; 9 x 8 beams, anchored, 12
// states of 746 KB a row, 60.5 us (98 %); one sequence of 4 beams, 48 states of 77
// KB a row, 4.2 us.
#include <algorithm>
#include <utility>

#include "requests.cuh"
#include "sm100.cuh"

namespace wql {
namespace {

constexpr int kThreads = 256;
constexpr int kStates = 64;              // of one launch (4 KB of arguments)

struct States {
  wql_state s[kStates];
};

template <typename V> struct Zero;
template <> struct Zero<uint4> { static __device__ __forceinline__ uint4 get() { return make_uint4(0u, 0u, 0u, 0u); } };
template <> struct Zero<uint32_t> { static __device__ __forceinline__ uint32_t get() { return 0u; } };
template <> struct Zero<uint8_t> { static __device__ __forceinline__ uint8_t get() { return 0; } };

// Moves one V of all rows of a sequence at `at`.
template <typename V, int BEAMS>
__device__ __forceinline__ void move(unsigned char* at, int64_t row_stride, const int* parent,
                                     int beams) {
  V v[BEAMS];
#pragma unroll
  for (int j = 0; j < BEAMS; ++j) {
    v[j] = Zero<V>::get();
    if (j < beams && parent[j] != j)
      v[j] = *reinterpret_cast<const V*>(at + parent[j] * row_stride);
  }
#pragma unroll
  for (int j = 0; j < BEAMS; ++j)
    if (j < beams && parent[j] != j) *reinterpret_cast<V*>(at + j * row_stride) = v[j];
}

// grid: (tiles, sequences, states).  A run is a piece of a row without gaps:
// a block's positions where they touch, else one position.  Runs are cut into
// pieces of sizeof(V) bytes, the last one of a run moved in parts.
template <typename V, int BEAMS>
__global__ void __launch_bounds__(kThreads) beam_reorder_kernel(const States states,
                                                                const int32_t* parents, int beams,
                                                                const int32_t* lengths) {
  __shared__ int parent[BEAMS];
  __shared__ int moved;
  griddep_launch_dependents();
  griddep_wait();
  const wql_state& s = states.s[blockIdx.z];
  const int b = blockIdx.y;
  if (threadIdx.x == 0) moved = 0;
  __syncthreads();
  if (threadIdx.x < beams) {
    int p = parents[(size_t)b * beams + threadIdx.x];
    if ((uint32_t)p >= (uint32_t)beams) p = threadIdx.x;
    parent[threadIdx.x] = p;
    if (p != (int)threadIdx.x) moved = 1;
  }
  __syncthreads();
  if (!moved) return;
  int64_t length = s.positions;
  if (lengths) length = min(length, (int64_t)max(lengths[b], 0));
  const bool dense = s.position_stride == s.position_bytes;
  const int64_t run_bytes = dense ? length * s.position_bytes : s.position_bytes;
  const int64_t inner = dense ? 1 : length;                 // runs of a block
  const uint32_t pieces = (uint32_t)((run_bytes + sizeof(V) - 1) / sizeof(V));
  const uint64_t total = (uint64_t)s.outer * inner * pieces;  // below 2^32: bytes of a row
  unsigned char* data = static_cast<unsigned char*>(s.data) + (int64_t)b * beams * s.row_stride;
  for (uint64_t i = (uint64_t)blockIdx.x * kThreads + threadIdx.x; i < total;
       i += (uint64_t)gridDim.x * kThreads) {
    const uint32_t run = (uint32_t)i / pieces, piece = (uint32_t)i - run * pieces;
    uint32_t o = run, p = 0;
    if (!dense) {
      o = run / (uint32_t)length;
      p = run - o * (uint32_t)length;
    }
    const int64_t in_run = (int64_t)piece * (int64_t)sizeof(V);
    unsigned char* at = data + o * s.outer_stride + p * s.position_stride + in_run;
    if (in_run + (int64_t)sizeof(V) <= run_bytes) {
      move<V, BEAMS>(at, s.row_stride, parent, beams);
    } else {
      for (int64_t k = in_run; k < run_bytes; ++k, ++at)
        move<uint8_t, BEAMS>(at, s.row_stride, parent, beams);
    }
  }
}

// The same for 16-byte pieces of up to kAsyncBeams rows, without registers for
// what is under way: a thread's pieces of the parents go to its own places in
// shared memory, kStages columns ahead, and from there to the children.
constexpr int kAsyncBeams = 16;
constexpr int kStages = 3;

__global__ void __launch_bounds__(kThreads) beam_reorder_async_kernel(const States states,
                                                                      const int32_t* parents, int beams,
                                                                      const int32_t* lengths) {
  extern __shared__ uint4 ring[];              // [stage][beam][thread]
  __shared__ int parent[kAsyncBeams];
  griddep_launch_dependents();
  griddep_wait();
  const wql_state& s = states.s[blockIdx.z];
  const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
  // every warp for itself: the rows that are written, and those that are read
  int p = lane < beams ? parents[(size_t)b * beams + lane] : -1;
  const bool moves = (uint32_t)p < (uint32_t)beams && p != lane;
  if (tid < beams) parent[tid] = p;
  const uint32_t children = __ballot_sync(0xFFFFFFFFu, moves);
  const uint32_t read = __reduce_or_sync(0xFFFFFFFFu, moves ? 1u << p : 0u);
  __syncthreads();
  if (children == 0u) return;
  int64_t length = s.positions;
  if (lengths) length = min(length, (int64_t)max(lengths[b], 0));
  const bool dense = s.position_stride == s.position_bytes;
  const int64_t run_bytes = dense ? length * s.position_bytes : s.position_bytes;
  const uint32_t pieces = (uint32_t)((run_bytes + 15) / 16);
  const uint64_t total = (uint64_t)s.outer * (dense ? 1 : length) * pieces;    // below 2^32
  unsigned char* data = static_cast<unsigned char*>(s.data) + (int64_t)b * beams * s.row_stride;
  const uint64_t step = (uint64_t)gridDim.x * kThreads;
  uint64_t i = (uint64_t)blockIdx.x * kThreads + tid;

  struct Piece {
    unsigned char* at;                         // in row 0; null: none
    int bytes;
  };
  auto piece_at = [&](uint64_t k) {
    if (k >= total) return Piece{nullptr, 0};
    const uint32_t run = (uint32_t)k / pieces, piece = (uint32_t)k - run * pieces;
    uint32_t o = run, q = 0;
    if (!dense) {
      o = run / (uint32_t)length;
      q = run - o * (uint32_t)length;
    }
    const int64_t in_run = (int64_t)piece * 16;
    return Piece{data + o * s.outer_stride + q * s.position_stride + in_run,
                 (int)min((int64_t)16, run_bytes - in_run)};
  };
  const uint32_t mine = (uint32_t)__cvta_generic_to_shared(ring) + tid * 16;
  const uint32_t stage_bytes = (uint32_t)beams * kThreads * 16;
  auto load = [&](const Piece& w, uint32_t to) {
    if (w.bytes == 16)
      for (uint32_t m = read; m != 0u; m &= m - 1u) {
        const int r = __ffs(m) - 1;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + r * (kThreads * 16)),
                     "l"(w.at + r * s.row_stride) : "memory");
      }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto store = [&](const Piece& w, uint32_t from) {
    if (w.bytes == 16) {
      for (uint32_t m = children; m != 0u; m &= m - 1u) {
        const int j = __ffs(m) - 1;
        *reinterpret_cast<uint4*>(w.at + j * s.row_stride) = lds128(from + parent[j] * (kThreads * 16));
      }
    } else {                                   // the end of a run
      for (int k = 0; k < w.bytes; ++k) {
        uint8_t v[kAsyncBeams];
#pragma unroll
        for (int j = 0; j < kAsyncBeams; ++j)
          if (children >> j & 1u) v[j] = w.at[k + parent[j] * s.row_stride];
#pragma unroll
        for (int j = 0; j < kAsyncBeams; ++j)
          if (children >> j & 1u) w.at[k + j * s.row_stride] = v[j];
      }
    }
  };
  Piece queue[kStages];
#pragma unroll
  for (int k = 0; k < kStages; ++k) {
    queue[k] = piece_at(i + k * step);
    load(queue[k], mine + k * stage_bytes);
  }
  while (queue[0].at != nullptr) {
#pragma unroll
    for (int k = 0; k < kStages; ++k) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      store(queue[k], mine + k * stage_bytes);
      queue[k] = piece_at(i + (kStages + k) * step);
      load(queue[k], mine + k * stage_bytes);
    }
    i += kStages * step;
  }
}

template <typename V, int BEAMS>
cudaError_t launch(const States& st, int count, int64_t largest, const int32_t* parents, int batch,
                   int beams, const int32_t* lengths, cudaStream_t s) {
  // Enough blocks for eight waves, no more than the largest row has tiles.  (Of
  // those with shared memory an SM holds fewer: 9 x 8 beams anchored 60 us with
  // 8 waves, 84 with 32.)
  const int64_t tiles = (largest + kThreads * (int64_t)sizeof(V) - 1) / (kThreads * (int64_t)sizeof(V));
  const size_t smem = (size_t)kStages * beams * kThreads * 16;
  auto blocks = [&](int64_t resident) {
    const int64_t want = (8 * resident * device_sm_count() + (int64_t)batch * count - 1) / ((int64_t)batch * count);
    return dim3((unsigned)(tiles < want ? tiles : want), (unsigned)batch, (unsigned)count);
  };
  if constexpr (sizeof(V) == 16) {
    const int64_t resident = (int64_t)(200 * 1024 / smem) > 0 ? (int64_t)(200 * 1024 / smem) : 1;
    const dim3 grid = blocks(resident);
    // a column or two a thread: nothing to copy ahead (one sequence of 4 beams, 48
    // states of 77 KB a row: 4.2 us by registers, 5.2 through shared memory)
    if (beams <= kAsyncBeams && tiles > 2 * (int64_t)grid.x) {
      static LargestPerDevice limit;
      cudaError_t e = allow_smem(limit, beam_reorder_async_kernel, smem);
      if (e != cudaSuccess) return e;
      e = launch_pdl(beam_reorder_async_kernel, grid, dim3(kThreads), smem, s, st, parents, beams, lengths);
      if (e == cudaSuccess) note_launch();
      return e;
    }
  }
  const cudaError_t e = launch_pdl(beam_reorder_kernel<V, BEAMS>, blocks(8), dim3(kThreads), 0, s, st, parents,
                                   beams, lengths);
  if (e == cudaSuccess) note_launch();
  return e;
}

template <typename V>
cudaError_t launch_b(const States& st, int count, int64_t largest, const int32_t* parents, int batch,
                     int beams, const int32_t* lengths, cudaStream_t s) {
  if (beams <= 4) return launch<V, 4>(st, count, largest, parents, batch, beams, lengths, s);
  if (beams <= 8) return launch<V, 8>(st, count, largest, parents, batch, beams, lengths, s);
  if (beams <= 16) return launch<V, 16>(st, count, largest, parents, batch, beams, lengths, s);
  return launch<V, 32>(st, count, largest, parents, batch, beams, lengths, s);
}

// The widest access that a state's addresses allow.
int width_of(const wql_state& s) {
  const bool dense = s.position_stride == s.position_bytes;
  const uint64_t bits = reinterpret_cast<uintptr_t>(s.data) | (uint64_t)s.row_stride |
                        (s.outer > 1 ? (uint64_t)s.outer_stride : 0) |
                        (dense ? 0 : (uint64_t)s.position_stride);
  return bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 1;
}

}  // namespace

cudaError_t launch_beam_reorder(const wql_state* states, int64_t count, const int32_t* parents,
                                int batch, int beams, const int32_t* lengths, cudaStream_t s) {
  for (const int width : {16, 4, 1}) {
    States st;
    int have = 0;
    int64_t largest = 0;
    for (int64_t i = 0; i < count; ++i) {
      const wql_state& w = states[i];
      const int64_t bytes = w.outer * w.positions * w.position_bytes;
      if (bytes > 0 && width_of(w) == width) {
        st.s[have++] = w;
        if (bytes > largest) largest = bytes;
      }
      if (have == kStates || (i + 1 == count && have > 0)) {
        const cudaError_t e =
            width == 16 ? launch_b<uint4>(st, have, largest, parents, batch, beams, lengths, s)
            : width == 4 ? launch_b<uint32_t>(st, have, largest, parents, batch, beams, lengths, s)
                         : launch_b<uint8_t>(st, have, largest, parents, batch, beams, lengths, s);
        if (e != cudaSuccess) return e;
        have = 0;
        largest = 0;
      }
    }
  }
  return cudaSuccess;
}

// ---------------------------------------------------------------------------
// Overlap, on the host.  Inside a state rows, blocks and positions are nested
// in some order of their strides; each must hold what is inside it.  Two states
// whose spans meet must have the same stride at every level that repeats, and
// at one of them lie apart between its repetitions.
// ---------------------------------------------------------------------------
namespace {

struct Level {
  int64_t count, stride;
};
struct Shape {
  uintptr_t at;
  Level level[3];                        // largest stride first, those that repeat
  int levels;
  int64_t inner;                         // bytes without gaps
  int64_t extent[4];                     // of one element of level i (extent[levels] = inner)
};

// False where a state overlaps itself.
bool shape_of(const wql_state& s, int64_t rows, Shape* out) {
  Level all[3] = {{rows, s.row_stride}, {s.outer, s.outer_stride}, {s.positions, s.position_stride}};
  out->at = reinterpret_cast<uintptr_t>(s.data);
  out->levels = 0;
  for (const Level& l : all)
    if (l.count > 1) out->level[out->levels++] = l;
  for (int i = 0; i < out->levels; ++i)
    for (int j = i + 1; j < out->levels; ++j)
      if (out->level[j].stride > out->level[i].stride) std::swap(out->level[i], out->level[j]);
  out->inner = s.position_bytes;
  int64_t size = s.position_bytes;
  for (int i = out->levels - 1; i >= 0; --i) {
    out->extent[i + 1] = size;
    if (out->level[i].stride < size) return false;
    size = (out->level[i].count - 1) * out->level[i].stride + size;
  }
  out->extent[0] = size;
  return true;
}

// Whether elements of level i share bytes, b's starting d behind a's.
bool meet(const Shape& a, const Shape& b, int i, int64_t d) {
  if (d >= a.extent[i] || -d >= b.extent[i]) return false;
  if (i == a.levels || i == b.levels || a.level[i].stride != b.level[i].stride) return true;
  const int64_t stride = a.level[i].stride;
  const int64_t r = ((d % stride) + stride) % stride;
  // (an element is no larger than the stride: these are its neighbours)
  return meet(a, b, i + 1, r) || meet(a, b, i + 1, r - stride);
}

// Whether all states lie apart modulo a stride that their levels i have in
// common and that divides the strides outside: layers that share rows or
// positions.  (160 of one allocation: 12 us of the host, 223 in pairs.)
bool apart_at(const Shape* shapes, int count, int i) {
  std::pair<int64_t, int64_t> part[WQL_MAX_STATES];        // where it begins, its bytes
  const int64_t stride = shapes[0].levels > i ? shapes[0].level[i].stride : 0;
  for (int k = 0; k < count; ++k) {
    const Shape& s = shapes[k];
    if (s.levels <= i || s.level[i].stride != stride) return false;
    for (int o = 0; o < i; ++o)
      if (s.level[o].stride % stride != 0) return false;
    part[k] = {(int64_t)(s.at % (uintptr_t)stride), s.extent[i + 1]};
  }
  std::sort(part, part + count);
  for (int k = 0; k + 1 < count; ++k)
    if (part[k].first + part[k].second > part[k + 1].first) return false;
  return part[count - 1].first + part[count - 1].second <= part[0].first + stride;
}

}  // namespace

bool states_overlap(const wql_state* states, int64_t count, int64_t rows) {
  Shape shapes[WQL_MAX_STATES];
  int have = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (states[i].outer * states[i].positions * states[i].position_bytes == 0) continue;
    if (!shape_of(states[i], rows, &shapes[have++])) return true;
  }
  std::sort(shapes, shapes + have, [](const Shape& x, const Shape& y) { return x.at < y.at; });
  bool near = false;
  uintptr_t end = 0;
  for (int i = 0; i < have && !near; ++i) {
    near = shapes[i].at < end;
    end = std::max(end, shapes[i].at + (uintptr_t)shapes[i].extent[0]);
  }
  if (!near) return false;
  for (int i = 0; i < 3; ++i)
    if (apart_at(shapes, have, i)) return false;
  for (int i = 0; i < have; ++i)
    for (int j = i + 1; j < have && shapes[j].at - shapes[i].at < (uintptr_t)shapes[i].extent[0]; ++j)
      if (meet(shapes[i], shapes[j], 0, (int64_t)(shapes[j].at - shapes[i].at))) return true;
  return false;
}

}  // namespace wql
