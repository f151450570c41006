// requests.cuh -- arguments and launchers of the operators for requests with
// adapters and for beam search (lora.cu, beam_select.cu, beam_reorder.cu),
// shared with the C-ABI layer (wql_api.cu).
#pragma once

#include "wql_common.cuh"

namespace wql {

// ---------------------------------------------------------------------------
// Adapters
// ---------------------------------------------------------------------------
// Ranks are padded to 16, 32, 64 or 128: chunks of 16, the k of one mma.
inline int lora_chunks(int rank) { return rank <= 16 ? 1 : rank <= 32 ? 2 : rank <= 64 ? 4 : 8; }

// Tokens are grouped by adapter in slices.
constexpr int kLoraSlice = 256;

struct LoraArgs {
  const void* a;
  const void* b;
  const float* scale;         // or null
  const void* x;
  const int32_t* ids;
  const void* y;
  void* out;
  uint4* u;                   // workspace: [m][chunks][4] fragments
  float* factor;              // workspace: [m]
  int dtype, rank, chunks;
  int count, n, k, m;
};
cudaError_t launch_lora_add(const LoraArgs& a, cudaStream_t s);

// ---------------------------------------------------------------------------
// Beam search
// ---------------------------------------------------------------------------
struct BeamSelectArgs {
  const void* logits;
  int dtype;
  int batch, beams, n, eos, order;
  const float* scores;
  int32_t* tokens;
  int32_t* parents;
  float* scores_out;
  float* ended;               // or null
  float2* stats;              // workspace: [rows][parts]
  uint64_t* keys;             // workspace: [rows][parts][beams]
  int parts, part_chunks;     // beam_parts()
};
// Parts of a row, and chunks of one.
struct BeamParts {
  int parts, chunks;
};
BeamParts beam_parts(int64_t rows, int64_t n, int dtype);
cudaError_t launch_beam_select(const BeamSelectArgs& a, cudaStream_t s);

cudaError_t launch_beam_reorder(const wql_state* states, int64_t count, const int32_t* parents,
                                int batch, int beams, const int32_t* lengths, cudaStream_t s);
// Whether two positions or states share memory.
bool states_overlap(const wql_state* states, int64_t count, int64_t rows);

}  // namespace wql
