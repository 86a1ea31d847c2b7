// Internal launchers of the beam search operators. Each enqueues on `stream`
// and returns the HIP status of the launch; shapes are already validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tkp {

// Quotients of 31-bit numbers by a fixed divisor: floor(x * m / 2^(31 + s))
// with m = ceil(2^(31 + s) / d), 2^s >= d. What m is too large by, below 1 in
// d's share of 2^(31 + s), moves the quotient of x < 2^31 by less than 1 / d.
struct Div {
  uint32_t d, m, s;
};
inline Div make_div(uint32_t d) {
  uint32_t s = 0;
  while ((uint64_t{1} << s) < d) ++s;
  return Div{d, static_cast<uint32_t>(((uint64_t{1} << (31 + s)) + d - 1) / d), s};
}
__device__ __forceinline__ uint32_t quotient(uint32_t x, const Div& v) {
  return static_cast<uint32_t>((static_cast<uint64_t>(x) * v.m) >> (31 + v.s));
}

struct BeamSelectArgs {
  const void* logits;        // [N * K, V], rows ld elements apart
  int64_t ld;
  int64_t N;
  int K, V, n;
  const float* scores;       // [N, K] accumulated log-probabilities
  const uint8_t* finished;   // [N, K] or NULL
  int32_t end_token;
  const float* weights;      // [N, K] or NULL
  float* out_scores;         // [N, n]
  int32_t* out_parents;      // [N, n]
  int32_t* out_tokens;       // [N, n]
  void* workspace;           // beam_select_workspace() bytes, 16-byte aligned
};

// Chunks that a row is split into, and 16-byte vectors per chunk.
struct BeamSplit {
  int chunks;
  int vecs;
};
BeamSplit beam_select_split(int dtype, int64_t rows, int V, int n);
int64_t beam_select_workspace(int dtype, int64_t N, int K, int V, int n);
hipError_t launch_beam_select(int dtype, const BeamSelectArgs& a, hipStream_t stream);

// One state of beam_reorder_states, sizes in elements of the axes and strides
// in bytes: rows, three axes of any kind, positions, and a contiguous run.
struct BeamState {
  char* data;
  int64_t row_stride;
  int64_t size[3];
  int64_t stride[3];
  int64_t positions;
  int64_t position_stride;
  int64_t run;
};

// States one launch moves at most: their descriptions travel as kernel arguments.
constexpr int kMaxStates = 24;

// Whether launch_beam_reorder takes the state: its units per row stay below 2^31.
bool beam_state_fits(const BeamState& s, int K);
// count <= kMaxStates states whose memory is disjoint; bytes: what all states
// of the call hold together.
hipError_t launch_beam_reorder(const BeamState* states, int count, const int32_t* parents, int64_t N, int K,
                               const int32_t* lengths, int64_t bytes, hipStream_t stream);

struct BeamBacktraceArgs {
  const int32_t* tokens;   // [T, N, K]
  const int32_t* parents;  // [T, N, K]
  const int32_t* beams;    // [N, M] or NULL (hypothesis m ends at beam m)
  const int32_t* lengths;  // [N, M] or NULL (T)
  int32_t* out;            // [N, M, T]
  int64_t T, N;
  int K, M;
  int32_t pad;
};
hipError_t launch_beam_backtrace(const BeamBacktraceArgs& a, hipStream_t stream);

}  // namespace tkp
