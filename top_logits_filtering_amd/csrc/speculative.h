// Internal launcher of the verification of drafted tokens. It enqueues on
// `stream` and returns the HIP status of the launch; arguments are validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tkp {

struct VerifyArgs {
  const void* logits;        // [N * (D + 1), V], rows ld elements apart
  int64_t ld;
  const void* draft_logits;  // [N * D, V], rows ld_draft elements apart, or NULL
  int64_t ld_draft;
  int64_t N;
  int D, V;
  const int32_t* drafts;     // [N, D]
  const float* uniforms;     // [N, D + 1], or NULL: greedy
  const int32_t* parents;    // [N, D], or NULL: each draft follows the one before it
  const int32_t* lengths;    // [N], or NULL: D
  int32_t* out_tokens;       // [N, D + 1]
  int32_t* out_accepted;     // [N]
  int32_t* out_path;         // [N, D] or NULL
  void* workspace;           // verify_workspace() bytes, 16-byte aligned
};

int64_t verify_workspace(int dtype, int64_t N, int D, int V, bool draft_logits);
hipError_t launch_verify(int dtype, const VerifyArgs& a, hipStream_t stream);

}  // namespace tkp
