// Internal launchers of the paged cache operators. Each enqueues on `stream`
// and returns the HIP status of the launch; arguments are validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "beam.h"

namespace tkp {

// A page table: row r's positions p lie in page tables[r * ld + p / S], slot p % S.
struct PageTable {
  int32_t* tables;
  int64_t ld;
  int64_t R;          // rows
  int C;              // pages of a row at most; C * S < 2^31
  int S;              // slots of a page
  int32_t* lengths;   // [R] positions that a row holds
  int32_t* uses;      // [P] rows' entries that name a page
  int64_t P;
};

hipError_t launch_pages_fork(const PageTable& t, const int32_t* parents, int64_t N, int K, hipStream_t stream);

int64_t pages_resize_workspace(int64_t R, int64_t P);
// A cache's rows are the pages and its positions the slots. can_copy: the caches
// are there (those without elements are left out).
hipError_t launch_pages_resize(const PageTable& t, const int32_t* new_lengths, const BeamState* caches, int64_t count,
                               bool can_copy, void* workspace, hipStream_t stream);

struct CompactArgs {
  const int32_t* tables;
  int64_t ld;
  int64_t N;
  int C, S, D;
  int64_t P;
  const int32_t* starts;  // [N]
  const int32_t* path;    // [N, D]
  const int32_t* counts;  // [N]
};
hipError_t launch_pages_compact(const BeamState* caches, int64_t count, const CompactArgs& a, hipStream_t stream);

// Whether the launchers take the cache: columns of a page below 2^31.
bool page_state_fits(const BeamState& s);

}  // namespace tkp
