// How a verification of drafted tokens is cut into workgroups and launches: plain
// functions, which the host's tests run as well.
#pragma once

#include <stdint.h>

namespace tkp {
namespace verify {

constexpr int kWaveLanes = 64;
constexpr int kT = 256;    // threads of a workgroup that sums chunks
constexpr int kBlock = 8;  // neighbouring elements of a thread
constexpr int kPiece = kWaveLanes * kBlock;  // of a wave
// Threads of a workgroup that works on the row where a path ends, which is cut into
// parts of whole pieces, one for each wave, and no more parts than kFew.
constexpr int kFew = 256, kMany = 1024;

// A row in chunks of so many vectors of 16 bytes.
struct Split {
  int chunks, vecs;
};

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int kUnits = 256;     // compute units
constexpr int kMaxLayers = 32;  // vectors of a thread at most, 16-bit types (fp32: twice)

// Chunks of few rows: no more of all than compute units, and none of less than a
// group of vectors. (16 sequences of 4 drafts with draft logits, V 151936 bf16, take
// 24.7 us, and 25.8 with twice as many chunks; 24 of 3, V 128256 fp32, 23.0 and 25.3.)
inline Split split_of(int dtype, int64_t rows, int V) {
  const int64_t per = dtype == 0 ? 4 : 8;
  const int64_t nv = V / per;
  const int64_t largest = kT * kMaxLayers * 8 / per, smallest = kT * 32 / per;
  const int64_t least = ceil_div(nv, largest), most = ceil_div(nv, smallest);
  int64_t c = rows > 0 ? kUnits / rows : 1;
  c = c < most ? c : most;
  c = c > least ? c : least;
  c = c > 1 ? c : 1;
  return Split{static_cast<int>(c), static_cast<int>(ceil_div(nv, c))};
}

// Up to so many workgroups of kFew threads run at a time with what they hold of
// shared memory, and one sequence alone is done sooner by them (V 151936 bf16, 5
// drafts: 15.5 us and 16.7); beyond, kMany threads share one look at the path: 64
// sequences of 4 drafts 52 us and 71, 128 of 3, V 128256 fp32, 113 and 156.
constexpr int kFewBlocks = 512;
// What a workgroup does besides, in pieces of a wave (counting none, 420 sequences
// of 2 proposals, V 151936 bf16, are cut in 7 and take 217 us instead of 122).
constexpr int kTurnPieces = 3;
// Workgroups for the row where a sequence's path ends, their threads, and pieces of
// their waves.
struct Cut {
  int threads, groups, pieces;
};
inline Cut cut_of(int64_t N, int V) {
  const int64_t all = V > 0 ? ceil_div(V, kPiece) : 1;
  const int64_t few = ceil_div(all, kFew);  // pieces, for no more parts than threads
  if (N * ceil_div(all, few * (kFew / kWaveLanes)) <= kFewBlocks)
    return Cut{kFew, static_cast<int>(ceil_div(all, few * (kFew / kWaveLanes))), static_cast<int>(few)};
  // one workgroup fills a compute unit: as many for a sequence as take the fewest turns
  constexpr int kWaves = kMany / kWaveLanes;
  Cut best{kMany, 1, static_cast<int>(ceil_div(all, kWaves))};
  int64_t least = INT64_MAX;
  for (int g = 1; g <= kFew / kWaves && (g - 1) * kWaves < all; ++g) {
    const int64_t pieces = ceil_div(all, g * kWaves), cost = ceil_div(N * g, kUnits) * (pieces + kTurnPieces);
    if (cost < least) {
      least = cost;
      best.groups = g;
      best.pieces = static_cast<int>(pieces);
    }
  }
  return best;
}

// A path through a tree needs few of its rows. Where there is much to read, the first
// rows are summed before, then (kStagedBytes) what is left behind the one that each
// path goes on at, or (kTwiceBytes) first that one alone. Trees of 39 drafts, three
// behind each, V 151936 bf16, with all rows read at once, one step and two: 4 of them
// (49 MB) 24.0, 26.5 and 32.5 us, 8 (97 MB) 34.1, 30.7 and 34.8, 16 (194 MB) 48.7, 37.6
// and 37.4, 32 81, 50 and 42.
// (Chains do not gain: 64 of 4 drafts with draft logits take 59 us with half of their
// rows read first, 54 all at once; 128 of 3 drafts, V 128256 fp32, 113 both ways.)
constexpr int64_t kStagedBytes = int64_t{80} << 20, kTwiceBytes = int64_t{160} << 20;
constexpr int kStagedElements = 16384;  // of a chunk
// Workgroups for all that is left, as many as run at a time.
constexpr int kBehindBlocks = 1280;  // 5 of a compute unit
inline int behind_groups(int64_t N, int D, const Split& split) {
  const int64_t most = static_cast<int64_t>(D) * split.chunks;
  int64_t g = kBehindBlocks / N;
  g = g > split.chunks ? g : split.chunks;
  return static_cast<int>(g < most ? g : most);
}

// How a call is cut.
struct Plan {
  int steps;  // of a tree, behind its first rows; 0: all rows at once
  Split split;
  Cut cut;
};
inline Plan plan_of(int dtype, int64_t N, int D, int V, bool draft, bool tree) {
  const int64_t rows = N * (D + 1 + (draft ? D : 0)), bytes = rows * V * (dtype == 0 ? 4 : 2);
  Plan p{tree && D > 0 ? (bytes > kStagedBytes) + (bytes > kTwiceBytes) : 0, split_of(dtype, rows, V), cut_of(N, V)};
  if (p.steps > 0) {
    const int64_t nv = V / (dtype == 0 ? 4 : 8), c = ceil_div(V, kStagedElements);
    p.split = Split{static_cast<int>(c), static_cast<int>(ceil_div(nv, c))};
  }
  return p;
}

inline int targets_of(const Plan& p, int D) { return p.steps > 0 ? 1 : D + 1; }

// Workgroups of a sequence in the first kernel, and for the row where its path ends.
inline int64_t rows_groups(const Plan& p, int D, bool draft) {
  return static_cast<int64_t>(targets_of(p, D) + (draft ? D : 0)) * p.split.chunks;
}
inline int final_groups(const Plan& p, bool greedy) { return greedy ? 1 : p.cut.groups; }
inline int final_threads(const Plan& p, bool greedy) { return greedy ? kFew : p.cut.threads; }

// Sequences of a launch: a grid of any of the kernels has at most 2^30 threads (it has
// to hold fewer than 2^32), or is that of one sequence.
inline int64_t sequences_of_launch(const Plan& p, int64_t N, int D, bool draft, bool greedy) {
  const int64_t rows = rows_groups(p, D, draft) * kT, behind = p.steps > 0 ? behind_groups(N, D, p.split) * int64_t{kT} : 0;
  int64_t threads = static_cast<int64_t>(final_groups(p, greedy)) * final_threads(p, greedy);
  threads = threads > rows ? threads : rows;
  threads = threads > behind ? threads : behind;
  const int64_t n = (int64_t{1} << 30) / threads;
  return n > 1 ? n : 1;
}

}  // namespace verify
}  // namespace tkp
