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

// Up to so many workgroups of kFew threads are taken, beyond them those of kMany, which
// share one look at the path. Where the two take as long depends on the type and on
// whether there are draft logits, and lies between 400 and 900 (us, kFew and kMany):
//   bf16, V 151936, 4 drafts with draft logits: 152 workgroups 17.7 and 19.2, 380 24.6
//   and 24.5, 532 26.3 and 24.6, 988 34.8 and 30.9;
//   fp32, V 128256, 3 with draft logits: 378 19.1 and 20.0, 630 22.3 and 22.3, 882 25.6
//   and 24.1, 2016 44.4 and 37.6;
//   fp16, V 32003, 4 with draft logits: 256 17.0 and 19.3, 512 20.7 and 21.9, 768 22.6
//   and 22.2; 2 proposals: 512 14.2 and 15.0, 1024 17.5 and 16.6.
// (1024 of kFew run at a time, as their registers allow four a SIMD. Short rows of large
// batches would do better with kFew: 400 sequences, V 5000 fp32, 29.9 and 34.3.)
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
// and 37.4, 32 86, 54 and 43. The same trees in fp32, V 128256: 4 (82 MB) 28.8, 30.6 and
// 35.2, 8 (164 MB) 44.6, 35.3 and 37.8, 16 66.5, 45.0 and 40.6; V 32003 bf16: 40 (102 MB)
// 35.6, 31.9 and 37.8, 160 91, 60 and 47. The host does not see what the trees are like:
// a chain given as parents, of which far more lies behind, loses (32 of 39 drafts, V
// 151936 bf16, 83, 102 and 105; 128 of 8 85, 98 and 103) and is better given without.
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
