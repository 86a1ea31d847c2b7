// Reordering of beam states in place: row n*K+b of every state becomes the
// former row n*K+parents[n][b].
//
// One thread owns a column: the same 16 bytes of all K rows of a prompt. It
// reads the parents' columns of every beam that changes, then writes them, so
// no order among beams has to be found (cycles and copies alike) and no second
// buffer is needed: each changed row is read and written once, where gathering
// into a new tensor and copying it back moves twice that. Rows that stay are
// not touched. The K values wait in registers, so wide beams take narrower
// columns.

#include "beam.h"
#include "device_common.h"

namespace tkp {
namespace {

constexpr int kMoveThreads = 256;

// A state cut into panels (one index of each of the three axes) of columns.
struct MoveState {
  char* data;
  int64_t row_stride;
  int64_t stride[3];
  int64_t position_stride;
  Div panel;           // columns per panel
  Div size1, size2;
  Div run;             // columns per run; run.d == 0: positions are contiguous
  uint32_t columns;    // panels * columns per panel
  uint32_t run_bytes;  // bytes of a position, for the length's end
};

struct MoveArgs {
  uint32_t first[kMaxStates];  // each state's first block; the largest number behind the last state
  MoveState state[kMaxStates];
  Div items;
  int K;
  const int32_t* parents;
  const int32_t* lengths;
};

template <int W>
struct Column;
template <>
struct Column<16> { using type = uint4; };
template <>
struct Column<4> { using type = uint32_t; };
template <>
struct Column<2> { using type = uint16_t; };
template <>
struct Column<1> { using type = uint8_t; };

// KMAX: beams held; W: bytes of a column; U: columns per thread.
template <int KMAX, int W, int U>
__global__ __launch_bounds__(kMoveThreads) void beam_move_kernel(const MoveArgs a) {
  using col_t = typename Column<W>::type;
  int si = 0;
#pragma unroll
  for (int i = 1; i < kMaxStates; ++i) si += blockIdx.x >= a.first[i] ? 1 : 0;
  const MoveState& s = a.state[si];
  const uint32_t local = blockIdx.x - a.first[si];
  const uint32_t tile = quotient(local, a.items);
  const int64_t item = local - tile * a.items.d;

  const int32_t* __restrict__ parents = a.parents + item * a.K;
  const int64_t len = a.lengths != nullptr ? a.lengths[item] : INT64_MAX;
  if (len <= 0) return;

  // byte offsets of this thread's columns, and how many bytes of each count
  int64_t off[U];
  int live[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t c = tile * (kMoveThreads * U) + u * kMoveThreads + threadIdx.x;
    live[u] = 0;
    off[u] = 0;
    if (c < s.columns) {
      const uint32_t p = quotient(c, s.panel);
      const uint32_t j = c - p * s.panel.d;
      const uint32_t p2 = quotient(p, s.size2), i2 = p - p2 * s.size2.d;
      const uint32_t i0 = quotient(p2, s.size1), i1 = p2 - i0 * s.size1.d;
      off[u] = i0 * s.stride[0] + i1 * s.stride[1] + i2 * s.stride[2];
      if (s.run.d == 0) {  // positions follow each other: the panel is one piece
        const int64_t at = static_cast<int64_t>(j) * W;
        off[u] += at;
        const int64_t end = len < INT32_MAX ? len * s.run_bytes : INT64_MAX;
        live[u] = at >= end ? 0 : (end - at < W ? static_cast<int>(end - at) : W);
      } else {
        const uint32_t pos = quotient(j, s.run);
        off[u] += pos * s.position_stride + static_cast<int64_t>(j - pos * s.run.d) * W;
        live[u] = pos < len ? W : 0;
      }
    }
  }

  char* base = s.data + item * a.K * s.row_stride;
  col_t val[U][KMAX];
#pragma unroll
  for (int b = 0; b < KMAX; ++b) {
    if (b < a.K) {
      const int p = parents[b];
      if (p != b && p >= 0 && p < a.K) {
        const char* from = base + p * s.row_stride;
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (live[u] > 0) val[u][b] = *reinterpret_cast<const col_t*>(from + off[u]);
      }
    }
  }
#pragma unroll
  for (int b = 0; b < KMAX; ++b) {
    if (b < a.K) {
      const int p = parents[b];
      if (p != b && p >= 0 && p < a.K) {
        char* to = base + b * s.row_stride;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (live[u] == W) {
            *reinterpret_cast<col_t*>(to + off[u]) = val[u][b];
          } else if constexpr (W == 16) {  // the length ends inside: whole words up to it
            uint32_t* w = reinterpret_cast<uint32_t*>(to + off[u]);
            if (live[u] >= 4) w[0] = val[u][b].x;
            if (live[u] >= 8) w[1] = val[u][b].y;
            if (live[u] >= 12) w[2] = val[u][b].z;
          }
        }
      }
    }
  }
}

int64_t low_bit(int64_t x) { return x & -x; }

// Bytes of a column: what every address is aligned to, at most 16, and for
// wide beams what fits the registers. Columns of 16 bytes may reach past the
// length inside a piece of whole words; smaller ones never do.
int column_bytes(const BeamState& s, int K) {
  int64_t w = 16 | reinterpret_cast<int64_t>(s.data) | s.row_stride;
  for (int i = 0; i < 3; ++i)
    if (s.size[i] > 1) w |= s.stride[i];
  const bool joined = s.positions == 1 || s.position_stride == s.run;
  if (joined) w |= s.positions * s.run;
  else w |= s.position_stride | s.run;
  w = low_bit(w);
  const int64_t unit = low_bit(s.run | 16);
  if (joined && unit < 4 && w > unit) w = unit;
  if (w >= 16 && K <= 32) return 16;
  if (joined && w > unit) w = unit;
  return w >= 4 ? 4 : static_cast<int>(w);
}

// Bytes of a row, saturated (every size is at least 1).
uint64_t row_bytes(const BeamState& s) {
  const uint64_t most = uint64_t{1} << 62;
  uint64_t n = static_cast<uint64_t>(s.run);
  for (uint64_t f : {static_cast<uint64_t>(s.positions), static_cast<uint64_t>(s.size[0]),
                     static_cast<uint64_t>(s.size[1]), static_cast<uint64_t>(s.size[2])})
    n = n > most / f ? most : n * f;
  return n;
}

// Launches a.state[0, count) for all N prompts, as many of them at a time as
// keep a grid below 2^32 threads.
template <int KMAX, int W, int U>
hipError_t move_all(const MoveArgs& a, int count, int64_t N, hipStream_t stream) {
  constexpr int64_t kMost = int64_t{1} << 23;
  int64_t tiles[kMaxStates], sum = 0;
  for (int i = 0; i < count; ++i) {
    tiles[i] = (static_cast<int64_t>(a.state[i].columns) + kMoveThreads * U - 1) / (kMoveThreads * U);
    sum += tiles[i];
  }
  if (sum > kMost && count > 1) {
    for (int i = 0; i < count; ++i) {
      MoveArgs one = a;
      one.state[0] = a.state[i];
      if (const hipError_t e = move_all<KMAX, W, U>(one, 1, N, stream)) return e;
    }
    return hipSuccess;
  }
  const int64_t step = kMost / sum;  // tiles of one state are below 2^23
  for (int64_t n0 = 0; n0 < N; n0 += step) {
    const int64_t n = N - n0 < step ? N - n0 : step;
    MoveArgs b = a;
    int64_t blocks = 0;
    for (int i = 0; i < kMaxStates; ++i) {
      b.first[i] = i < count ? static_cast<uint32_t>(blocks) : 0xFFFFFFFFu;
      if (i >= count) continue;
      b.state[i].data += n0 * a.K * a.state[i].row_stride;
      blocks += tiles[i] * n;
    }
    b.items = make_div(static_cast<uint32_t>(n));
    b.parents += n0 * a.K;
    if (b.lengths != nullptr) b.lengths += n0;
    hipLaunchKernelGGL((beam_move_kernel<KMAX, W, U>), dim3(static_cast<unsigned>(blocks)), dim3(kMoveThreads), 0,
                       stream, b);
    if (const hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

}  // namespace

bool beam_state_fits(const BeamState& s, int K) {
  if (s.run > INT32_MAX) return false;
  return row_bytes(s) / column_bytes(s, K) < (uint64_t{1} << 31);
}

hipError_t launch_beam_reorder(const BeamState* states, int count, const int32_t* parents, int64_t N, int K,
                               const int32_t* lengths, hipStream_t stream) {
  // states of one column width share a launch
  for (const int w : {16, 4, 2, 1}) {
    MoveArgs a{};
    int held = 0;
    for (int i = 0; i < count; ++i) {
      const BeamState& s = states[i];
      if (column_bytes(s, K) != w) continue;
      MoveState& m = a.state[held++];
      m.data = s.data;
      m.row_stride = s.row_stride;
      for (int k = 0; k < 3; ++k) m.stride[k] = s.stride[k];
      m.position_stride = s.position_stride;
      const bool joined = s.positions == 1 || s.position_stride == s.run;
      const uint32_t per = static_cast<uint32_t>(s.positions * s.run / w);
      m.panel = make_div(per);
      m.size1 = make_div(static_cast<uint32_t>(s.size[1]));
      m.size2 = make_div(static_cast<uint32_t>(s.size[2]));
      m.run = joined ? Div{0, 0, 0} : make_div(static_cast<uint32_t>(s.run / w));
      m.columns = static_cast<uint32_t>(per * static_cast<uint64_t>(s.size[0] * s.size[1] * s.size[2]));
      m.run_bytes = static_cast<uint32_t>(s.run);
    }
    if (held == 0) continue;
    a.K = K;
    a.parents = parents;
    a.lengths = lengths;
    hipError_t e;
    if (w == 16) {
      if (K <= 4) e = move_all<4, 16, 4>(a, held, N, stream);
      else if (K <= 8) e = move_all<8, 16, 2>(a, held, N, stream);
      else if (K <= 16) e = move_all<16, 16, 1>(a, held, N, stream);
      else e = move_all<32, 16, 1>(a, held, N, stream);
    } else if (w == 4) {
      e = K <= 32 ? move_all<32, 4, 1>(a, held, N, stream) : move_all<128, 4, 1>(a, held, N, stream);
    } else {
      e = w == 2 ? move_all<128, 2, 1>(a, held, N, stream) : move_all<128, 1, 1>(a, held, N, stream);
    }
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace tkp
