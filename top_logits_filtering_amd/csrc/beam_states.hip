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
//
// Memory bounds it: each changed row written once and each of their parents read
// once. On one MI355X, rates of those bytes in columns of 16 bytes: 4 beams 2.4 GB
// in 410 us (5.9 TB/s), 6 beams 219 MB in one state 38 us (5.7), 17 and 32 beams 5.4
// and 5.1 TB/s; 64 and 128 beams, in columns of 4, 3.8 and 4.2, and 2.5 and 2.9
// where the length ends halfway. Few beams in narrow columns are bound by the number
// of loads and stores: 4 beams in columns of 4 bytes 2.0 to 2.7 TB/s, of 2 and of 1,
// which take the registers of 128 beams, 0.25 to 0.34 and 0.17. Four small states of
// one prompt take 4.2 us.

#include "beam.h"
#include "device_common.h"

namespace tkp {
namespace {

constexpr int kMoveThreads = 256;
constexpr int64_t kCacheBytes = int64_t{256} << 20;  // the last-level cache

// A state cut into panels (one index of each of the three axes) of columns.
struct MoveState {
  char* data;
  int64_t row_stride;
  int64_t stride[3];
  int64_t position_stride;
  Div panel;           // columns per panel
  Div size1, size2;
  Div run;             // columns per run; run.d == 0: positions are contiguous
  Div tiles;           // workgroups per prompt
  uint32_t columns;    // panels * columns per panel
  uint32_t run_bytes;  // bytes of a position, for the length's end
};

struct MoveArgs {
  uint32_t first[kMaxStates];  // each state's first block; the largest number behind the last state
  MoveState state[kMaxStates];
  int K;
  const int32_t* parents;
  const int32_t* lengths;
};

template <int W>
struct Column;
template <>
struct Column<16> { using type = uint32_t __attribute__((ext_vector_type(4))); };
template <>
struct Column<4> { using type = uint32_t; };
template <>
struct Column<2> { using type = uint16_t; };
template <>
struct Column<1> { using type = uint8_t; };

// One tile of 256 columns of one state and prompt. KMAX: beams held; W: bytes of
// a column; NT: reads that leave no copy in the caches. Writes never do: the rows
// are next read by another step. (A thread with 2, 4 or 8 columns, to read the
// parents' numbers less often, took 425, 456 and 482 us where this takes 411.)
template <int KMAX, int W, bool NT>
__global__ __launch_bounds__(kMoveThreads) void beam_move_kernel(const MoveArgs a) {
  using col_t = typename Column<W>::type;
  int si = 0;
#pragma unroll
  for (int i = 1; i < kMaxStates; ++i) si += blockIdx.x >= a.first[i] ? 1 : 0;
  const MoveState& s = a.state[si];
  const uint32_t local = blockIdx.x - a.first[si];
  const uint32_t item32 = quotient(local, s.tiles);
  const uint32_t tile = local - item32 * s.tiles.d;
  const int64_t item = item32;

  const int64_t len = a.lengths != nullptr ? a.lengths[item] : INT64_MAX;
  if (len <= 0) return;
  // lane b (and 64 + b) holds beam b's parent, K where the beam stays
  const int lane = threadIdx.x % kWave;
  auto parent_of = [&](int b) -> int {
    const int p = b < a.K ? a.parents[item * a.K + b] : a.K;
    return p >= 0 && p != b ? p : a.K;
  };
  const int par0 = parent_of(lane), par1 = KMAX > kWave ? parent_of(kWave + lane) : a.K;

  // this thread's column: its byte offset, and how many of its bytes count
  const uint32_t c = tile * kMoveThreads + threadIdx.x;
  int64_t off = 0;
  int live = 0;
  if (c < s.columns) {
    const uint32_t p = quotient(c, s.panel);
    const uint32_t j = c - p * s.panel.d;
    const uint32_t p2 = quotient(p, s.size2), i2 = p - p2 * s.size2.d;
    const uint32_t i0 = quotient(p2, s.size1), i1 = p2 - i0 * s.size1.d;
    off = i0 * s.stride[0] + i1 * s.stride[1] + i2 * s.stride[2];
    if (s.run.d == 0) {  // positions follow each other: the panel is one piece
      const int64_t at = static_cast<int64_t>(j) * W;
      off += at;
      const int64_t end = len < INT32_MAX ? len * s.run_bytes : INT64_MAX;
      live = at >= end ? 0 : (end - at < W ? static_cast<int>(end - at) : W);
    } else {
      const uint32_t pos = quotient(j, s.run);
      off += pos * s.position_stride + static_cast<int64_t>(j - pos * s.run.d) * W;
      live = pos < len ? W : 0;
    }
  }

  // Every parent is read once, and then written to all that follow it.
  char* base = s.data + item * a.K * s.row_stride + off;
  col_t val[KMAX];
#pragma unroll
  for (int p = 0; p < KMAX; ++p) {
    if (p < a.K && (__ballot(par0 == p) | __ballot(par1 == p)) != 0 && live > 0) {
      const col_t* from = reinterpret_cast<const col_t*>(base + p * s.row_stride);
      val[p] = NT ? __builtin_nontemporal_load(from) : *from;
    }
  }
  auto put = [&](char* to, int p) __attribute__((always_inline)) {
    if (live == W) {
      __builtin_nontemporal_store(val[p], reinterpret_cast<col_t*>(to));
    } else if constexpr (W == 16) {  // the length ends inside: whole words up to it
      uint32_t* w = reinterpret_cast<uint32_t*>(to);
      if (live >= 4) w[0] = val[p].x;
      if (live >= 8) w[1] = val[p].y;
      if (live >= 12) w[2] = val[p].z;
    }
  };
#pragma unroll
  for (int p = 0; p < KMAX; ++p) {
    if (p < a.K) {
      for (uint64_t m = __ballot(par0 == p); m != 0; m &= m - 1) put(base + __builtin_ctzll(m) * s.row_stride, p);
      if constexpr (KMAX > kWave)
        for (uint64_t m = __ballot(par1 == p); m != 0; m &= m - 1)
          put(base + (kWave + __builtin_ctzll(m)) * s.row_stride, p);
    }
  }
}

int64_t low_bit(int64_t x) { return x & -x; }

// Bytes of a column: what every address is aligned to, at most 16, and for
// wide beams what fits the registers (2.4 GB of 4 beams take 410 us in columns of
// 16 bytes, 1170 in columns of 4). Columns of 16 bytes may reach past the
// length inside a piece of whole words; smaller ones never do, so that a piece whose
// positions follow each other in runs that are no whole words (keys held transposed
// in 16 bits, an odd head size) is moved 2 bytes or 1 at a time up to the length.
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
template <int KMAX, int W, bool NT>
hipError_t move_all(const MoveArgs& a, int count, int64_t N, hipStream_t stream) {
  constexpr int64_t kMost = int64_t{1} << 23;
  int64_t tiles[kMaxStates], sum = 0;
  for (int i = 0; i < count; ++i) {
    tiles[i] = (static_cast<int64_t>(a.state[i].columns) + kMoveThreads - 1) / kMoveThreads;
    sum += tiles[i];
  }
  if (sum > kMost && count > 1) {
    for (int i = 0; i < count; ++i) {
      MoveArgs one = a;
      one.state[0] = a.state[i];
      if (const hipError_t e = move_all<KMAX, W, NT>(one, 1, N, stream)) return e;
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
      b.state[i].tiles = make_div(static_cast<uint32_t>(tiles[i]));
      b.state[i].data += n0 * a.K * a.state[i].row_stride;
      blocks += tiles[i] * n;
    }
    b.parents += n0 * a.K;
    if (b.lengths != nullptr) b.lengths += n0;
    hipLaunchKernelGGL((beam_move_kernel<KMAX, W, NT>), dim3(static_cast<unsigned>(blocks)), dim3(kMoveThreads), 0,
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
                               const int32_t* lengths, int64_t bytes, hipStream_t stream) {
  const bool streamed = bytes > kCacheBytes;
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
      // Calls on more than the last-level cache holds read past it: 2.1 GB in
      // 32 states take 410 us so and 448 us otherwise, 194 MB in one state 48
      // and 39 us.
      // Room for 16 beams costs 4 nothing (411 us either way), room for 32 leaves
      // fewer waves (562 us).
      if (streamed)
        e = K <= 16 ? move_all<16, 16, true>(a, held, N, stream) : move_all<32, 16, true>(a, held, N, stream);
      else
        e = K <= 16 ? move_all<16, 16, false>(a, held, N, stream) : move_all<32, 16, false>(a, held, N, stream);
    } else if (w == 4) {
      e = K <= 32 ? move_all<32, 4, false>(a, held, N, stream) : move_all<128, 4, false>(a, held, N, stream);
    } else {
      e = w == 2 ? move_all<128, 2, false>(a, held, N, stream) : move_all<128, 1, false>(a, held, N, stream);
    }
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace tkp
