// Sequences out of a beam search's history. Hypothesis m of prompt n ends in
// step e = lengths[n][m] - 1 at beam beams[n][m]; its token of step t is
// tokens[t][n][b_t] with b_{t-1} = parents[t][n][b_t].
//
// Followed step by step that is a chain of T dependent reads. Each step is a
// map of K beams, and maps compose, so time is cut twice, into segments of 16
// steps and groups of 16 segments: all segments' maps are formed at once (a
// thread per segment and start beam), then all groups' maps, a path hops from
// group to group, and the same downwards gives its beam in every step: five
// chains of about 16 reads of bytes in shared memory instead of one of T. Tokens are
// fetched at the end, side by side. A history that does not fit is taken in
// pieces from its end.

#include "beam.h"
#include "device_common.h"

namespace tkp {
namespace {

constexpr int kTraceThreads = 512;
constexpr int kSegment = 16;       // steps of a segment, and segments of a group
constexpr int kTracePaths = 32;    // hypotheses of a workgroup at most
constexpr int kTraceBytes = 49152; // parents and paths of a piece
constexpr int kMapBytes = kTraceBytes / kSegment + 512;
constexpr int kTraceBeams = 128;
constexpr int kDies = 8;
constexpr int kTraceUnroll = 8;
constexpr int kTraceTarget = 256;  // workgroups wanted
constexpr uint8_t kNowhere = 255;

struct TraceSmem {
  uint8_t bytes[kTraceBytes];
  // beam before a segment (a group), by the beam in its last step
  uint8_t map[kMapBytes];
  uint8_t group_map[kMapBytes / kSegment + kTraceBeams];
  // a path's beam in the last step of a segment (a group), or where it begins
  uint8_t entry[kMapBytes];
  uint8_t group_entry[kMapBytes / kSegment + kTracePaths];
  uint8_t begin[kTracePaths];  // the beam at which a path begins
  uint8_t at[kTracePaths];     // its beam before the segment, the group, the piece where it was last
  int end[kTracePaths];        // its last step
};

__global__ __launch_bounds__(kTraceThreads) void beam_backtrace_kernel(BeamBacktraceArgs a, Div beams, Div tiles,
                                                                       int paths, int steps, int64_t step_stride) {
  __shared__ TraceSmem sm;
  const int tid = threadIdx.x;
  // Neighbouring prompts share cache lines of the history, and workgroups go to
  // the 8 dies in turn: each die takes a run of prompts.
  const uint32_t block = (blockIdx.x % kDies) * (gridDim.x / kDies) + blockIdx.x / kDies;
  const uint32_t item32 = quotient(block, tiles);
  if (item32 >= a.N) return;
  const int64_t item = item32;
  const int m0 = static_cast<int>(block - item32 * tiles.d) * paths;
  const int M = a.M - m0 < paths ? a.M - m0 : paths;
  const int K = a.K, T = static_cast<int>(a.T);
  uint8_t* parent = sm.bytes;            // [steps][K]
  uint8_t* path = sm.bytes + steps * K;  // [M][steps]
  const int64_t at0 = item * K;

  if (tid < M) {
    const int64_t h = item * a.M + m0 + tid;
    int len = a.lengths != nullptr ? a.lengths[h] : T;
    len = len < 0 ? 0 : (len > T ? T : len);
    const int b = a.beams != nullptr ? a.beams[h] : m0 + tid;
    sm.end[tid] = len - 1;
    sm.begin[tid] = b >= 0 && b < K ? static_cast<uint8_t>(b) : kNowhere;
    sm.at[tid] = kNowhere;
  }

  for (int t1 = T; t1 > 0; t1 -= steps) {  // the piece [t0, t1)
    const int t0 = t1 > steps ? t1 - steps : 0;
    const int n = t1 - t0;
    const int segs = (n + kSegment - 1) / kSegment, groups = (segs + kSegment - 1) / kSegment;
    auto last_of = [&](int s) { return ((s + 1) * kSegment < n ? (s + 1) * kSegment : n) - 1; };
    auto last_seg = [&](int g) { return ((g + 1) * kSegment < segs ? (g + 1) * kSegment : segs) - 1; };
    lds_barrier();
    const int32_t* __restrict__ from = a.parents + t0 * step_stride + at0;
    for (int f0 = tid; f0 < n * K; f0 += kTraceUnroll * kTraceThreads) {
      int p[kTraceUnroll];
#pragma unroll
      for (int u = 0; u < kTraceUnroll; ++u) {
        const int f = f0 + u * kTraceThreads;
        const int t = static_cast<int>(quotient(static_cast<uint32_t>(f), beams));
        p[u] = f < n * K ? from[t * step_stride + (f - t * K)] : -1;
      }
#pragma unroll
      for (int u = 0; u < kTraceUnroll; ++u) {
        const int f = f0 + u * kTraceThreads;
        if (f < n * K) parent[f] = p[u] >= 0 && p[u] < K ? static_cast<uint8_t>(p[u]) : kNowhere;
      }
    }
    lds_barrier();

    // the segments' maps; and where the paths that begin in this piece are before their first segment
    for (int f = tid; f < segs * K + M; f += kTraceThreads) {
      if (f < segs * K) {
        const int s = static_cast<int>(quotient(static_cast<uint32_t>(f), beams));
        int b = f - s * K;
        for (int t = last_of(s); t >= s * kSegment && b != kNowhere; --t) b = parent[t * K + b];
        sm.map[f] = static_cast<uint8_t>(b);
      } else {
        const int m = f - segs * K, e = sm.end[m] - t0;
        if (e >= 0 && e < n) {
          int b = sm.begin[m];
          for (int t = e; t >= e / kSegment * kSegment && b != kNowhere; --t) b = parent[t * K + b];
          sm.at[m] = static_cast<uint8_t>(b);
        }
      }
    }
    lds_barrier();
    // the same with groups
    for (int f = tid; f < groups * K + M; f += kTraceThreads) {
      if (f < groups * K) {
        const int g = static_cast<int>(quotient(static_cast<uint32_t>(f), beams));
        int b = f - g * K;
        for (int s = last_seg(g); s >= g * kSegment && b != kNowhere; --s) b = sm.map[s * K + b];
        sm.group_map[f] = static_cast<uint8_t>(b);
      } else {
        const int m = f - groups * K, e = sm.end[m] - t0;
        if (e >= 0 && e < n) {
          const int first = e / kSegment;
          int b = sm.at[m];
          sm.entry[first * M + m] = sm.begin[m];
          for (int s = first - 1; s >= first / kSegment * kSegment; --s) {
            sm.entry[s * M + m] = static_cast<uint8_t>(b);
            if (b != kNowhere) b = sm.map[s * K + b];
          }
          sm.at[m] = static_cast<uint8_t>(b);
        }
      }
    }
    lds_barrier();
    // a path's way through the groups that it passes from end to end
    if (tid < M) {
      const int e = sm.end[tid] - t0;
      int g = e >= n ? groups - 1 : (e < 0 ? -1 : e / (kSegment * kSegment) - 1);
      int b = sm.at[tid];
      for (; g >= 0; --g) {
        sm.group_entry[g * M + tid] = static_cast<uint8_t>(b);
        if (b != kNowhere) b = sm.group_map[g * K + b];
      }
      sm.at[tid] = static_cast<uint8_t>(b);
    }
    lds_barrier();
    // its way through their segments
    for (int f = tid; f < groups * M; f += kTraceThreads) {
      const int g = f / M, m = f - g * M, e = sm.end[m] - t0;
      if (e >= n || e / (kSegment * kSegment) > g) {
        int b = sm.group_entry[g * M + m];
        for (int s = last_seg(g); s >= g * kSegment; --s) {
          sm.entry[s * M + m] = static_cast<uint8_t>(b);
          if (b != kNowhere) b = sm.map[s * K + b];
        }
      }
    }
    lds_barrier();
    // and through their steps
    for (int f = tid; f < segs * M; f += kTraceThreads) {
      const int s = f / M, m = f - s * M, e = sm.end[m] - t0;
      int b = e >= s * kSegment ? sm.entry[s * M + m] : kNowhere;
      for (int t = last_of(s); t >= s * kSegment; --t) {
        path[m * steps + t] = t > e ? kNowhere : static_cast<uint8_t>(b);
        if (t <= e && b != kNowhere) b = parent[t * K + b];
      }
    }
    lds_barrier();

    const int32_t* __restrict__ tokens = a.tokens + t0 * step_stride + at0;
    for (int m = 0; m < M; ++m) {
      int32_t* __restrict__ out = a.out + (item * a.M + m0 + m) * a.T + t0;
      for (int s0 = tid; s0 < n; s0 += kTraceUnroll * kTraceThreads) {
        int32_t v[kTraceUnroll];
#pragma unroll
        for (int u = 0; u < kTraceUnroll; ++u) {
          const int t = s0 + u * kTraceThreads;
          const int b = t < n ? path[m * steps + t] : kNowhere;
          v[u] = b != kNowhere ? tokens[t * step_stride + b] : a.pad;
        }
#pragma unroll
        for (int u = 0; u < kTraceUnroll; ++u)
          if (s0 + u * kTraceThreads < n) out[s0 + u * kTraceThreads] = v[u];
      }
    }
  }
}

}  // namespace

hipError_t launch_beam_backtrace(const BeamBacktraceArgs& a, hipStream_t stream) {
  // Few prompts: their hypotheses are spread over more workgroups, each of
  // which forms the maps again (they come from the same cache lines).
  int64_t paths = (a.N * a.M + kTraceTarget - 1) / kTraceTarget;
  paths = paths < kTracePaths ? paths : kTracePaths;
  paths = paths < a.M ? paths : a.M;
  const int tiles = static_cast<int>((a.M + paths - 1) / paths);
  const int64_t fit = kTraceBytes / (a.K + paths) / kSegment * kSegment;
  const int steps = static_cast<int>(a.T < fit ? a.T : fit);
  const int64_t most = int64_t{1} << 22;  // a grid holds below 2^32 threads
  const int64_t per = most / tiles > 0 ? most / tiles : 1;
  for (int64_t i = 0; i < a.N; i += per) {
    const int64_t items = a.N - i < per ? a.N - i : per;
    BeamBacktraceArgs b = a;
    b.N = items;
    b.tokens += i * a.K;
    b.parents += i * a.K;
    if (b.beams != nullptr) b.beams += i * a.M;
    if (b.lengths != nullptr) b.lengths += i * a.M;
    b.out += i * a.M * a.T;
    hipLaunchKernelGGL(beam_backtrace_kernel, dim3(static_cast<unsigned>((items * tiles + kDies - 1) / kDies * kDies)),
                       dim3(kTraceThreads), 0,
                       stream, b, make_div(static_cast<uint32_t>(a.K)), make_div(static_cast<uint32_t>(tiles)),
                       static_cast<int>(paths), steps, a.N * a.K);
    if (const hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

}  // namespace tkp
