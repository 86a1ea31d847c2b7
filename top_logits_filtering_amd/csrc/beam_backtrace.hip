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
//
// Dependent steps bound it, not its bytes: 100 steps of 4 prompts and 4 beams take
// 7.4 us on one MI355X; 2048 steps of 64 prompts and 8 beams (10.5 MB) 14.6, where
// a first form with one level of maps, formed from loads one at a time, took 45. A
// row of that history is 2 KB of which a prompt has 32 bytes, so a workgroup reads
// 2048 cache lines for its parents and again for its tokens.

#include "beam.h"
#include "device_common.h"

namespace tkp {
namespace {

constexpr int kTraceThreads = 1024;
constexpr int kSegment = 16;        // steps of a segment, and segments of a group
constexpr int kTracePaths = 32;     // hypotheses of a workgroup at most
constexpr int kTraceBytes = 49152;  // parents and paths of a piece
constexpr int kTraceBeams = 128;
constexpr int kRowMost = kTraceBeams + 4;
constexpr int kMapBytes = kTraceBytes / kSegment + kSegment * kRowMost;
constexpr int kGroupBytes = kMapBytes / kSegment + kRowMost;
constexpr int kTraceUnroll = 4;
constexpr int kTraceTarget = 256;   // workgroups wanted
constexpr int kDies = 8;

// Bytes of a step's parents: K beams, and at K the beam "nowhere", which stays nowhere.
__host__ __device__ constexpr int row_bytes_of(int K) { return (K + 4) & ~3; }

struct TraceSmem {
  alignas(16) uint8_t bytes[kTraceBytes];
  // beam before a segment (a group), by the beam in its last step
  alignas(16) uint8_t map[kMapBytes];
  uint8_t group_map[kGroupBytes];
  // a path's beam in the last step of a segment (a group); nowhere where it has not begun
  uint8_t entry[kMapBytes];
  uint8_t group_entry[kGroupBytes];
  uint8_t begin[kTracePaths];  // the beam at which a path begins
  uint8_t at[kTracePaths];     // its beam before what was passed last
  int end[kTracePaths];        // its last step
};

__global__ __launch_bounds__(kTraceThreads) void beam_backtrace_kernel(BeamBacktraceArgs a, Div beams, Div quads,
                                                                       Div tiles, int paths, Div piece,
                                                                       int64_t step_stride) {
  __shared__ TraceSmem sm;
  const int tid = threadIdx.x;
  // Neighbouring prompts share cache lines of the history, and workgroups go to
  // the 8 dies in turn: each die takes a run of prompts (14.6 us; 20.0 in turn).
  const uint32_t block = (blockIdx.x % kDies) * (gridDim.x / kDies) + blockIdx.x / kDies;
  const uint32_t item32 = quotient(block, tiles);
  if (item32 >= a.N) return;
  const int64_t item = item32;
  const int m0 = static_cast<int>(block - item32 * tiles.d) * paths;
  const int M = a.M - m0 < paths ? a.M - m0 : paths;
  const int K = a.K, T = static_cast<int>(a.T), row = row_bytes_of(K);
  const int steps = static_cast<int>(piece.d);
  uint8_t* parent = sm.bytes;              // [steps][row]
  uint8_t* path = sm.bytes + steps * row;  // [M][steps]
  const int64_t at0 = item * K;

  if (tid < M) {
    const int64_t h = item * a.M + m0 + tid;
    int len = a.lengths != nullptr ? a.lengths[h] : T;
    len = len < 0 ? 0 : (len > T ? T : len);
    const int b = a.beams != nullptr ? a.beams[h] : m0 + tid;
    sm.end[tid] = len - 1;
    sm.begin[tid] = static_cast<uint8_t>(b >= 0 && b < K ? b : K);
    sm.at[tid] = static_cast<uint8_t>(K);
  }

  for (int t1 = T; t1 > 0; t1 -= steps) {  // the piece [t0, t1), filled up with steps that change nothing
    const int t0 = t1 > steps ? t1 - steps : 0;
    const int n = t1 - t0;
    const int segs = (n + kSegment - 1) / kSegment, groups = (segs + kSegment - 1) / kSegment;
    lds_barrier();
    const int32_t* __restrict__ from = a.parents + t0 * step_stride + at0;
    auto byte_of = [&](int p) -> uint32_t { return p >= 0 && p < K ? p : K; };
    if (quads.d != 0) {  // four beams at a time, if aligned: 14.6 us, 16.0 one at a time
      const int count = n * static_cast<int>(quads.d);
      for (int f0 = tid; f0 < count; f0 += kTraceUnroll * kTraceThreads) {
        int4 p[kTraceUnroll];
#pragma unroll
        for (int u = 0; u < kTraceUnroll; ++u) {
          const int f = f0 + u * kTraceThreads;
          const int t = static_cast<int>(quotient(static_cast<uint32_t>(f), quads));
          p[u] = int4{0, 0, 0, 0};
          if (f < count)
            p[u] = *reinterpret_cast<const int4*>(from + t * step_stride + (f - t * static_cast<int>(quads.d)) * 4);
        }
#pragma unroll
        for (int u = 0; u < kTraceUnroll; ++u) {
          const int f = f0 + u * kTraceThreads;
          const int t = static_cast<int>(quotient(static_cast<uint32_t>(f), quads));
          if (f < count)
            *reinterpret_cast<uint32_t*>(parent + t * row + (f - t * static_cast<int>(quads.d)) * 4) =
                byte_of(p[u].x) | byte_of(p[u].y) << 8 | byte_of(p[u].z) << 16 | byte_of(p[u].w) << 24;
        }
      }
    } else {
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
          const int t = static_cast<int>(quotient(static_cast<uint32_t>(f), beams));
          if (f < n * K) parent[t * row + (f - t * K)] = static_cast<uint8_t>(byte_of(p[u]));
        }
      }
    }
    for (int t = tid; t < segs * kSegment; t += kTraceThreads) {
      if (t < n) {
        parent[t * row + K] = static_cast<uint8_t>(K);
      } else {
        for (int k = 0; k <= K; ++k) parent[t * row + k] = static_cast<uint8_t>(k);
      }
    }
    for (int s = segs + tid; s < groups * kSegment; s += kTraceThreads)
      for (int k = 0; k <= K; ++k) sm.map[s * row + k] = static_cast<uint8_t>(k);
    lds_barrier();

    // the segments' maps, and each path's beam before the segment in which it begins
    for (int f = tid; f < segs * K + M; f += kTraceThreads) {
      const bool own = f >= segs * K;
      const int m = f - segs * K, e = own ? sm.end[m] - t0 : -1;
      if (own && (e < 0 || e >= n)) continue;
      const int s = own ? e / kSegment : static_cast<int>(quotient(static_cast<uint32_t>(f), beams));
      const int k = f - s * K, begin = own ? sm.begin[m] : K;
      int b = own ? K : k;
#pragma unroll
      for (int i = kSegment - 1; i >= 0; --i) {
        if (s * kSegment + i == e) b = begin;
        b = parent[(s * kSegment + i) * row + b];
      }
      if (own) sm.at[m] = static_cast<uint8_t>(b);
      else sm.map[s * row + k] = static_cast<uint8_t>(b);
    }
    for (int s = tid; s < segs; s += kTraceThreads) sm.map[s * row + K] = static_cast<uint8_t>(K);
    lds_barrier();
    // the same with groups, whose steps are segments
    for (int f = tid; f < groups * K + M; f += kTraceThreads) {
      const bool own = f >= groups * K;
      const int m = f - groups * K, e = own ? sm.end[m] - t0 : -1;
      if (own && (e < 0 || e >= n)) continue;
      const int s = own ? e / kSegment : -1;
      const int g = own ? s / kSegment : static_cast<int>(quotient(static_cast<uint32_t>(f), beams));
      const int k = f - g * K, begin = own ? sm.at[m] : K;
      int b = own ? K : k;
#pragma unroll
      for (int i = kSegment - 1; i >= 0; --i) {
        const int q = g * kSegment + i;
        const int next = sm.map[q * row + b];
        if (own && q < segs) sm.entry[q * M + m] = static_cast<uint8_t>(b);
        b = q == s ? begin : next;
      }
      if (own) sm.at[m] = static_cast<uint8_t>(b);
      else sm.group_map[g * row + k] = static_cast<uint8_t>(b);
    }
    for (int g = tid; g < groups; g += kTraceThreads) sm.group_map[g * row + K] = static_cast<uint8_t>(K);
    lds_barrier();
    // a path's way through the groups that it passes from end to end
    if (tid < M) {
      const int e = sm.end[tid] - t0;
      int g = e >= n ? groups - 1 : (e < 0 ? -1 : e / (kSegment * kSegment) - 1);
      int b = sm.at[tid];
      for (; g >= 0; --g) {
        sm.group_entry[g * M + tid] = static_cast<uint8_t>(b);
        b = sm.group_map[g * row + b];
      }
      sm.at[tid] = static_cast<uint8_t>(b);
    }
    lds_barrier();
    // its way through their segments
    for (int f = tid; f < groups * M; f += kTraceThreads) {
      const int g = f / M, m = f - g * M, e = sm.end[m] - t0;
      if (e >= n || e / (kSegment * kSegment) > g) {
        int b = sm.group_entry[g * M + m];
#pragma unroll
        for (int i = kSegment - 1; i >= 0; --i) {
          const int q = g * kSegment + i;
          if (q < segs) sm.entry[q * M + m] = static_cast<uint8_t>(b);
          b = sm.map[q * row + b];
        }
      }
    }
    lds_barrier();
    // and through their steps
    for (int f = tid; f < segs * M; f += kTraceThreads) {
      const int s = f / M, m = f - s * M, begin = sm.begin[m];
      int e = sm.end[m] - t0;
      if (e >= n) e = INT32_MAX;  // it begins behind the piece, not in the steps that fill it up
      int b = e >= (s + 1) * kSegment ? sm.entry[s * M + m] : K;
#pragma unroll
      for (int i = kSegment - 1; i >= 0; --i) {
        const int t = s * kSegment + i;
        if (t == e) b = begin;
        if (t < n) path[m * steps + t] = static_cast<uint8_t>(b);
        b = parent[t * row + b];
      }
    }
    lds_barrier();

    const int32_t* __restrict__ tokens = a.tokens + t0 * step_stride + at0;
    int32_t* __restrict__ out = a.out + (item * a.M + m0) * a.T + t0;
    for (int f0 = tid; f0 < M * steps; f0 += kTraceUnroll * kTraceThreads) {
      int32_t v[kTraceUnroll];
#pragma unroll
      for (int u = 0; u < kTraceUnroll; ++u) {
        const int f = f0 + u * kTraceThreads, m = static_cast<int>(quotient(static_cast<uint32_t>(f), piece));
        const int t = f - m * steps;
        const int b = f < M * steps && t < n ? path[f] : K;
        v[u] = b < K ? tokens[t * step_stride + b] : a.pad;
      }
#pragma unroll
      for (int u = 0; u < kTraceUnroll; ++u) {
        const int f = f0 + u * kTraceThreads, m = static_cast<int>(quotient(static_cast<uint32_t>(f), piece));
        const int t = f - m * steps;
        if (f < M * steps && t < n) out[m * a.T + t] = v[u];
      }
    }
  }
}

}  // namespace

hipError_t launch_beam_backtrace(const BeamBacktraceArgs& a, hipStream_t stream) {
  // Few prompts: their hypotheses are spread over more workgroups, each of
  // which forms the maps again (they come from the same cache lines). 64 prompts of
  // 8: 64 workgroups 19.8 us, 128 15.6, 256 14.6, 512 23.7.
  int64_t paths = (a.N * a.M + kTraceTarget - 1) / kTraceTarget;
  paths = paths < kTracePaths ? paths : kTracePaths;
  paths = paths < a.M ? paths : a.M;
  const int tiles = static_cast<int>((a.M + paths - 1) / paths);
  // steps of a piece, whole segments
  const int64_t fit = kTraceBytes / (row_bytes_of(a.K) + paths) / kSegment * kSegment;
  const int64_t whole = (a.T + kSegment - 1) / kSegment * kSegment;
  const int steps = static_cast<int>(whole < fit ? whole : fit);
  const bool aligned = a.K % 4 == 0 && reinterpret_cast<uintptr_t>(a.parents) % 16 == 0;
  const Div quads = aligned ? make_div(static_cast<uint32_t>(a.K / 4)) : Div{0, 0, 0};
  const int64_t most = int64_t{1} << 21;  // a grid holds below 2^32 threads
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
                       stream, b, make_div(static_cast<uint32_t>(a.K)), quads, make_div(static_cast<uint32_t>(tiles)),
                       static_cast<int>(paths), make_div(static_cast<uint32_t>(steps)), a.N * a.K);
    if (const hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

}  // namespace tkp
