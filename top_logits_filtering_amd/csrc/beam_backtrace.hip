// Sequences out of a beam search's history. Hypothesis m of prompt n ends in
// step e = lengths[n][m] - 1 at beam beams[n][m]; its token of step t is
// tokens[t][n][b_t] with b_{t-1} = parents[t][n][b_t].
//
// Followed step by step that is a chain of T dependent reads. Each step is a
// map of K beams, and maps compose, so time is cut into segments: every
// segment's map is formed by itself (a thread per segment and start beam), a
// path hops from segment to segment through them, and then every segment's
// part of the path is walked by a thread of its own. The walks read parents as
// bytes from shared memory; tokens are fetched at the end, side by side. A
// history that does not fit is taken in pieces from its end.

#include "beam.h"
#include "device_common.h"

namespace tkp {
namespace {

constexpr int kTraceThreads = 512;
constexpr int kTraceBytes = 57344;  // parents and paths of a piece
constexpr int kTracePaths = 32;     // hypotheses of a workgroup
constexpr int kSegment = 32;        // steps of a segment at least
constexpr int kSegments = 64;       // segments of a piece at most
constexpr int kTraceBeams = 128;
constexpr uint8_t kNowhere = 255;

struct TraceSmem {
  uint8_t bytes[kTraceBytes];
  uint8_t map[kSegments * kTraceBeams];   // beam before a segment, by the beam in its last step
  uint8_t entry[kSegments * kTracePaths]; // a path's beam in a segment's last step (or where it begins)
  uint8_t at[kTracePaths];                // a path's beam in the last step of the piece
  int end[kTracePaths];                   // a path's last step
};

__global__ __launch_bounds__(kTraceThreads) void beam_backtrace_kernel(BeamBacktraceArgs a, int tiles, int steps) {
  __shared__ TraceSmem sm;
  const int tid = threadIdx.x;
  const int64_t item = blockIdx.x / static_cast<unsigned>(tiles);
  const int m0 = static_cast<int>(blockIdx.x % static_cast<unsigned>(tiles)) * kTracePaths;
  const int M = a.M - m0 < kTracePaths ? a.M - m0 : kTracePaths;
  const int K = a.K, T = static_cast<int>(a.T);
  uint8_t* parent = sm.bytes;              // [steps][K]
  uint8_t* path = sm.bytes + steps * K;    // [M][steps]
  const int64_t at0 = item * K, step_stride = a.N * K;

  if (tid < M) {
    const int64_t h = item * a.M + m0 + tid;
    int len = a.lengths != nullptr ? a.lengths[h] : T;
    len = len < 0 ? 0 : (len > T ? T : len);
    sm.end[tid] = len - 1;
    sm.at[tid] = kNowhere;
  }

  for (int t1 = T; t1 > 0; t1 -= steps) {  // the piece [t0, t1)
    const int t0 = t1 > steps ? t1 - steps : 0;
    const int n = t1 - t0;
    int seg = (n + kSegments - 1) / kSegments;
    seg = seg > kSegment ? seg : kSegment;
    const int segs = (n + seg - 1) / seg;
    __syncthreads();
    for (int f = tid; f < n * K; f += kTraceThreads) {
      const int t = f / K, k = f - t * K;
      const int p = a.parents[(t0 + t) * step_stride + at0 + k];
      parent[f] = p >= 0 && p < K ? static_cast<uint8_t>(p) : kNowhere;
    }
    __syncthreads();

    for (int f = tid; f < segs * K; f += kTraceThreads) {
      const int s = f / K;
      int b = f - s * K;
      const int last = (s + 1) * seg < n ? (s + 1) * seg : n;
      for (int t = last - 1; t >= s * seg && b != kNowhere; --t) b = parent[t * K + b];
      sm.map[s * kTraceBeams + f - s * K] = static_cast<uint8_t>(b);
    }
    __syncthreads();

    if (tid < M) {
      const int e = sm.end[tid] - t0;  // last step within the piece (n - 1 and more: it goes on behind)
      int b = sm.at[tid];
      for (int s = segs - 1; s >= 0; --s) {
        uint8_t in = kNowhere;
        const int last = (s + 1) * seg < n ? (s + 1) * seg : n;
        if (e >= s * seg) {
          if (e < last) {  // the path begins here
            const int64_t h = item * a.M + m0 + tid;
            b = a.beams != nullptr ? a.beams[h] : m0 + tid;
            if (b < 0 || b >= K) b = kNowhere;
            in = static_cast<uint8_t>(b);
            for (int t = e; t >= s * seg && b != kNowhere; --t) b = parent[t * K + b];
          } else {
            in = static_cast<uint8_t>(b);
            if (b != kNowhere) b = sm.map[s * kTraceBeams + b];
          }
        }
        sm.entry[s * kTracePaths + tid] = in;
      }
      sm.at[tid] = static_cast<uint8_t>(b);
    }
    __syncthreads();

    for (int f = tid; f < segs * M; f += kTraceThreads) {
      const int s = f / M, m = f - s * M;
      int b = sm.entry[s * kTracePaths + m];
      const int e = sm.end[m] - t0;
      const int last = ((s + 1) * seg < n ? (s + 1) * seg : n) - 1;
      for (int t = last; t >= s * seg; --t) {
        if (t > e) {
          path[m * steps + t] = kNowhere;
        } else {
          path[m * steps + t] = static_cast<uint8_t>(b);
          if (b != kNowhere) b = parent[t * K + b];
        }
      }
    }
    __syncthreads();

    for (int m = 0; m < M; ++m) {
      int32_t* out = a.out + (item * a.M + m0 + m) * a.T + t0;
      for (int t = tid; t < n; t += kTraceThreads) {
        const int b = path[m * steps + t];
        out[t] = b != kNowhere ? a.tokens[(t0 + t) * step_stride + at0 + b] : a.pad;
      }
    }
  }
}

}  // namespace

hipError_t launch_beam_backtrace(const BeamBacktraceArgs& a, hipStream_t stream) {
  const int tiles = (a.M + kTracePaths - 1) / kTracePaths;
  const int paths = a.M < kTracePaths ? a.M : kTracePaths;
  const int64_t fit = kTraceBytes / (a.K + paths);
  const int steps = static_cast<int>(a.T < fit ? a.T : fit);
  const int64_t most = int64_t{1} << 22;  // a grid holds below 2^32 threads
  const int64_t per = most / tiles > 0 ? most / tiles : 1;
  for (int64_t i = 0; i < a.N; i += per) {
    const int64_t items = a.N - i < per ? a.N - i : per;
    BeamBacktraceArgs b = a;
    b.tokens += i * a.K;
    b.parents += i * a.K;
    if (b.beams != nullptr) b.beams += i * a.M;
    if (b.lengths != nullptr) b.lengths += i * a.M;
    b.out += i * a.M * a.T;
    hipLaunchKernelGGL(beam_backtrace_kernel, dim3(static_cast<unsigned>(items * tiles)), dim3(kTraceThreads), 0,
                       stream, b, tiles, steps);
    if (const hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

}  // namespace tkp
