// Beam search selection: the n best continuations over K beams and V tokens.
//
// With c[b] the accumulated log-probability of beam b and x[b] its logits,
//   L[b] = log sum_v exp x[b,v],   s[b,v] = c[b] + x[b,v] - L[b],
// and candidates are ranked by s[b,v] * w[b] (descending), then by beam, then
// by logit (descending), then by token. Within a beam that is the order of
// (logit, token), so the n best of a prompt are among the n best of each beam:
//   1. beam_chunk_kernel splits every row into chunks that fit a workgroup's
//      registers. A chunk is read once and leaves sum exp(x - ref) and its n
//      best (logit, token) in descending order.
//   2. beam_merge_kernel, one workgroup per prompt, joins the chunks' sums to
//      L[b] and picks the n best of all lists.
//
// L[b] is formed in 64 bits: parents and tokens are whole numbers whose order
// between beams hangs on c[b] - L[b], and an error of fp32's size (1e-7)
// would swap candidates that lie as close. FP64 vector instructions run at
// the rate of unpacked FP32 ones on gfx950, so exp costs the same chain of
// multiply-adds either way: exp(x) = 2^k exp(f), k = rint(x / ln 2),
// |f| <= ln 2 / 2, and exp(f) is a polynomial of degree 7, found by Remez
// exchange for the smallest relative error (4.0e-11).

#include <float.h>

#include "beam.h"
#include "device_common.h"
#include "reg_tile.h"

namespace tkp {
namespace {

constexpr int kChunkThreads = 256;
constexpr int kChunkWaves = kChunkThreads / kWave;
constexpr int kChunkCap = 1024;   // candidate slots of a chunk
constexpr int kMaxVecs = 16;      // vectors per thread at most
constexpr int kMergeThreads = 512;
constexpr int kMergeCap = 2048;   // candidate slots of a prompt
constexpr int kHeads = 512;       // group maxima that bound a prompt's candidates
constexpr int kMaxBeams = 128;
constexpr int kTokenBits = 20;

// sum exp(x - ref) over a chunk; bad: a NaN or +inf was among the logits.
struct ChunkStat {
  double sum;
  float ref;
  int bad;
};

// Monotone image of a float (IEEE order, -0 as +0); 0 is below every value's.
__device__ __forceinline__ uint32_t order_key(float x) { return F32T::key(__float_as_uint(x)); }
__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float(F32T::raw_of_key(k)); }

// Monotone image of a finite double (-0 as +0).
__device__ __forceinline__ uint64_t order_key64(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x + 0.0);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

// (logit, token) as one number: a larger logit first, then a lower token.
__device__ __forceinline__ uint64_t pack(uint32_t key, uint32_t token) {
  return (static_cast<uint64_t>(key) << 32) | (0xFFFFFFFFu - token);
}

// exp(y) for |y| <= 1100 (finite result for y <= 709).
__device__ __forceinline__ double exp64(double y) {
  constexpr double kMagic = 6755399441055744.0;  // 1.5 * 2^52: its low bits hold rint()
  const double nm = __builtin_fma(y, 1.4426950408889634074, kMagic);
  const int k = static_cast<int>(__builtin_bit_cast(uint64_t, nm));
  const double f = __builtin_fma(nm - kMagic, -0.69314718055994530942, y);
  double p = 0.00019775160531026297389;
  p = __builtin_fma(p, f, 0.0013948195139022652005);
  p = __builtin_fma(p, f, 0.0083335611766106098887);
  p = __builtin_fma(p, f, 0.041666225250020369325);
  p = __builtin_fma(p, f, 0.16666665125242092947);
  p = __builtin_fma(p, f, 0.50000001045984631318);
  p = __builtin_fma(p, f, 1.0000000002432869351);
  p = __builtin_fma(p, f, 0.99999999996165148826);
  const uint64_t u = __builtin_bit_cast(uint64_t, p);
  const uint32_t hi = static_cast<uint32_t>(u >> 32) + (static_cast<uint32_t>(k) << 20);
  return __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | static_cast<uint32_t>(u));
}

// The chunks' sums are taken of exp(x) itself while the chunk's maximum lies
// in [kLowMax, kHighMax], which no logit of a model leaves: then no maximum is
// needed before the sum. Terms are clamped to +-kHighMax, so 2^15 of them stay
// finite and what the clamp adds (exp(-650), also for -inf) is below 2^-140 of
// the largest. Other chunks are read and summed again, less their maximum.
constexpr float kHighMax = 650.0f;
constexpr float kLowMax = -550.0f;

__device__ __forceinline__ double exp_term(float x) {
  return exp64(static_cast<double>(__builtin_amdgcn_fmed3f(x, -kHighMax, kHighMax)));
}

// exp(x - ref) for x <= ref, both finite, or x = -inf.
__device__ __forceinline__ double exp_below(float x, float ref) {
  const double y = static_cast<double>(x) - static_cast<double>(ref);
  return y < -kHighMax ? 0.0 : exp64(y);
}

// Key bits that tell this dtype's values apart; the bits below them are all
// zeros for positive and all ones for negative values.
template <class DT>
constexpr int key_low_bits() {
  return DT::kPerVec == 4 ? 0 : (DT::kNegInf == 0xFF80u ? 16 : 13);
}

// A beam whose score or weight rules it out proposes nothing.
__device__ __forceinline__ bool beam_alive(float c, float w) {
  const uint32_t cb = __float_as_uint(c) & 0x7FFFFFFFu, wb = __float_as_uint(w);
  return cb < 0x7F800000u && wb > 0u && wb < 0x7F800000u;  // c finite, w finite and > 0
}

__device__ __forceinline__ uint32_t count_ballot(bool p) { return __builtin_popcountll(__ballot(p)); }

// A copy that the compiler cannot trace: what one traversal of the vectors
// derives from them (conversions, keys) is not kept in registers for the next.
__device__ __forceinline__ vec_t opaque(vec_t q) {
  asm volatile("" : "+v"(q));
  return q;
}

struct ChunkSmem {
  uint64_t list[kChunkCap];
  uint32_t key[kChunkThreads];
  double sum[kChunkWaves];
  uint32_t abs[kChunkWaves];
  uint32_t scan[kChunkWaves];
  uint32_t count;
};

// Exclusive prefix of v over the block; total: the block's sum.
__device__ __forceinline__ uint32_t block_excl(uint32_t v, uint32_t& total, ChunkSmem& sm) {
  const int wave = threadIdx.x / kWave;
  const uint32_t incl = wave_incl_scan_u32(v);
  __syncthreads();
  if (threadIdx.x % kWave == kWave - 1) sm.scan[wave] = incl;
  __syncthreads();
  uint32_t below = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kChunkWaves; ++w) {
    if (w < wave) below += sm.scan[w];
    total += sm.scan[w];
  }
  return below + incl - v;
}

template <class DT, int NV>
__global__ __launch_bounds__(kChunkThreads) void beam_chunk_kernel(BeamSelectArgs a, BeamSplit split, int64_t row0,
                                                                   ChunkStat* __restrict__ stats,
                                                                   uint64_t* __restrict__ lists) {
  using raw_t = typename DT::raw_t;
  constexpr int P = DT::kPerVec;
  constexpr int kLow = key_low_bits<DT>();
  __shared__ ChunkSmem sm;

  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int ch = static_cast<int>(blockIdx.x % static_cast<unsigned>(split.chunks));
  const int64_t row = row0 + blockIdx.x / static_cast<unsigned>(split.chunks);
  if (!beam_alive(a.scores[row], a.weights != nullptr ? a.weights[row] : 1.0f)) return;
  if (a.finished != nullptr && a.finished[row] != 0) return;

  // The row as elements before the first 16-byte boundary, whole vectors, and
  // the elements behind the last one; the few single elements are held one per
  // thread, in the first and the last chunk.
  const raw_t* rowp = static_cast<const raw_t*>(a.logits) + row * a.ld;
  int head = static_cast<int>((16u - (reinterpret_cast<uintptr_t>(rowp) & 15u)) & 15u) / static_cast<int>(sizeof(raw_t));
  head = head < a.V ? head : a.V;
  const int nfull = (a.V - head) / P;
  const int tail0 = head + nfull * P;
  const int v0 = ch * split.vecs;
  int cnt = nfull - v0;
  cnt = cnt < 0 ? 0 : (cnt < split.vecs ? cnt : split.vecs);
  const int first = head + v0 * P;  // token of the chunk's first vector

  const __amdgpu_buffer_rsrc_t rs = row_rsrc(rowp + (cnt > 0 ? first : 0), cnt * P);
  vec_t v[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i)
    v[i] = __builtin_amdgcn_raw_buffer_load_b128(rs, (i * kChunkThreads + tid) * 16, 0, kLoadPolicy);

  int te = -1;
  if (ch == 0 && tid < head) te = tid;
  if (ch == split.chunks - 1 && tid >= 16 && tid - 16 < a.V - tail0) te = tail0 + tid - 16;
  raw_t re = DT::kNegInf;
  if (te >= 0) re = rowp[te];
  const float xe = DT::value(re);

  if (tid == 0) sm.count = 0;
  // One pass: the sum of exp, the largest value, the largest magnitude (for NaN).
  constexpr uint32_t kAbs = P == 4 ? 0x7FFFFFFFu : 0x7FFF7FFFu;
  constexpr uint32_t kNeg = P == 4 ? static_cast<uint32_t>(DT::kNegInf)
                                   : static_cast<uint32_t>(DT::kNegInf) * 0x00010001u;
  using pair_t = uint16_t __attribute__((ext_vector_type(2)));
  double sum = exp_term(xe);
  float tm = xe;
  uint32_t am = re & kAbs;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (i * kChunkThreads + tid >= cnt) v[i] = vec_t{kNeg, kNeg, kNeg, kNeg};
    __builtin_amdgcn_sched_barrier(0);  // one vector's terms at a time, or their 64-bit values fill the registers
    double part = 0.0;
    const vec_t q = opaque(v[i]);
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const float x = DT::value(lane_of<raw_t>(q, j));
      part += exp_term(x);
      tm = fmaxf(tm, x);
    }
    sum += part;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t u = vword(q, w) & kAbs;
      if constexpr (P == 4) {
        am = am > u ? am : u;
      } else {
        am = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(pair_t, am),
                                                                    __builtin_bit_cast(pair_t, u)));
      }
    }
  }
  if constexpr (P != 4) am = (am & 0xFFFFu) > (am >> 16) ? (am & 0xFFFFu) : (am >> 16);

  const uint32_t tkey = tm > -INFINITY ? order_key(tm) : 0u;
  sm.key[tid] = tkey;
  sum = wave_sum_f64(sum);
  am = wave_max_u32(am);
  if (lane == 0) {
    sm.sum[wave] = sum;
    sm.abs[wave] = am;
  }
  __syncthreads();

  // Every wave holds all the threads' maxima, four per lane.
  const uint4 k4 = reinterpret_cast<const uint4*>(sm.key)[lane];
  uint32_t top = k4.x > k4.y ? k4.x : k4.y;
  top = top > k4.z ? top : k4.z;
  top = wave_max_u32(top > k4.w ? top : k4.w);
  sum = 0.0;
  am = 0;
#pragma unroll
  for (int w = 0; w < kChunkWaves; ++w) {
    sum += sm.sum[w];
    am = am > sm.abs[w] ? am : sm.abs[w];
  }
  constexpr uint32_t kInfBits = P == 4 ? 0x7F800000u : (DT::kNegInf & 0x7FFFu);
  const int64_t slot = row * split.chunks + ch;
  uint64_t* out = lists + slot * a.n;
  if (am > kInfBits || top >= order_key(INFINITY)) {  // a NaN or +inf: the beam proposes nothing
    if (tid == 0) stats[slot] = ChunkStat{0.0, 0.0f, 1};
    return;
  }
  // Rare paths read the chunk again rather than hold code and registers for it.
  auto again = [&](int i) __attribute__((always_inline)) -> vec_t {
    const vec_t q = __builtin_amdgcn_raw_buffer_load_b128(rs, (i * kChunkThreads + tid) * 16, 0, 0);
    return i * kChunkThreads + tid < cnt ? q : vec_t{kNeg, kNeg, kNeg, kNeg};
  };
  float ref = 0.0f;
  if (top == 0u) {
    sum = 0.0;  // nothing but -inf
  } else if (key_value(top) > kHighMax || key_value(top) < kLowMax) {
    ref = key_value(top);
    double part = exp_below(xe, ref);
#pragma unroll 1
    for (int i = 0; i * kChunkThreads < cnt; ++i) {
      const vec_t q = again(i);
#pragma unroll
      for (int j = 0; j < P; ++j) part += exp_below(DT::value(lane_of<raw_t>(q, j)), ref);
    }
    part = wave_sum_f64(part);
    __syncthreads();
    if (lane == 0) sm.sum[wave] = part;
    __syncthreads();
    sum = 0.0;
#pragma unroll
    for (int w = 0; w < kChunkWaves; ++w) sum += sm.sum[w];
  }
  if (tid == 0) stats[slot] = ChunkStat{sum, ref, 0};

  // The n-th largest of the threads' maxima is a lower bound of the chunk's
  // n-th largest value: largest T with at least n maxima >= T, bit by bit.
  const uint32_t n = static_cast<uint32_t>(a.n);
  uint32_t T = 0;
#pragma unroll 1
  for (int bit = 31; bit >= kLow; --bit) {
    const uint32_t t = T | (1u << bit);
    const uint32_t c = count_ballot(k4.x >= t) + count_ballot(k4.y >= t) + count_ballot(k4.z >= t) +
                       count_ballot(k4.w >= t);
    if (c >= n) T = t;
  }
  if (T == 0u) T = order_key(-FLT_MAX);  // fewer than n maxima: all finite values
  else if (!(T & 0x80000000u)) T |= (1u << kLow) - 1u;
  float bound = key_value(T);

  auto push = [&](float x, uint32_t token) __attribute__((always_inline)) {
    const uint32_t at = atomicAdd(&sm.count, 1u);
    if (at < kChunkCap) sm.list[at] = pack(order_key(x), token);
  };
  if (xe >= bound) push(xe, static_cast<uint32_t>(te));
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const vec_t q = opaque(v[i]);
    float m = DT::value(lane_of<raw_t>(q, 0));
#pragma unroll
    for (int j = 1; j < P; ++j) m = fmaxf(m, DT::value(lane_of<raw_t>(q, j)));
    if (m >= bound) {
      const uint32_t token = static_cast<uint32_t>(first + (i * kChunkThreads + fresh_tid()) * P);
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const float x = DT::value(lane_of<raw_t>(q, j));
        if (x >= bound) push(x, token + j);
      }
    }
  }
  __syncthreads();
  uint32_t M = sm.count;

  if (M > kChunkCap) {
    // Many values at or above the bound: find the n-th largest value exactly,
    // list what lies above it, then the equal ones in the order of their tokens.
    auto key_of = [](raw_t r) -> uint32_t {
      const float x = DT::value(r);
      return x >= -FLT_MAX ? order_key(x) : 0u;
    };
    auto count_from = [&](uint32_t t) __attribute__((always_inline)) -> uint32_t {
      uint32_t c = key_of(re) >= t ? 1u : 0u;
#pragma unroll 1
      for (int i = 0; i * kChunkThreads < cnt; ++i) {
        const vec_t q = again(i);
#pragma unroll
        for (int j = 0; j < P; ++j) c += key_of(lane_of<raw_t>(q, j)) >= t ? 1u : 0u;
      }
      uint32_t total;
      block_excl(c, total, sm);
      return total;
    };
    // first whether the bound itself is that value (fewer than n above it), as
    // where many are equal; else it is found bit by bit
    const uint32_t bound_key = T;
#pragma unroll 1
    for (int bit = 32; bit >= kLow; --bit) {
      const uint32_t c = count_from(bit == 32 ? bound_key + 1u : (T | (1u << bit)));
      if (bit == 32) {
        if (c < n) break;
        T = 0;
      } else if (c >= n) {
        T |= 1u << bit;
      }
    }
    if (!(T & 0x80000000u)) T |= (1u << kLow) - 1u;
    __syncthreads();
    if (tid == 0) sm.count = 0;
    __syncthreads();
    auto push_above = [&](raw_t r, uint32_t token) __attribute__((always_inline)) {
      const uint32_t k = key_of(r);
      if (k > T) {
        const uint32_t at = atomicAdd(&sm.count, 1u);
        if (at < kChunkCap) sm.list[at] = pack(k, token);
      }
    };
    push_above(re, static_cast<uint32_t>(te));
#pragma unroll 1
    for (int i = 0; i * kChunkThreads < cnt; ++i) {
      const vec_t q = again(i);
      const uint32_t token = static_cast<uint32_t>(first + (i * kChunkThreads + tid) * P);
#pragma unroll
      for (int j = 0; j < P; ++j)
        push_above(lane_of<raw_t>(q, j), token + j);
    }
    __syncthreads();
    uint32_t have = sm.count;  // < n
    // equal values: the elements before the vectors, the vectors layer by layer, the elements behind
    auto push_equal = [&](uint32_t mask, uint32_t token) __attribute__((always_inline)) {
      uint32_t total;
      uint32_t at = have + block_excl(__builtin_popcount(mask), total, sm);
      for (uint32_t m = mask; m != 0u && at < n; m &= m - 1u, ++at)
        sm.list[at] = pack(T, token + static_cast<uint32_t>(__builtin_ctz(m)));
      have += total;
    };
    const bool equal_e = key_of(re) == T;
    push_equal(equal_e && te >= 0 && te < head ? 1u : 0u, static_cast<uint32_t>(te));
#pragma unroll 1
    for (int i = 0; i * kChunkThreads < cnt && have < n; ++i) {
      uint32_t mask = 0;
      const vec_t q = again(i);
#pragma unroll
      for (int j = 0; j < P; ++j) mask |= (key_of(lane_of<raw_t>(q, j)) == T ? 1u : 0u) << j;
      push_equal(mask, static_cast<uint32_t>(first + (i * kChunkThreads + tid) * P));
    }
    if (have < n) push_equal(equal_e && te >= tail0 ? 1u : 0u, static_cast<uint32_t>(te));
    M = have < n ? have : n;
    __syncthreads();
  }

  // The candidates are distinct numbers: each one's rank is the count of larger ones.
  for (uint32_t e = tid; e < M; e += kChunkThreads) {
    const uint64_t mine = sm.list[e];
    uint32_t r = 0;
    for (uint32_t j = 0; j < M; ++j) r += sm.list[j] > mine ? 1u : 0u;
    if (r < n) out[r] = mine;
  }
  for (uint32_t e = M + tid; e < n; e += kChunkThreads) out[e] = 0;
}

// A candidate of a prompt: the rank value's image, then beam, logit and token
// (59 bits) such that the larger number ranks first.
struct Cand {
  uint64_t hi, lo;
};
__device__ __forceinline__ bool above(const Cand& a, const Cand& b) {
  return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo);
}

struct MergeSmem {
  Cand list[kMergeCap];
  double ref[kMaxBeams];     // L = ref + rest; apart, as ref may be as large as the type goes
  double rest[kMaxBeams];
  double score[kMaxBeams];
  double weight[kMaxBeams];
  int state[kMaxBeams];      // 0: proposes nothing, 1: its lists, 2: finished
  uint32_t heads[kHeads];
  Cand best[kMergeThreads / kWave];
  uint32_t count;
  uint32_t more;
};

__global__ __launch_bounds__(kMergeThreads) void beam_merge_kernel(BeamSelectArgs a, int C, int64_t item0,
                                                                   const ChunkStat* __restrict__ stats,
                                                                   const uint64_t* __restrict__ lists) {
  __shared__ MergeSmem sm;
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int64_t item = item0 + blockIdx.x;
  const int K = a.K;
  const uint32_t n = static_cast<uint32_t>(a.n);

  // L of each beam from its chunks' sums: a wave per beam, lanes over chunks.
  for (int b = wave; b < K; b += kMergeThreads / kWave) {
    const int64_t row = item * K + b;
    const float c = a.scores[row], w = a.weights != nullptr ? a.weights[row] : 1.0f;
    int state = 0;
    double ref = 0.0, rest = 0.0;
    if (beam_alive(c, w)) {
      if (a.finished != nullptr && a.finished[row] != 0) {
        state = 2;
      } else {
        uint32_t rk = 0, bad = 0;
        for (int i = lane; i < C; i += kWave) {
          const ChunkStat s = stats[row * C + i];
          bad |= static_cast<uint32_t>(s.bad);
          if (s.sum > 0.0) rk = rk > order_key(s.ref) ? rk : order_key(s.ref);
        }
        rk = wave_max_u32(rk);
        bad = wave_max_u32(bad);
        ref = rk != 0 ? static_cast<double>(key_value(rk)) : 0.0;
        double sum = 0.0;
        for (int i = lane; i < C; i += kWave) {
          const ChunkStat s = stats[row * C + i];
          if (s.sum > 0.0) {
            const double d = s.ref - ref;
            sum += d == 0.0 ? s.sum : (d < -2000.0 ? 0.0 : s.sum * exp(d));
          }
        }
        sum = wave_sum_f64(sum);
        if (bad == 0 && sum > 0.0) {
          state = 1;
          rest = log(sum);
        }
      }
    }
    if (lane == 0) {
      sm.ref[b] = ref;
      sm.rest[b] = rest;
      sm.score[b] = c;
      sm.weight[b] = w;
      sm.state[b] = state;
    }
  }
  if (tid < kHeads) sm.heads[tid] = 0;
  if (tid == 0) {
    sm.count = 0;
    sm.more = 0;
  }
  __syncthreads();

  const int nl = K * C;  // lists of this prompt
  const int64_t list0 = item * nl;
  // Entry j of list q as a candidate; hi is 0 where there is none.
  auto cand = [&](int q, uint32_t j) -> Cand {
    const int b = q / C;
    const int st = sm.state[b];
    if (st == 0) return Cand{0, 0};
    const uint64_t beam = static_cast<uint64_t>(kMaxBeams - 1 - b) << (32 + kTokenBits);
    if (st == 2) {
      if (j != 0 || q != b * C) return Cand{0, 0};
      return Cand{order_key64(sm.score[b] * sm.weight[b]), beam};
    }
    const uint64_t e = lists[(list0 + q) * n + j];
    if (e == 0) return Cand{0, 0};
    const uint32_t key = static_cast<uint32_t>(e >> 32);
    const uint32_t back = ((1u << kTokenBits) - 1u) - (0xFFFFFFFFu - static_cast<uint32_t>(e));
    const double s = sm.score[b] + ((static_cast<double>(key_value(key)) - sm.ref[b]) - sm.rest[b]);
    return Cand{order_key64(s * sm.weight[b]), beam | (static_cast<uint64_t>(key) << kTokenBits) | back};
  };

  // A bound: the largest T that n of the lists' first entries reach (by the
  // upper half of the rank's image), over at most kHeads group maxima.
  const uint32_t deep = (n + nl - 1) / nl;  // entries of each list, so that there are n
  const uint32_t nh = deep * nl;
  uint32_t mine = 0;
  for (uint32_t f = tid; f < nh; f += kMergeThreads) {
    const uint32_t h = static_cast<uint32_t>(cand(static_cast<int>(f / deep), f % deep).hi >> 32);
    mine = mine > h ? mine : h;
  }
  sm.heads[tid] = mine;
  __syncthreads();
  uint32_t h[kHeads / kWave];
#pragma unroll
  for (int i = 0; i < kHeads / kWave; ++i) h[i] = sm.heads[i * kWave + lane];
  uint32_t T = 0;
#pragma unroll 1
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t t = T | (1u << bit);
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < kHeads / kWave; ++i) c += count_ballot(h[i] >= t);
    if (c >= n) T = t;
  }
  if (T == 0u) T = 1u;  // fewer than n: every candidate

  // Candidates from T on, in windows of entries while a list's last one still reaches it.
  const uint32_t window = nl < kMergeThreads ? kMergeThreads / nl : 1u;
  for (uint32_t j0 = 0; j0 < n; j0 += window) {
    const uint32_t wide = n - j0 < window ? n - j0 : window;
    bool more = false;
    for (uint32_t f = tid; f < wide * nl; f += kMergeThreads) {
      const uint32_t j = f % wide;
      const Cand k = cand(static_cast<int>(f / wide), j0 + j);
      if (static_cast<uint32_t>(k.hi >> 32) >= T) {
        const uint32_t at = atomicAdd(&sm.count, 1u);
        if (at < kMergeCap) sm.list[at] = k;
        more |= j == wide - 1;
      }
    }
    if (!__syncthreads_or(more)) break;
  }
  __syncthreads();
  uint32_t M = sm.count;

  if (M > kMergeCap) {
    // More ties in the upper half than the list holds: take the best ones one
    // by one, each the largest candidate below the last.
    __syncthreads();
    Cand last{~0ull, ~0ull};
    uint32_t r = 0;
    for (; r < n; ++r) {
      Cand best{0, 0};
      for (uint32_t f = tid; f < n * static_cast<uint32_t>(nl); f += kMergeThreads) {
        const Cand k = cand(static_cast<int>(f / n), f % n);
        if (above(last, k) && above(k, best)) best = k;
      }
#pragma unroll
      for (int d = 1; d < kWave; d *= 2) {
        const Cand o{__shfl_xor(best.hi, d), __shfl_xor(best.lo, d)};
        if (above(o, best)) best = o;
      }
      __syncthreads();
      if (lane == 0) sm.best[wave] = best;
      __syncthreads();
      best = sm.best[0];
#pragma unroll
      for (int w = 1; w < kMergeThreads / kWave; ++w)
        if (above(sm.best[w], best)) best = sm.best[w];
      if (best.hi == 0) break;
      if (tid == 0) sm.list[r] = best;
      last = best;
    }
    M = r;
    __syncthreads();
  }

  // Ranks by counting; decode and write.
  for (uint32_t e = tid; e < M; e += kMergeThreads) {
    const Cand k = sm.list[e];
    uint32_t r = 0;
    for (uint32_t j = 0; j < M; ++j) r += above(sm.list[j], k) ? 1u : 0u;
    if (r < n) {
      const int b = kMaxBeams - 1 - static_cast<int>(k.lo >> (32 + kTokenBits));
      double s = sm.score[b];
      int32_t token = a.end_token;
      if (sm.state[b] == 1) {
        s += (static_cast<double>(key_value(static_cast<uint32_t>(k.lo >> kTokenBits))) - sm.ref[b]) - sm.rest[b];
        token = static_cast<int32_t>(((1u << kTokenBits) - 1u) - (static_cast<uint32_t>(k.lo) & ((1u << kTokenBits) - 1u)));
      }
      const int64_t o = item * n + r;
      a.out_scores[o] = static_cast<float>(s);
      a.out_parents[o] = b;
      a.out_tokens[o] = token;
    }
  }
  for (uint32_t e = M + tid; e < n; e += kMergeThreads) {
    const int64_t o = item * n + e;
    a.out_scores[o] = -INFINITY;
    a.out_parents[o] = -1;
    a.out_tokens[o] = -1;
  }
}

template <class DT, int NV>
void launch_chunks(const BeamSelectArgs& a, BeamSplit s, int64_t item0, int64_t items, ChunkStat* stats,
                   uint64_t* lists, hipStream_t stream) {
  const unsigned blocks = static_cast<unsigned>(items * a.K * s.chunks);
  hipLaunchKernelGGL((beam_chunk_kernel<DT, NV>), dim3(blocks), dim3(kChunkThreads), 0, stream, a, s, item0 * a.K,
                     stats, lists);
}

template <class DT>
void launch_dtype(const BeamSelectArgs& a, BeamSplit s, int64_t item0, int64_t items, ChunkStat* stats,
                  uint64_t* lists, hipStream_t stream) {
  const int per = (s.vecs + kChunkThreads - 1) / kChunkThreads;
  if (per <= 1) launch_chunks<DT, 1>(a, s, item0, items, stats, lists, stream);
  else if (per <= 2) launch_chunks<DT, 2>(a, s, item0, items, stats, lists, stream);
  else if (per <= 4) launch_chunks<DT, 4>(a, s, item0, items, stats, lists, stream);
  else if (per <= 8) launch_chunks<DT, 8>(a, s, item0, items, stats, lists, stream);
  else launch_chunks<DT, kMaxVecs>(a, s, item0, items, stats, lists, stream);
}

}  // namespace

// Chunks as large as a workgroup's registers hold, but enough of them to give
// every compute unit four workgroups when there are few rows.
BeamSplit beam_select_split(int dtype, int64_t rows, int V) {
  const int64_t per = dtype == 0 ? 4 : 8;
  const int64_t nv = V / per;
  const int64_t least = (nv + kChunkThreads * kMaxVecs - 1) / (kChunkThreads * kMaxVecs);
  const int64_t most = (nv + kChunkThreads - 1) / kChunkThreads;
  int64_t c = rows > 0 ? 1024 / rows : 1;
  c = c < most ? c : most;
  c = c > least ? c : least;
  c = c > 1 ? c : 1;
  return BeamSplit{static_cast<int>(c), static_cast<int>((nv + c - 1) / c)};
}

int64_t beam_select_workspace(int dtype, int64_t N, int K, int V, int n) {
  const BeamSplit s = beam_select_split(dtype, N * K, V);
  return N * K * s.chunks * (static_cast<int64_t>(sizeof(ChunkStat)) + 8 * static_cast<int64_t>(n));
}

hipError_t launch_beam_select(int dtype, const BeamSelectArgs& a, hipStream_t stream) {
  const BeamSplit s = beam_select_split(dtype, a.N * a.K, a.V);
  ChunkStat* stats = static_cast<ChunkStat*>(a.workspace);
  uint64_t* lists = reinterpret_cast<uint64_t*>(stats + a.N * a.K * s.chunks);
  // a launch holds at most 2^22 workgroups of 256 threads
  const int64_t step = (int64_t{1} << 22) / (static_cast<int64_t>(a.K) * s.chunks);
  for (int64_t i = 0; i < a.N; i += step) {
    const int64_t items = a.N - i < step ? a.N - i : step;
    if (dtype == 0) launch_dtype<F32T>(a, s, i, items, stats, lists, stream);
    else if (dtype == 1) launch_dtype<F16T>(a, s, i, items, stats, lists, stream);
    else launch_dtype<BF16T>(a, s, i, items, stats, lists, stream);
    hipLaunchKernelGGL(beam_merge_kernel, dim3(static_cast<unsigned>(items)), dim3(kMergeThreads), 0, stream, a,
                       s.chunks, i, stats, lists);
    if (const hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

}  // namespace tkp
