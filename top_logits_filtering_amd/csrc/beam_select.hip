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
// Parents and tokens are whole numbers whose order between beams hangs on
// c[b] - L[b]. The chunks' sums use the hardware's exp2 with a correction for
// the rounding of its argument, 7 or 8 instructions an element, and are within
// kSumError of the exact ones; where candidates of two beams come so close that
// this could swap them, the merge sums those beams' rows again in 64 bits. So
// the order is that of 64-bit values at the price of 32-bit ones: with sums in
// 64 bits throughout (16 instructions an element) the chunks of 256 rows of
// 151936 bf16 logits took 30 us against 20, and those of 1024 rows of 128256
// fp32 ones 110 us against 89 (85 today).
//
// The logits have to be read once and nothing else is of their size. Times on
// one MI355X, chunks + merge, V tokens: a prompt of 4 beams, V 151936 bf16: 5.8 +
// 6.3 us, chains of dependent steps; 64 such prompts: 20 + 6 us (3.9 TB/s); 128
// prompts of 8 beams, V 128256 fp32: 85 to 88 + 9 us (6.0 to 6.2 TB/s); 2 prompts of
// 64 beams, V 151936 bf16, 128 continuations: 21 + 17 us.

#include <float.h>

#include <type_traits>

#include "beam.h"
#include "device_common.h"
#include "exp_sum.h"
#include "reg_tile.h"

namespace tkp {
namespace {

constexpr int kChunkThreads = 256;
constexpr int kChunkWaves = kChunkThreads / kWave;
constexpr int kChunkCap = 1024;  // candidate slots of a chunk
constexpr int kUnits = 16;       // units of a thread at most
constexpr int kHits = 1024;      // units that may reach the bound
// Chunks wanted where rows are few. Each adds a list of n for the merge to go
// through, so half of them for many candidates. Against 1024 chunks: 2 prompts of
// 64 beams, n 128: 45 -> 41 us, 4 of 100 beams, n 200: 84 -> 54 us; n <= 32 the
// same (up to 1 us either way), and with 256 40 prompts of 4 beams, V 100000
// fp32, 25 us against 23 to 24.
constexpr int kTargetBlocks = 512;
constexpr int kMergeThreads = 512;
constexpr int kMergeWaves = kMergeThreads / kWave;
constexpr int kMergeCap = 2048;  // candidate slots of a prompt
constexpr int kHeld = 4;         // list entries a thread of the merge holds from the start
constexpr uint32_t kRoom = kHeld * kMergeThreads;
// Up to so many candidates a chunk takes its bound from 64 maxima, which is 1.4
// us less than from 512. For more of them it would leave ever longer lists.
constexpr uint32_t kGroupBound = 32;
// The same for the merge, whose entries are sorted by list, so that large ones lie
// in one group: 2 prompts of 64 beams with n 24 take 23 us like this and 30 with
// the bound of the chunks, 64 of 16 with n 32 27.5 and 31.6; but one prompt of 4
// beams with n 32 15.4 and 14.0. With n 16 64 maxima are up to 3 us faster.
constexpr uint32_t kMergeGroupBound = 16;
constexpr int kBoundBits = 14;          // bits of a bound from the first that differs on
// So many candidates are ranked without a bound, which takes 4.6 us instead of
// 7.3 for 32 of them, 1 us less for 128, and 4 us more for 256 and 128 prompts.
constexpr uint32_t kAllRanked = 128;
// A longer list is cut to few more than n before it is ranked in time M^2: n 200
// takes 37 us so and 143 without; cut from 64 on, n 8 10.6 instead of 8.8.
constexpr uint32_t kLongList = 320;
constexpr int kQuadStep = 2;  // reads of four elements that overlap; 6.5 us instead of 7.5 for one
constexpr uint32_t kChunkStep = 8, kMergeStep = 4;  // comparisons side by side
constexpr int kMaxBeams = 128;
constexpr int kMaxCandidates = 256;
constexpr int kTokenBits = 20;
// A prompt has no more lists than the merge holds the first entries of: few rows
// are split into kTargetBlocks chunks together, and many beams' rows into as many
// as the longest row needs.
static_assert(kTargetBlocks + kMaxBeams <= kRoom);
static_assert(((1 << kTokenBits) / (kChunkThreads * kUnits * 16)) * kMaxBeams <= kRoom);

// A thread's vectors: 16 elements make a unit, which shares one maximum, and 32
// a group, which is loaded while the one before is summed (fp32 groups of half
// the size took 90 us instead of 84 for 1024 rows of 128256).
template <class DT>
constexpr int kUnitOf = 16 / DT::kPerVec;
template <class DT>
constexpr int kGroupOf = 32 / DT::kPerVec;

// sum exp(x - ref) over a chunk; bad: a NaN or +inf was among the logits.
struct ChunkStat {
  double sum;  // within kSumError
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

// A rank is rounded four times, x - ref, less rest, plus c and times w, all but the
// last to numbers below |s|, or for positive c below |s| + 2c: with and without
// kSumError, and of two ranks, by less than 2^-49 |s w| and for those 2^-49 c w
// together. That shows with scores from 1e9 on.
constexpr double kRounding = 0x1p-48;

// exp(x - ref) in 64 bits, for finite ref and x below ref + 700 or -inf.
__device__ __forceinline__ double exp_below(float x, float ref) {
  return exp(static_cast<double>(x) - static_cast<double>(ref));
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

// The largest T with at least n of the keys k (COUNT per lane; 0: none) at or
// above it, bit by bit: not lower than `stop`, the first `bits` bits that can
// differ. 0 if there are fewer than n keys.
template <int COUNT>
__device__ __forceinline__ uint32_t nth_key(const uint32_t (&k)[COUNT], uint32_t n, int bits, int stop) {
  uint32_t top = 0, low = 0xFFFFFFFFu;
#pragma unroll
  for (int i = 0; i < COUNT; ++i) {
    top = top > k[i] ? top : k[i];
    if (k[i] != 0) low = low < k[i] ? low : k[i];
  }
  top = wave_max_u32(top);
  low = wave_min_u32(low);
  auto count = [&](uint32_t t) __attribute__((always_inline)) -> uint32_t {
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < COUNT; ++i) c += count_ballot(k[i] >= t);
    return c;
  };
  if (top == 0 || count(low) < n) return 0;
  if (low == top) return top;
  int bit = 31 - __builtin_clz(top ^ low);
  const int last = bit - bits + 1 > stop ? bit - bits + 1 : stop;
  uint32_t T = top & ~((2u << bit) - 1u);
#pragma unroll 1
  for (; bit >= last; --bit) {
    const uint32_t t = T | (1u << bit);
    if (count(t) >= n) T = t;
  }
  return T > low ? T : low;
}

// The maximum over groups of SIZE (4 or 8) neighbouring lanes, in all of them.
template <int SIZE>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  auto most = [](uint32_t x, uint32_t y) { return x > y ? x : y; };
  v = most(v, dpp_u32<dpp::kQuad1032>(v, 0u));
  v = most(v, dpp_u32<dpp::kQuad2301>(v, 0u));
  if constexpr (SIZE == 8) v = most(v, dpp_u32<dpp::kRowHalfMirror>(v, 0u));
  return v;
}

// rank[e] = how many of list[0, M) rank above list[e]. The threads share each
// entry's comparisons, so that short lists take few steps. The list has room for
// STEP more entries, which become Item{}, above no other.
template <int THREADS, uint32_t STEP, class Item, class Above>
__device__ __forceinline__ void count_ranks(Item* list, uint32_t* rank, uint32_t M, Above above) {
  const uint32_t tid = threadIdx.x;
  for (uint32_t e = tid; e < M; e += THREADS) rank[e] = 0;
  if (tid < STEP) list[M + tid] = Item{};
  lds_barrier();
  uint32_t span = kWave;
  while (span < M && span < THREADS) span *= 2;
  const uint32_t parts = THREADS / span, part = tid / span;
  const uint32_t seg = (M + parts * STEP - 1) / (parts * STEP) * STEP;
  const uint32_t j0 = part * seg, j1 = j0 + seg < M ? j0 + seg : M;
  for (uint32_t e = tid & (span - 1u); e < M; e += span) {
    const Item mine = list[e];
    uint32_t r = 0;
    for (uint32_t j = j0; j < j1; j += STEP) {
#pragma unroll
      for (uint32_t i = 0; i < STEP; ++i) r += above(list[j + i], mine) ? 1u : 0u;
    }
    if (r != 0) atomicAdd(&rank[e], r);
  }
  lds_barrier();
}

struct ChunkSmem {
  uint64_t list[kChunkCap + kChunkStep];
  uint32_t rank[kChunkCap];
  uint32_t half[2 * kChunkThreads];  // largest of a thread's even and of its odd units, as keys
  double sum[kChunkWaves];
  uint32_t wave_top[kChunkWaves];
  uint32_t group[kWave];
  uint32_t scan[kChunkWaves];
  uint32_t count;
  uint32_t hits;
  uint16_t hit[kHits];               // units that reach the bound: unit * 256 + thread
};
// What finds the elements of those units: the units themselves, or every unit's maximum.
template <class DT>
struct ShortSmem : ChunkSmem {
  vec_t unit[2 * kChunkThreads][kUnitOf<DT>];  // a thread of a short chunk has two
};
struct LongSmem : ChunkSmem {
  float top[kUnits][kChunkThreads];
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

// One chunk: its sum of exp and its n best. Each thread reads its vectors once,
// the next group of them in flight while one is summed, past the caches (525 MB:
// 96 us in all, 103 through them), and notes a maximum per unit. The n-th largest
// of some of these maxima bounds the n-th largest element from below, so only
// units that reach it, a few more than n, are looked at again; their elements
// that reach it are ranked against each other. What bounds it: memory for fp32
// (6.0 to 6.2 TB/s at 525 MB); for 256 rows of 151936 16-bit logits (3.9 TB/s) the seven
// instructions an element in part (with the correction that fp32 needs, two more,
// they take 21.6 us instead of 19.8), and that all 768 workgroups start and end
// together, so that none's 4 us from the last load to the last store are hidden;
// with few chunks those 4 us.
// SHORT: the chunk is one group of layers, which stays in registers (6.5 us
// instead of 6.8 for 64 rows of 32000 fp16); otherwise groups stream through and
// the few vectors that matter are read again.
template <class DT, bool SHORT>
__global__ __launch_bounds__(kChunkThreads) void beam_chunk_kernel(BeamSelectArgs a, BeamSplit split, int64_t row0,
                                                                   ChunkStat* __restrict__ stats,
                                                                   uint64_t* __restrict__ lists) {
  using raw_t = typename DT::raw_t;
  constexpr int P = DT::kPerVec;
  constexpr int kLow = key_low_bits<DT>();
  constexpr int kUnit = kUnitOf<DT>, kGroup = kGroupOf<DT>;
  __shared__ std::conditional_t<SHORT, ShortSmem<DT>, LongSmem> sm;

  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int ch = static_cast<int>(blockIdx.x % static_cast<unsigned>(split.chunks));
  const int64_t row = row0 + blockIdx.x / static_cast<unsigned>(split.chunks);

  // The row as elements before the first 16-byte boundary, whole vectors, and
  // the elements behind the last one; the few single elements are held one per
  // thread, in the first and the last chunk.
  const raw_t* rowp = static_cast<const raw_t*>(a.logits) + row * a.ld;
  const int head = head_of(rowp, a.V);
  const int nfull = (a.V - head) / P;
  const int tail0 = head + nfull * P;
  const int v0 = ch * split.vecs;
  int cnt = nfull - v0;
  cnt = cnt < 0 ? 0 : (cnt < split.vecs ? cnt : split.vecs);
  const int first = head + v0 * P;  // token of the chunk's first vector

  const __amdgpu_buffer_rsrc_t rs = row_rsrc(rowp + (cnt > 0 ? first : 0), cnt * P);
  constexpr uint32_t kNeg = P == 4 ? static_cast<uint32_t>(DT::kNegInf)
                                   : static_cast<uint32_t>(DT::kNegInf) * 0x00010001u;
  // Vector i * 256 + tid; zeros behind the chunk's end.
  auto load = [&](int i) __attribute__((always_inline)) -> vec_t {
    return __builtin_amdgcn_raw_buffer_load_b128(rs, (i * kChunkThreads + tid) * 16, 0, kLoadPolicy);
  };
  // The same for a second look, with -inf behind the end.
  auto again = [&](int at) __attribute__((always_inline)) -> vec_t {
    const vec_t q = __builtin_amdgcn_raw_buffer_load_b128(rs, at * 16, 0, 0);
    return at < cnt ? q : vec_t{kNeg, kNeg, kNeg, kNeg};
  };

  vec_t next[kGroup];
#pragma unroll
  for (int g = 0; g < kGroup; ++g) next[g] = load(g);
  int te = -1;
  if (ch == 0 && tid < head) te = tid;
  if (ch == split.chunks - 1 && tid >= 16 && tid - 16 < a.V - tail0) te = tail0 + tid - 16;
  raw_t re = DT::kNegInf;
  if (te >= 0) re = rowp[te];
  // (the first loads are under way before it is known whether the row counts: of 64
  // rows of 32000 fp16 that are short chunks throughout, 16 of them finished, all are
  // read, 4.6 MB with the lists where the other 48 have 3.1)
  if (!beam_alive(a.scores[row], a.weights != nullptr ? a.weights[row] : 1.0f)) return;
  if (a.finished != nullptr && a.finished[row] != 0) return;
  if (tid == 0) sm.count = sm.hits = 0;

  // One pass: the sum of exp and the largest value of each unit.
  // maximum() keeps a NaN, so that one shows in the chunk's maximum.
  double sum = 0.0, sum_rest = 0.0;
  float half0 = -INFINITY, half1 = -INFINITY;
  const int layers = (cnt + kChunkThreads - 1) / kChunkThreads;
  float tops[kGroup / kUnit];
  auto take = [&](int i0, vec_t (&now)[kGroup]) __attribute__((always_inline)) {
    if ((i0 + kGroup) * kChunkThreads > cnt) {  // the last group
#pragma unroll
      for (int g = 0; g < kGroup; ++g)
        if ((i0 + g) * kChunkThreads + tid >= cnt) now[g] = vec_t{kNeg, kNeg, kNeg, kNeg};
    }
#pragma unroll
    for (int g = 0; g < kGroup; ++g) {
      float m = g % kUnit == 0 ? -INFINITY : tops[g / kUnit];
      float e[P], rest = 0.0f;
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const float x = DT::value(lane_of<raw_t>(now[g], j));
        e[j] = exp_parts<DT>(x, rest);
        m = __builtin_elementwise_maximum(m, x);
      }
      tops[g / kUnit] = m;
#pragma unroll
      for (int d = 1; d < P; d *= 2) {
#pragma unroll
        for (int j = 0; j < P; j += 2 * d) e[j] += e[j + d];
      }
      if constexpr (P == 4) {
        sum += static_cast<double>(__builtin_fmaf(rest, kLn2, e[0]));
      } else {
        sum += static_cast<double>(e[0]);
        sum_rest += static_cast<double>(rest);
      }
    }
#pragma unroll
    for (int u = 0; u < kGroup / kUnit; u += 2) {
      half0 = __builtin_elementwise_maximum(half0, tops[u]);
      half1 = __builtin_elementwise_maximum(half1, tops[u + 1]);
    }
  };
  if constexpr (SHORT) {
    take(0, next);
  } else {
#pragma unroll 1
    for (int i0 = 0; i0 < layers; i0 += kGroup) {
      vec_t now[kGroup];
#pragma unroll
      for (int g = 0; g < kGroup; ++g) now[g] = next[g];
      if (i0 + kGroup < layers) {
#pragma unroll
        for (int g = 0; g < kGroup; ++g) next[g] = load(i0 + kGroup + g);
      }
      take(i0, now);
#pragma unroll
      for (int u = 0; u < kGroup / kUnit; ++u) sm.top[i0 / kUnit + u][tid] = tops[u];
    }
  }
  const float xe = DT::value(re);
  {
    float rest = 0.0f;
    sum += static_cast<double>(exp_parts<DT>(xe, rest));
    sum_rest += static_cast<double>(rest);
    sum = sum_of<DT>(sum, sum_rest);  // (fp32: of this element alone)
  }
  half0 = __builtin_elementwise_maximum(half0, xe);

  // Keys of NaN lie above +inf's: positive ones by order_key, negative ones by this.
  auto key_or_nan = [](float x) -> uint32_t {
    if ((__float_as_uint(x) & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
    return __float_as_uint(x) == 0xFF800000u ? 0u : order_key(x);
  };
  const uint32_t n = static_cast<uint32_t>(a.n);
  const uint32_t pair[2] = {key_or_nan(half0), key_or_nan(half1)};
  const uint32_t own = pair[0] > pair[1] ? pair[0] : pair[1];

  // The n-th largest of some maxima is a lower bound of the chunk's n-th
  // largest value; kBoundBits of it suffice to leave few candidates. For small n
  // of the maxima of 64 groups of threads, one per lane.
  const bool grouped = n <= kGroupBound;
  uint32_t top = wave_max_u32(own);
  sum = wave_sum_f64(sum);
  if (grouped) {
    const uint32_t g = group_max<kChunkThreads / kWave>(own);
    if (tid % (kChunkThreads / kWave) == 0) sm.group[tid / (kChunkThreads / kWave)] = g;
  }
  if (lane == 0) {
    sm.sum[wave] = sum;
    sm.wave_top[wave] = top;
  }
  // For larger n of two maxima of each thread, which every wave then holds,
  // eight per lane.
  auto block_nth = [&](int bits) __attribute__((always_inline)) -> uint32_t {
    sm.half[tid] = pair[0];
    sm.half[kChunkThreads + tid] = pair[1];
    lds_barrier();
    constexpr int kHalf = 2 * kChunkThreads / kWave;
    uint32_t k[kHalf];
#pragma unroll
    for (int i = 0; i < kHalf; ++i) k[i] = sm.half[i * kWave + lane];
    return nth_key(k, n, bits, kLow);
  };
  lds_barrier();
  sum = 0.0;
  top = 0u;
#pragma unroll
  for (int w = 0; w < kChunkWaves; ++w) {
    sum += sm.sum[w];
    top = top > sm.wave_top[w] ? top : sm.wave_top[w];
  }
  uint32_t T = 0u;
  if (grouped) {
    const uint32_t g[1] = {sm.group[lane]};
    T = nth_key(g, n, kBoundBits, kLow);
  }
  const int64_t slot = row * split.chunks + ch;
  uint64_t* out = lists + slot * a.n;
  if (top >= order_key(INFINITY)) {  // a NaN or +inf: the beam proposes nothing
    if (tid == 0) stats[slot] = ChunkStat{0.0, 0.0f, 1};
    return;
  }
  float ref = 0.0f;
  if (top == 0u) {
    sum = 0.0;  // nothing but -inf
  } else if (key_value(top) > kHighMax || key_value(top) < kLowMax) {
    ref = key_value(top);
    double part = exp_below(xe, ref);
#pragma unroll 1
    for (int i = 0; i < layers; ++i) {
      const vec_t q = again(i * kChunkThreads + tid);
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
  if (T == 0u) T = block_nth(kBoundBits);
  if (T == 0u) T = order_key(-FLT_MAX);  // fewer than n maxima: all finite values
  else if (!(T & 0x80000000u)) T |= (1u << kLow) - 1u;
  const float bound = key_value(T);

  auto push = [&](float x, uint32_t token) __attribute__((always_inline)) {
    const uint32_t at = atomicAdd(&sm.count, 1u);
    if (at < kChunkCap) sm.list[at] = pack(order_key(x), token);
  };
  if (xe >= bound) push(xe, static_cast<uint32_t>(te));

  // Units that reach the bound, then their elements, four a thread.
  auto hit = [&](int u, bool is) __attribute__((always_inline)) -> uint32_t {
    if (!is) return kHits;
    const uint32_t at = atomicAdd(&sm.hits, 1u);
    if (at < kHits) sm.hit[at] = static_cast<uint16_t>(u * kChunkThreads + tid);
    return at;
  };
  if constexpr (SHORT) {
#pragma unroll
    for (int u = 0; u < kGroup / kUnit; ++u) {
      const uint32_t at = hit(u, tops[u] >= bound);
      if (at < 2 * kChunkThreads) {
#pragma unroll
        for (int g = 0; g < kUnit; ++g) sm.unit[at][g] = next[u * kUnit + g];
      }
    }
  } else {
    const int units = (layers + kUnit - 1) / kUnit;
    for (int u = 0; u < units; ++u) hit(u, sm.top[u][tid] >= bound);
  }
  lds_barrier();
  const uint32_t hits = sm.hits;
  if (hits <= kHits) {
    constexpr int kQuads = kUnit * P / 4;
    struct Quad {
      raw_t r[4];
    };
    const uint32_t total = hits * kQuads;
    for (uint32_t e0 = tid; e0 < total; e0 += kQuadStep * kChunkThreads) {
      Quad q[kQuadStep];
      uint32_t token[kQuadStep];
#pragma unroll
      for (int u = 0; u < kQuadStep; ++u) {
        q[u] = Quad{{DT::kNegInf, DT::kNegInf, DT::kNegInf, DT::kNegInf}};
        token[u] = 0;
        const uint32_t e = e0 + u * kChunkThreads;
        if (u * kChunkThreads < total && e < total) {
          const int h = sm.hit[e / kQuads], part = static_cast<int>(e % kQuads) * 4;
          const int at = ((h / kChunkThreads) * kUnit + part / P) * kChunkThreads + h % kChunkThreads;
          token[u] = static_cast<uint32_t>(first + at * P + part % P);
          if constexpr (SHORT) q[u] = reinterpret_cast<const Quad*>(sm.unit[e / kQuads])[e % kQuads];
          else if (at < cnt) q[u] = *reinterpret_cast<const Quad*>(rowp + token[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < kQuadStep; ++u) {
        if (u * kChunkThreads >= total) break;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float x = DT::value(q[u].r[j]);
          if (x >= bound) push(x, token[u] + j);
        }
      }
    }
  }
  lds_barrier();
  uint32_t M = sm.count;

  if (hits > kHits || M > kChunkCap) {
    // Many values at or above the bound: find the n-th largest value exactly,
    // list what lies above it, then the equal ones in the order of their tokens.
    auto key_of = [](raw_t r) -> uint32_t {
      const float x = DT::value(r);
      return x >= -FLT_MAX ? order_key(x) : 0u;
    };
    auto count_from = [&](uint32_t t) __attribute__((always_inline)) -> uint32_t {
      uint32_t c = key_of(re) >= t ? 1u : 0u;
#pragma unroll 1
      for (int i = 0; i < layers; ++i) {
        const vec_t q = again(i * kChunkThreads + tid);
#pragma unroll
        for (int j = 0; j < P; ++j) c += key_of(lane_of<raw_t>(q, j)) >= t ? 1u : 0u;
      }
      uint32_t total;
      block_excl(c, total, sm);
      return total;
    };
    // first whether the n-th largest maximum is that value (fewer than n above
    // it), as where many are equal; else it is found bit by bit
    const uint32_t exact = block_nth(32);
    if (exact != 0) T = exact;
    if (!(T & 0x80000000u)) T |= (1u << kLow) - 1u;
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
      const uint32_t key = key_of(r);
      if (key > T) {
        const uint32_t at = atomicAdd(&sm.count, 1u);
        if (at < kChunkCap) sm.list[at] = pack(key, token);
      }
    };
    push_above(re, static_cast<uint32_t>(te));
#pragma unroll 1
    for (int i = 0; i < layers; ++i) {
      const vec_t q = again(i * kChunkThreads + tid);
      const uint32_t token = static_cast<uint32_t>(first + (i * kChunkThreads + tid) * P);
#pragma unroll
      for (int j = 0; j < P; ++j) push_above(lane_of<raw_t>(q, j), token + j);
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
    for (int i = 0; i < layers && have < n; ++i) {
      uint32_t mask = 0;
      const vec_t q = again(i * kChunkThreads + tid);
#pragma unroll
      for (int j = 0; j < P; ++j) mask |= (key_of(lane_of<raw_t>(q, j)) == T ? 1u : 0u) << j;
      push_equal(mask, static_cast<uint32_t>(first + (i * kChunkThreads + tid) * P));
    }
    if (have < n) push_equal(equal_e && te >= tail0 ? 1u : 0u, static_cast<uint32_t>(te));
    M = have < n ? have : n;
    __syncthreads();
  }

  // The candidates are distinct numbers: each one's place is its rank.
  count_ranks<kChunkThreads, kChunkStep>(sm.list, sm.rank, M, [](uint64_t x, uint64_t y) { return x > y; });
  for (uint32_t e = tid; e < M; e += kChunkThreads) {
    const uint32_t r = sm.rank[e];
    if (r < n) out[r] = sm.list[e];
  }
  for (uint32_t e = M + tid; e < n; e += kChunkThreads) out[e] = 0;
  if (tid == 0) stats[slot] = ChunkStat{sum, ref, 0};
}

// A candidate of a prompt: the rank value's image, then beam, logit and token
// (59 bits) such that the larger number ranks first.
struct Cand {
  uint64_t hi, lo;
};
__device__ __forceinline__ int beam_of(const Cand& k) {
  return kMaxBeams - 1 - static_cast<int>(k.lo >> (32 + kTokenBits));
}
__device__ __forceinline__ bool above(const Cand& a, const Cand& b) {
  return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo);
}

// Candidates of two beams come too close and may be in the wrong order; or they are
// equal and in the right order if the beams' rows are alike.
constexpr int kAgain = 1, kEqual = 2;

struct MergeSmem {
  Cand list[kMergeCap + kMergeStep];
  Cand sorted[kMaxCandidates];
  uint32_t upper[kMergeCap];  // the candidates' upper halves of hi
  uint32_t rank[kMergeCap];
  double ref[kMaxBeams];      // L = ref + rest; apart, as ref may be as large as the type goes
  double rest[kMaxBeams];
  double score[kMaxBeams];
  double weight[kMaxBeams];
  int state[kMaxBeams];       // 0: proposes nothing, 1: its lists, 2: finished
  int close[kMaxBeams];       // a candidate comes too close to another beam's
  int like[kMaxBeams];        // of those, the first beam found to have the same row
  int again;                  // kAgain and kEqual
  uint64_t part[2][kMergeWaves];
  uint32_t heads[kMergeThreads];
  Cand best[kMergeWaves];
  uint32_t count;
  uint32_t votes[2];
  uint32_t active[2];               // lists that go on, in two turns
  uint16_t list_of[2][kRoom];
};

// One beam's L and state out of its chunks, held by all threads that pass the
// same row: lane i of `lanes` takes chunks i, i + lanes, ...
template <class Max, class Sum>
__device__ __forceinline__ void beam_total(const ChunkStat* __restrict__ s, int C, int i, int lanes, float c, float w,
                                           bool finished, Max max_of, Sum sum_of, double& ref, double& rest,
                                           int& state) {
  uint32_t rk = 0, bad = 0;
  const bool reads = beam_alive(c, w) && !finished;
  ref = rest = 0.0;
  state = beam_alive(c, w) ? (finished ? 2 : 1) : 0;
  double sum = 0.0;
  if (C <= lanes) {
    ChunkStat t{0.0, 0.0f, 0};
    if (i < C) t = s[i];
    if (reads && t.bad == 0 && t.sum > 0.0) rk = order_key(t.ref);
    bad = max_of(static_cast<uint32_t>(t.bad));
    rk = max_of(rk);
    if (rk != 0) ref = key_value(rk);
    const double d = t.ref - ref;
    if (reads && t.bad == 0 && t.sum > 0.0) sum = d == 0.0 ? t.sum : (d < -2000.0 ? 0.0 : t.sum * exp(d));
  } else if (reads) {
    for (int j = i; j < C; j += lanes) {
      const ChunkStat t = s[j];
      bad |= static_cast<uint32_t>(t.bad);
      if (t.sum > 0.0) rk = rk > order_key(t.ref) ? rk : order_key(t.ref);
    }
    bad = max_of(bad);
    rk = max_of(rk);
    if (rk != 0) ref = key_value(rk);
    for (int j = i; j < C; j += lanes) {
      const ChunkStat t = s[j];
      const double d = t.ref - ref;
      if (t.sum > 0.0) sum += d == 0.0 ? t.sum : (d < -2000.0 ? 0.0 : t.sum * exp(d));
    }
  }
  sum = sum_of(sum);
  if (state == 1) {
    if (bad != 0 || !(sum > 0.0)) state = 0;
    else rest = log(sum);
  }
}

// A sum of terms in [0, 1] that does not depend on their order, so that beams
// with the same logits get the same sum wherever their rows begin: two integers,
// in steps of 2^-42 and of 2^-84, exact for 2^20 terms.
struct ExactSum {
  int64_t high = 0, low = 0;
  __device__ __forceinline__ void add(double t) {
    const double scaled = t * 0x1p42, whole = rint(scaled);
    high += static_cast<int64_t>(whole);
    low += static_cast<int64_t>(rint((scaled - whole) * 0x1p42));
  }
};

// sum exp(x - top) over a whole row in 64 bits, by all threads; top: its maximum.
template <class DT>
__device__ double row_sum(const BeamSelectArgs& a, int64_t row, float top, MergeSmem& sm) {
  using raw_t = typename DT::raw_t;
  constexpr int P = DT::kPerVec;
  const int tid = threadIdx.x;
  const raw_t* rowp = static_cast<const raw_t*>(a.logits) + row * a.ld;
  const int head = head_of(rowp, a.V), nfull = (a.V - head) / P;
  ExactSum sum;
  for (int i = tid; i < head; i += kMergeThreads) sum.add(exp_below(DT::value(rowp[i]), top));
  for (int i = head + nfull * P + tid; i < a.V; i += kMergeThreads) sum.add(exp_below(DT::value(rowp[i]), top));
  const vec_t* v = reinterpret_cast<const vec_t*>(rowp + head);
  for (int i = tid; i < nfull; i += kMergeThreads) {
    const vec_t q = v[i];
#pragma unroll 1  // seldom run: kept small in registers
    for (int j = 0; j < P; ++j) sum.add(exp_below(DT::value(lane_of_dyn<raw_t>(q, j)), top));
  }
  const uint64_t high = wave_sum_u64(static_cast<uint64_t>(sum.high));
  const uint64_t low = wave_sum_u64(static_cast<uint64_t>(sum.low));
  __syncthreads();
  if (tid % kWave == 0) {
    sm.part[0][tid / kWave] = high;
    sm.part[1][tid / kWave] = low;
  }
  __syncthreads();
  uint64_t h = 0, l = 0;
#pragma unroll
  for (int w = 0; w < kMergeWaves; ++w) {
    h += sm.part[0][w];
    l += sm.part[1][w];
  }
  const double rest = static_cast<double>(static_cast<int64_t>(l)) * 0x1p-42;
  return (static_cast<double>(static_cast<int64_t>(h)) + rest) * 0x1p-42;
}

// Whether two rows hold the same bits; asked by all threads. Rows need not begin
// at 16-byte boundaries, which loads of vectors from memory allow.
template <class DT>
__device__ bool rows_alike(const BeamSelectArgs& a, int64_t row0, int64_t row1) {
  using raw_t = typename DT::raw_t;
  constexpr int P = DT::kPerVec;
  const raw_t* x = static_cast<const raw_t*>(a.logits) + row0 * a.ld;
  const raw_t* y = static_cast<const raw_t*>(a.logits) + row1 * a.ld;
  const int nv = a.V / P, tid = threadIdx.x;
  uint32_t differ = 0;
  auto compare = [&](int i) __attribute__((always_inline)) {
    vec_t u, v;
    __builtin_memcpy(&u, x + static_cast<int64_t>(i) * P, 16);
    __builtin_memcpy(&v, y + static_cast<int64_t>(i) * P, 16);
    const vec_t d = u ^ v;
    differ |= d.x | d.y | d.z | d.w;
  };
  if (tid < nv) compare(tid);  // most that differ do so here
  if (__syncthreads_or(static_cast<int>(differ != 0))) return false;
#pragma unroll 4
  for (int i = kMergeThreads + tid; i < nv; i += kMergeThreads) compare(i);
  for (int i = nv * P + tid; i < a.V; i += kMergeThreads) differ |= static_cast<uint32_t>(x[i] != y[i]);
  return !__syncthreads_or(static_cast<int>(differ != 0));
}

// The upper half of the image of a rank value by `margin` and its rounding below T's.
__device__ __forceinline__ uint32_t lowered(uint32_t T, double margin) {
  const uint64_t u = static_cast<uint64_t>(T) << 32;
  const uint64_t bits = (u >> 63) ? u & 0x7FFFFFFFFFFFFFFFull : ~u;
  const double value = __builtin_bit_cast(double, bits);
  const uint32_t t = static_cast<uint32_t>(order_key64(value - (margin + kRounding * fabs(value))) >> 32);
  return t < T && t > 0u ? t : T;
}

// One prompt: L of its beams out of their chunks' sums, then the n best of all
// lists. The lists' first entries are held in registers from the start; the n-th
// of the threads' best bounds the n-th candidate, lists whose last entry held
// still reaches the bound are read on, and what reaches it is ranked. A chain of
// some ten dependent steps in shared memory, 5 to 9.6 us for up to 16
// candidates, and 17 us for 128 of 64 beams: more workgroups than one to a prompt
// would have to meet again at its end.
template <class DT>
__global__ __launch_bounds__(kMergeThreads) void beam_merge_kernel(BeamSelectArgs a, Div chunks, Div window,
                                                                   int64_t item0, const ChunkStat* __restrict__ stats,
                                                                   const uint64_t* __restrict__ lists) {
  __shared__ MergeSmem sm;
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int64_t item = item0 + blockIdx.x;
  const int K = a.K;
  const uint32_t n = static_cast<uint32_t>(a.n);
  const int C = static_cast<int>(chunks.d);
  const uint32_t nl = static_cast<uint32_t>(K * C);  // lists of this prompt
  const uint64_t* __restrict__ mine = lists + item * nl * n;

  // The first entries of every list, `wide` of each, are under way while L is
  // formed. (Lists of beams that propose nothing hold anything; they are not used.)
  const uint32_t wide = window.d, heldn = nl * wide < kRoom ? nl * wide : kRoom;
  uint64_t held[kHeld];
#pragma unroll
  for (int u = 0; u < kHeld; ++u) {
    const uint32_t f = u * kMergeThreads + tid, q = quotient(f, window);
    held[u] = 0;
    if (u * kMergeThreads < heldn && f < heldn) held[u] = mine[q * n + (f - q * wide)];
  }

  // Ranks of two beams may be off against each other by this and kRounding of the rank.
  uint32_t most_w = 0, most_c = 0;  // the largest weight, and the upper half of the largest c w > 0
  for (int b = lane; b < K; b += kWave) {
    const float c = a.scores[item * K + b], w = a.weights != nullptr ? a.weights[item * K + b] : 1.0f;
    if (!beam_alive(c, w)) continue;
    const double cw = static_cast<double>(c) * static_cast<double>(w);
    const uint32_t upper = static_cast<uint32_t>(__builtin_bit_cast(uint64_t, cw) >> 32);
    most_w = most_w > __float_as_uint(w) ? most_w : __float_as_uint(w);
    if (c > 0.0f) most_c = most_c > upper ? most_c : upper;
  }
  const double margin = 2.0 * kSumError * __uint_as_float(wave_max_u32(most_w)) +
                        kRounding * __builtin_bit_cast(double, static_cast<uint64_t>(wave_max_u32(most_c) + 1u) << 32);

  if (tid == 0) sm.count = sm.active[0] = sm.again = 0;
  // A wave per beam, whose lanes take its chunks side by side (19 of them: 6.1 us
  // in all instead of 12.6); a thread per beam where there are more beams.
  if (K <= kMergeWaves) {
    if (wave < K) {
      const int64_t row = item * K + wave;
      const float c = a.scores[row], w = a.weights != nullptr ? a.weights[row] : 1.0f;
      const bool done = a.finished != nullptr && a.finished[row] != 0;
      double ref, rest;
      int state;
      beam_total(stats + row * C, C, lane, kWave, c, w, done, [](uint32_t v) { return wave_max_u32(v); },
                 [](double v) { return wave_sum_f64(v); }, ref, rest, state);
      if (lane == 0) {
        sm.ref[wave] = ref;
        sm.rest[wave] = rest;
        sm.score[wave] = c;
        sm.weight[wave] = w;
        sm.state[wave] = state;
      }
    }
  } else if (tid < K) {
    const int64_t row = item * K + tid;
    const float c = a.scores[row], w = a.weights != nullptr ? a.weights[row] : 1.0f;
    const bool done = a.finished != nullptr && a.finished[row] != 0;
    double ref, rest;
    int state;
    beam_total(stats + row * C, C, 0, 1, c, w, done, [](uint32_t v) { return v; }, [](double v) { return v; }, ref,
               rest, state);
    sm.ref[tid] = ref;
    sm.rest[tid] = rest;
    sm.score[tid] = c;
    sm.weight[tid] = w;
    sm.state[tid] = state;
  }
  if (tid < K) sm.close[tid] = 0;
  lds_barrier();

  // Entry j of list q, e, as a candidate; hi is 0 where there is none.
  auto cand = [&](uint64_t e, uint32_t q, uint32_t j) __attribute__((always_inline)) -> Cand {
    const uint32_t b = quotient(q, chunks);
    const int st = sm.state[b];
    const uint64_t beam = static_cast<uint64_t>(kMaxBeams - 1 - b) << (32 + kTokenBits);
    const uint32_t key = static_cast<uint32_t>(e >> 32);
    const uint32_t back = ((1u << kTokenBits) - 1u) - (0xFFFFFFFFu - static_cast<uint32_t>(e));
    double s = sm.score[b];
    if (st == 1) s += (static_cast<double>(key_value(key)) - sm.ref[b]) - sm.rest[b];
    const bool is = st == 1 ? e != 0 : (st == 2 && j == 0 && q == b * static_cast<uint32_t>(C));
    const uint64_t low = st == 1 ? (static_cast<uint64_t>(key) << kTokenBits) | back : 0;
    return is ? Cand{order_key64(s * sm.weight[b]), beam | low} : Cand{0, 0};
  };
  auto fetch = [&](uint32_t q, uint32_t j) __attribute__((always_inline)) -> Cand {
    return cand(mine[q * n + j], q, j);
  };

  // Once with the chunks' sums; and, if candidates come too close, once more.
  uint32_t M;
  for (bool last = false;; last = true) {
    Cand first[kHeld];
#pragma unroll
    for (int u = 0; u < kHeld; ++u) {
      const uint32_t f = u * kMergeThreads + tid, q = quotient(f, window);
      first[u] = Cand{0, 0};
      if (u * kMergeThreads < heldn && f < heldn) first[u] = cand(held[u], q, f - q * wide);
    }

    // A bound on the n-th candidate: the largest T (of the ranks' upper halves)
    // that n of the threads' best reach; its low bits are left open. Few
    // candidates need none.
    uint32_t T = 1u;
    if (nl * n > kAllRanked) {
      uint32_t best = 0;
#pragma unroll
      for (int u = 0; u < kHeld; ++u) {
        const uint32_t h = static_cast<uint32_t>(first[u].hi >> 32);
        best = best > h ? best : h;
      }
      T = 0u;
      if (n <= kMergeGroupBound) {
        const uint32_t g = group_max<kMergeThreads / kWave>(best);
        if (tid % (kMergeThreads / kWave) == 0) sm.heads[tid / (kMergeThreads / kWave)] = g;
        lds_barrier();
        const uint32_t mine[1] = {sm.heads[lane]};
        T = nth_key(mine, n, kBoundBits, 0);
        lds_barrier();
      }
      if (T == 0u) {
        sm.heads[tid] = best;
        lds_barrier();
        uint32_t h[kMergeWaves];
#pragma unroll
        for (int i = 0; i < kMergeWaves; ++i) h[i] = sm.heads[i * kWave + lane];
        T = nth_key(h, n, kBoundBits, 0);
      }
      T = T == 0u ? 1u : lowered(T, margin);  // fewer than n: every candidate counts
    }

    auto push = [&](const Cand& k) __attribute__((always_inline)) -> bool {
      const uint32_t h = static_cast<uint32_t>(k.hi >> 32);
      if (h < T) return false;
      const uint32_t at = atomicAdd(&sm.count, 1u);
      if (at < kMergeCap) {
        sm.list[at] = k;
        sm.upper[at] = h;
      }
      return true;
    };
    for (int tries = 0;; ++tries) {
      // Candidates from T on: those held, then, of the lists whose last one still
      // reaches T, further windows of entries.
      auto go_on = [&](int turn, uint32_t q) __attribute__((always_inline)) {
        const uint32_t at = atomicAdd(&sm.active[turn], 1u);
        sm.list_of[turn][at] = static_cast<uint16_t>(q);
      };
#pragma unroll
      for (int u = 0; u < kHeld; ++u) {
        if (u * kMergeThreads < heldn && push(first[u]) && wide < n) {
          const uint32_t f = u * kMergeThreads + tid, q = quotient(f, window);
          if (f - q * wide == wide - 1) go_on(0, q);
        }
      }
      int turn = 0;
      for (uint32_t j0 = wide; j0 < n; turn ^= 1) {
        if (tid == 0) sm.active[turn ^ 1] = 0;
        lds_barrier();
        const uint32_t active = sm.active[turn];
        if (active == 0) break;
        uint32_t w = kRoom / active;
        w = w < n - j0 ? w : n - j0;
        for (uint32_t f = tid; f < active * w; f += kMergeThreads) {
          const uint32_t q = sm.list_of[turn][f / w], j = f % w;
          if (push(fetch(q, j0 + j)) && j == w - 1) go_on(turn ^ 1, q);
        }
        lds_barrier();
        j0 += w;
      }
      lds_barrier();
      M = sm.count;
      if (M <= kMergeCap || tries == 4) break;
      // The list is full: the n-th best of what it holds is a better bound.
      uint32_t better = 0;
#pragma unroll 1
      for (int bit = 31; bit >= 0; --bit) {
        const uint32_t t = better | (1u << bit);
        uint32_t c = 0;
        if (tid == 0) sm.votes[bit & 1] = 0;
        __syncthreads();
        for (uint32_t e = tid; e < kMergeCap; e += kMergeThreads) c += sm.upper[e] >= t ? 1u : 0u;
        c = wave_sum_u32(c);
        if (lane == 0) atomicAdd(&sm.votes[bit & 1], c);
        __syncthreads();
        if (sm.votes[bit & 1] >= n) better = t;
      }
      better = lowered(better, margin);
      if (better <= T) break;  // that many are equal there
      T = better;
      __syncthreads();
      if (tid == 0) sm.count = sm.active[0] = 0;
      __syncthreads();
    }

    if (M > kMergeCap && !last && K > 1) {
      // More candidates share an upper half than the list holds, and which of
      // them are close is not seen: every sum is formed again.
      __syncthreads();
      if (tid < K) sm.close[tid] = 1;
      __syncthreads();
    } else {
      if (M > kMergeCap) {
        // Take the best ones one by one, each the largest below the last.
        __syncthreads();
        Cand prev{~0ull, ~0ull};
        uint32_t r = 0;
        for (; r < n; ++r) {
          Cand best{0, 0};
          for (uint32_t f = tid; f < n * nl; f += kMergeThreads) {
            const Cand k = fetch(f / n, f % n);
            if (above(prev, k) && above(k, best)) best = k;
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
          for (int w = 1; w < kMergeWaves; ++w)
            if (above(sm.best[w], best)) best = sm.best[w];
          if (best.hi == 0) break;
          if (tid == 0) {
            sm.list[r] = best;
            sm.upper[r] = static_cast<uint32_t>(best.hi >> 32);
          }
          prev = best;
        }
        M = r;
        __syncthreads();
      }

      // A long list is cut to what reaches the n-th of its upper halves.
      if (M > kLongList) {
        uint32_t cut = 0;
        if (M <= 8 * kWave) {
          uint32_t h[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            h[i] = static_cast<uint32_t>(i * kWave + lane) < M ? sm.upper[i * kWave + lane] : 0u;
          cut = nth_key(h, n, kBoundBits, 0);
        } else {
          uint32_t h[kMergeCap / kWave];
#pragma unroll
          for (int i = 0; i < kMergeCap / kWave; ++i)
            h[i] = static_cast<uint32_t>(i * kWave + lane) < M ? sm.upper[i * kWave + lane] : 0u;
          cut = nth_key(h, n, kBoundBits, 0);
        }
        if (cut != 0u) cut = lowered(cut, margin);
        Cand mine[kMergeCap / kMergeThreads];
#pragma unroll
        for (int u = 0; u < kMergeCap / kMergeThreads; ++u) {
          const uint32_t e = u * kMergeThreads + tid;
          mine[u] = e < M ? sm.list[e] : Cand{0, 0};
        }
        __syncthreads();
        if (tid == 0) sm.count = 0;
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kMergeCap / kMergeThreads; ++u) {
          if (mine[u].hi != 0 && static_cast<uint32_t>(mine[u].hi >> 32) >= cut) {
            const uint32_t at = atomicAdd(&sm.count, 1u);
            sm.list[at] = mine[u];
          }
        }
        __syncthreads();
        M = sm.count;
      }

      // Decode and write.
      count_ranks<kMergeThreads, kMergeStep>(sm.list, sm.rank, M,
                                             [](const Cand& x, const Cand& y) { return above(x, y); });
      for (uint32_t e = tid; e < M; e += kMergeThreads) {
        const Cand k = sm.list[e];
        const uint32_t r = sm.rank[e];
        if (r < n) {
          sm.sorted[r] = k;
          const int b = beam_of(k);
          double s = sm.score[b];
          int32_t token = a.end_token;
          if (sm.state[b] == 1) {
            const uint32_t low = static_cast<uint32_t>(k.lo) & ((1u << kTokenBits) - 1u);
            s += (static_cast<double>(key_value(static_cast<uint32_t>(k.lo >> kTokenBits))) - sm.ref[b]) - sm.rest[b];
            token = static_cast<int32_t>(((1u << kTokenBits) - 1u) - low);
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
      if (last || K == 1) break;
      lds_barrier();

      // Neighbours of different beams that lie closer than the sums are exact, and
      // what lies so close behind the n-th: those beams' sums are formed again.
      // Equal ranks do not show that the sums are: a logit far below another one is
      // lost in 32 bits. But of the same score, weight, logit and row they tie.
      auto pairs = [&](auto compare) __attribute__((always_inline)) {
        if (static_cast<uint32_t>(tid) + 1u < (M < n ? M : n)) compare(sm.sorted[tid], sm.sorted[tid + 1]);
        for (uint32_t e = tid; e < M; e += kMergeThreads)
          if (sm.rank[e] >= n) compare(sm.sorted[n - 1], sm.list[e]);
      };
      auto value = [](const Cand& k) -> double {
        return __builtin_bit_cast(double, (k.hi >> 63) ? k.hi & 0x7FFFFFFFFFFFFFFFull : ~k.hi);
      };
      auto near = [&](const Cand& p, const Cand& q) -> bool {
        return value(p) - value(q) <= margin + kRounding * fabs(value(q));
      };
      pairs([&](const Cand& p, const Cand& q) __attribute__((always_inline)) {
        const int bp = beam_of(p), bq = beam_of(q);
        if (bp == bq || !near(p, q) || (sm.state[bp] == 2 && sm.state[bq] == 2)) return;
        const bool tie = p.hi == q.hi && sm.state[bp] == sm.state[bq] && sm.score[bp] == sm.score[bq] &&
                         sm.weight[bp] == sm.weight[bq] && ((p.lo ^ q.lo) >> kTokenBits & 0xFFFFFFFFu) == 0;
        atomicOr(&sm.again, tie ? kEqual : kAgain);
        sm.close[bp] = sm.close[bq] = 1;
      });
      lds_barrier();
      const int again = sm.again;
      if (again == 0) break;
      if (again == kEqual) {
        // Rows are compared where their sums are equal, until two of them differ all
        // the same: 4 beams with the same row of 151936 bf16 take 31 us so, 64 of them
        // 0.85 ms. (Like rows at different offsets from 16 bytes may have unequal sums.)
        bool differ = false;
        for (int b = 0; b < K && !differ; ++b) {
          if (sm.close[b] == 0) continue;
          int like = 0;
          while (like < b && !(sm.close[like] != 0 && sm.like[like] == like && sm.ref[like] == sm.ref[b] &&
                               sm.rest[like] == sm.rest[b]))
            ++like;
          differ = like < b && !rows_alike<DT>(a, item * K + like, item * K + b);
          if (tid == 0) sm.like[b] = like;
          lds_barrier();
        }
        pairs([&](const Cand& p, const Cand& q) __attribute__((always_inline)) {
          const int bp = beam_of(p), bq = beam_of(q);
          if (!differ && sm.close[bp] != 0 && sm.close[bq] != 0 && sm.like[bp] != sm.like[bq] && near(p, q))
            sm.again = kAgain;
        });
        lds_barrier();
        if (!differ && sm.again == kEqual) break;
      }
      __syncthreads();  // what this pass wrote lies before what the next one writes
    }
    // A row with the bits of the last one summed has its sum: 64 beams with the same
    // row of 151937 bf16, at all offsets from 16 bytes, take 0.95 ms so and 4.9 with a
    // sum each, 4 of them 115 us and 306. (Like rows in turn with others are summed.)
    int before = -1;
    for (int b = 0; b < K; ++b) {
      if (sm.close[b] == 0 || sm.state[b] != 1) continue;
      if (before >= 0 && rows_alike<DT>(a, item * K + before, item * K + b)) {
        if (tid == 0) {
          sm.ref[b] = sm.ref[before];
          sm.rest[b] = sm.rest[before];
        }
        continue;
      }
      before = b;
      uint64_t most = 0;  // the row's maximum heads one of its lists
      for (int i = 0; i < C; ++i) {
        const uint64_t e = mine[static_cast<uint32_t>(b * C + i) * n];
        most = most > e ? most : e;
      }
      const float top = key_value(static_cast<uint32_t>(most >> 32));
      const double sum = row_sum<DT>(a, item * K + b, top, sm);
      if (tid == 0) {
        sm.ref[b] = top;
        sm.rest[b] = log(sum);
      }
    }
    if (tid == 0) sm.count = sm.active[0] = 0;
    __syncthreads();
  }
}

template <class DT>
void launch_both(const BeamSelectArgs& a, BeamSplit s, int64_t item0, int64_t items, ChunkStat* stats,
                 uint64_t* lists, hipStream_t stream) {
  const unsigned blocks = static_cast<unsigned>(items * a.K * s.chunks);
  // few layers: they stay in registers
  if (s.vecs <= kGroupOf<DT> * kChunkThreads)
    hipLaunchKernelGGL((beam_chunk_kernel<DT, true>), dim3(blocks), dim3(kChunkThreads), 0, stream, a, s, item0 * a.K,
                       stats, lists);
  else
    hipLaunchKernelGGL((beam_chunk_kernel<DT, false>), dim3(blocks), dim3(kChunkThreads), 0, stream, a, s,
                       item0 * a.K, stats, lists);
  // the window of entries that the merge holds of every list
  const uint32_t nl = static_cast<uint32_t>(a.K) * static_cast<uint32_t>(s.chunks);
  uint32_t wide = kRoom / nl;
  wide = wide < static_cast<uint32_t>(a.n) ? wide : static_cast<uint32_t>(a.n);
  hipLaunchKernelGGL(beam_merge_kernel<DT>, dim3(static_cast<unsigned>(items)), dim3(kMergeThreads), 0, stream, a,
                     make_div(static_cast<uint32_t>(s.chunks)), make_div(wide), item0, stats, lists);
}

}  // namespace

// Chunks of one group of layers or more when there are few rows, so that every
// compute unit gets some, and of as many layers as a workgroup notes maxima for
// when there are many.
BeamSplit beam_select_split(int dtype, int64_t rows, int V, int n) {
  const int64_t per = dtype == 0 ? 4 : 8;
  const int64_t nv = V / per;
  const int64_t largest = kChunkThreads * kUnits * 16 / per, smallest = kChunkThreads * 32 / per;
  const int64_t least = (nv + largest - 1) / largest;
  const int64_t most = (nv + smallest - 1) / smallest;
  const int64_t target = n <= static_cast<int>(kGroupBound) ? kTargetBlocks : kTargetBlocks / 2;
  int64_t c = rows > 0 ? (target + rows - 1) / rows : 1;
  c = c < most ? c : most;
  c = c > least ? c : least;
  c = c > 1 ? c : 1;
  return BeamSplit{static_cast<int>(c), static_cast<int>((nv + c - 1) / c)};
}

int64_t beam_select_workspace(int dtype, int64_t N, int K, int V, int n) {
  const BeamSplit s = beam_select_split(dtype, N * K, V, n);
  return N * K * s.chunks * (static_cast<int64_t>(sizeof(ChunkStat)) + 8 * static_cast<int64_t>(n));
}

hipError_t launch_beam_select(int dtype, const BeamSelectArgs& a, hipStream_t stream) {
  const BeamSplit s = beam_select_split(dtype, a.N * a.K, a.V, a.n);
  ChunkStat* stats = static_cast<ChunkStat*>(a.workspace);
  uint64_t* lists = reinterpret_cast<uint64_t*>(stats + a.N * a.K * s.chunks);
  // a launch holds at most 2^22 workgroups of 256 threads
  const int64_t step = (int64_t{1} << 22) / (static_cast<int64_t>(a.K) * s.chunks);
  for (int64_t i = 0; i < a.N; i += step) {
    const int64_t items = a.N - i < step ? a.N - i : step;
    if (dtype == 0) launch_both<F32T>(a, s, i, items, stats, lists, stream);
    else if (dtype == 1) launch_both<F16T>(a, s, i, items, stats, lists, stream);
    else launch_both<BF16T>(a, s, i, items, stats, lists, stream);
    if (const hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

}  // namespace tkp
