// Verification of drafted tokens.
//
// With p_w the softmax of row w of a sequence's target logits (row 0 follows the
// last token, row j + 1 draft j) and q_j that of draft row j, a draft d = drafts[j]
// behind an accepted one stands if u_j q_j(d) < p_j(d) (q = 1 where the draft
// came from no distribution). The token behind the accepted ones is drawn with
// the last uniform, by its place in the cumulative sum, from max(p - q, 0) where
// a draft was rejected (from p without the rejected tokens if there is no q) and
// from p where none was. Several drafts behind one token share its uniform: they
// cut [0, 1) into pieces of p(token). Tokens are whole numbers, so decisions are
// those of 64-bit sums.
//
//   1. verify_rows_kernel: sums of exp of chunks of the rows.
//   2. verify_final_kernel: every workgroup goes down the path by those sums, then
//      sums its chunk of the row where the path ends; the last workgroup of a
//      sequence finds the token.

#include <float.h>

#include "device_common.h"
#include "reg_tile.h"
#include "speculative.h"

namespace tkp {
namespace {

constexpr int kT = 256;  // threads of a workgroup
constexpr int kW = kT / kWave;
constexpr int kMaxRows = 256;  // D + 1 at most
constexpr int kBlock = 8;      // neighbouring elements of a thread
constexpr int kMaxParts = (1 << 20) / (kT * kBlock);
static_assert(kMaxParts <= 2 * kT);
// A residual of no more mass than this is what roundings of the logits leave; the
// token then comes from p itself.
constexpr double kLeast = 0x1p-40;

// sum exp(x - ref) over a chunk; bad: a NaN or +inf was among the logits. For the
// argmax, best holds (logit, token) as one number instead of the sum.
struct RowChunk {
  union {
    double sum;
    uint64_t best;
  };
  float ref;
  int bad;
};

// Sums over a chunk of the row where the path ends.
struct FinalPart {
  double all;    // of p's terms
  double kept;   // of those that are left: all but the rejected tokens', or where p > q
  double other;  // of q's terms where p > q
  double draft;  // of q's terms
  double close;  // of p's terms where p and q are too close to tell which is larger
};

// exp(x - ref) in 64 bits, for x <= ref or not far above it, or -inf.
__device__ __forceinline__ double exp_from(float x, float ref) {
  return exp(static_cast<double>(x) - static_cast<double>(ref));
}

__device__ __forceinline__ double wave_incl_scan_f64(double v) {
  auto step = [&](uint64_t moved) { v += __builtin_bit_cast(double, moved); };
  auto bits = [&]() { return __builtin_bit_cast(uint64_t, v); };
  step(dpp_u64<dpp::kRowShr1>(bits(), 0ull));
  step(dpp_u64<dpp::kRowShr2>(bits(), 0ull));
  step(dpp_u64<dpp::kRowShr4>(bits(), 0ull));
  step(dpp_u64<dpp::kRowShr8>(bits(), 0ull));
  step(dpp_u64<dpp::kRowBcast15, 0xA>(bits(), 0ull));
  step(dpp_u64<dpp::kRowBcast31, 0xC>(bits(), 0ull));
  return v;
}

// Elements v .. v + 7 of a row, -inf behind its end.
template <class DT>
__device__ __forceinline__ void load_block(const typename DT::raw_t* row, int v, int V, float (&x)[kBlock]) {
  using raw_t = typename DT::raw_t;
  if (v + kBlock <= V) {
    raw_t r[kBlock];  // rows begin at any element
    __builtin_memcpy(r, row + v, sizeof(r));
#pragma unroll
    for (int j = 0; j < kBlock; ++j) x[j] = DT::value(r[j]);
  } else {
#pragma unroll
    for (int j = 0; j < kBlock; ++j) x[j] = v + j < V ? DT::value(row[v + j]) : -INFINITY;
  }
}

struct WalkSmem {
  int32_t token[kMaxRows];   // -1: the draft counts as not there
  int32_t node[kMaxRows];    // the row that it follows
  float u[kMaxRows];
  float x[kMaxRows];         // its logit in that row
  float y[kMaxRows];         // and in the draft's row
  double sum[2][kMaxRows];   // of the rows (a chain's): target, draft
  float ref[2][kMaxRows];
  int32_t path[kMaxRows];
  double part[kW];
};

// A row's sum out of its chunks, in every lane of the wave. sum = 0: no
// distribution. In the same way the largest (logit, token): 0 for none.
struct RowSum {
  double sum;
  float ref;
};
__device__ __forceinline__ RowSum row_sum(const RowChunk* __restrict__ s, int chunks) {
  const int lane = threadIdx.x % kWave;
  uint32_t bad = 0;
  float top = -INFINITY;
  for (int c = lane; c < chunks; c += kWave) {
    bad |= static_cast<uint32_t>(s[c].bad);
    if (s[c].sum > 0.0) top = fmaxf(top, s[c].ref);
  }
  bad = wave_max_u32(bad);
  top = wave_max_f32(top);
  double sum = 0.0;
  for (int c = lane; c < chunks; c += kWave) {
    const double t = s[c].sum, d = static_cast<double>(s[c].ref) - top;
    if (t > 0.0) sum += d == 0.0 ? t : t * exp(d);
  }
  sum = wave_sum_f64(sum);
  return bad != 0 ? RowSum{0.0, 0.0f} : RowSum{sum, top};
}
__device__ __forceinline__ uint64_t row_best(const RowChunk* __restrict__ s, int chunks) {
  uint32_t bad = 0;
  uint64_t best = 0;
  for (int c = threadIdx.x % kWave; c < chunks; c += kWave) {
    bad |= static_cast<uint32_t>(s[c].bad);
    best = best > s[c].best ? best : s[c].best;
  }
  best = wave_reduce_u64(best, 0ull, [](uint64_t a, uint64_t b) { return a > b ? a : b; });
  return wave_max_u32(bad) != 0 ? 0ull : best;
}
__device__ __forceinline__ int best_token(uint64_t best) {
  return best == 0 ? -1 : static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(best));
}

template <class DT>
__device__ __forceinline__ const typename DT::raw_t* target_row(const VerifyArgs& a, int64_t seq, int w) {
  return static_cast<const typename DT::raw_t*>(a.logits) + (seq * (a.D + 1) + w) * a.ld;
}
template <class DT>
__device__ __forceinline__ const typename DT::raw_t* draft_row(const VerifyArgs& a, int64_t seq, int j) {
  return static_cast<const typename DT::raw_t*>(a.draft_logits) + (seq * a.D + j) * a.ld_draft;
}
__device__ __forceinline__ const RowChunk* target_stats(const VerifyArgs& a, const RowChunk* stats, int chunks,
                                                        int64_t seq, int w) {
  return stats + (seq * (a.D + 1) + w) * chunks;
}
__device__ __forceinline__ const RowChunk* draft_stats(const VerifyArgs& a, const RowChunk* stats, int chunks,
                                                       int64_t seq, int j) {
  return stats + (a.N * (a.D + 1) + seq * a.D + j) * chunks;
}
__device__ __forceinline__ int draft_count(const VerifyArgs& a, int64_t seq) {
  const int n = a.lengths != nullptr ? a.lengths[seq] : a.D;
  return n < 0 ? 0 : (n < a.D ? n : a.D);
}

// sum exp(x - ref) of a whole row in 64 bits, by the workgroup.
template <class DT>
__device__ double sum_again(const typename DT::raw_t* row, int V, float ref, WalkSmem& sm) {
  double sum = 0.0;
  for (int v = threadIdx.x * kBlock; v < V; v += kT * kBlock) {
    float x[kBlock];
    load_block<DT>(row, v, V, x);
#pragma unroll
    for (int j = 0; j < kBlock; ++j) sum += exp_from(x[j], ref);
  }
  sum = wave_sum_f64(sum);
  __syncthreads();
  if (threadIdx.x % kWave == 0) sm.part[threadIdx.x / kWave] = sum;
  __syncthreads();
  sum = 0.0;
#pragma unroll
  for (int w = 0; w < kW; ++w) sum += sm.part[w];
  return sum;
}

// Where the path of a sequence ends.
enum Kind : int { kNone = 0, kPlain = 1, kWithout = 2, kResidual = 3 };
struct Walk {
  int node;    // row
  int count;   // accepted drafts, in sm.path
  Kind kind;   // what the token is drawn from: nothing, p, p without rejected tokens, max(p - q, 0)
  RowSum p, q;
  uint64_t best;
};

// Relative error of a row's sum out of its chunks, and what decisions closer than
// that take: both sums again in 64 bits.
constexpr double kClose = 1e-6;

// Goes down a sequence's path. All threads of the workgroup take part and get the
// same result.
template <class DT>
__device__ Walk walk(const VerifyArgs& a, const RowChunk* stats, int chunks, int64_t seq, WalkSmem& sm) {
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int D = a.D, n = draft_count(a, seq);
  const bool greedy = a.uniforms == nullptr, chain = a.parents == nullptr;
  if (tid < D) {
    int token = a.drafts[seq * D + tid];
    const int parent = chain ? tid - 1 : a.parents[seq * D + tid];
    if (tid >= n || token < 0 || token >= a.V || parent < -1 || parent >= tid) token = -1;
    sm.token[tid] = token;
    sm.node[tid] = parent + 1;
    sm.x[tid] = token < 0 || greedy ? -INFINITY : DT::value(target_row<DT>(a, seq, parent + 1)[token]);
    sm.y[tid] = token < 0 || a.draft_logits == nullptr ? -INFINITY : DT::value(draft_row<DT>(a, seq, tid)[token]);
  }
  if (!greedy && tid <= D) sm.u[tid] = a.uniforms[seq * (D + 1) + tid];
  if (chain && !greedy) {
    for (int r = wave; r < n + 1; r += kW) {
      const RowSum t = row_sum(target_stats(a, stats, chunks, seq, r), chunks);
      RowSum q{0.0, 0.0f};
      if (a.draft_logits != nullptr && r < n) q = row_sum(draft_stats(a, stats, chunks, seq, r), chunks);
      if (lane == 0) {
        sm.sum[0][r] = t.sum;
        sm.ref[0][r] = t.ref;
        sm.sum[1][r] = q.sum;
        sm.ref[1][r] = q.ref;
      }
    }
  }
  __syncthreads();
  // a token that an earlier draft behind the same one has already counts once
  if (!chain) {
    bool twice = false;
    if (tid < D)
      for (int j = 0; j < tid; ++j) twice |= sm.node[j] == sm.node[tid] && sm.token[j] == sm.token[tid];
    __syncthreads();
    if (twice) sm.token[tid] = -1;
    __syncthreads();
  }

  Walk w{0, 0, kNone, {0.0, 0.0f}, {0.0, 0.0f}, 0ull};
  for (;;) {
    // the drafts behind this node: bits of the draft numbers
    uint64_t kids[kMaxRows / kWave];
    bool any = false;
#pragma unroll
    for (int i = 0; i < kMaxRows / kWave; ++i) {
      const int j = i * kWave + lane;
      kids[i] = __ballot(j < D && sm.token[j] >= 0 && sm.node[j] == w.node);
      any |= kids[i] != 0;
    }
    int taken = -1;
    if (greedy) {
      w.best = row_best(target_stats(a, stats, chunks, seq, w.node), chunks);
      const int token = best_token(w.best);
#pragma unroll
      for (int i = 0; i < kMaxRows / kWave; ++i)
        for (uint64_t m = kids[i]; m != 0 && taken < 0; m &= m - 1) {
          const int j = i * kWave + __builtin_ctzll(m);
          if (sm.token[j] == token) taken = j;
        }
    } else {
      w.p = chain ? RowSum{sm.sum[0][w.node], sm.ref[0][w.node]}
                  : row_sum(target_stats(a, stats, chunks, seq, w.node), chunks);
      w.q = RowSum{0.0, 0.0f};
      w.kind = !(w.p.sum > 0.0) ? kNone : kPlain;
      if (any && w.kind != kNone) {
        const double u = sm.u[w.node];
        if (a.draft_logits != nullptr) {
          const int j = w.node;
          w.q = RowSum{sm.sum[1][j], sm.ref[1][j]};
          const double pe = exp_from(sm.x[j], w.p.ref);
          const double qe = w.q.sum > 0.0 ? exp_from(sm.y[j], w.q.ref) : 0.0;
          // u q < p with both sums on the other side
          double left = u * qe * w.p.sum, right = pe * (w.q.sum > 0.0 ? w.q.sum : 1.0);
          if (right > 0.0 && left > right * (1.0 - kClose) && left < right * (1.0 + kClose)) {
            w.p.sum = sum_again<DT>(target_row<DT>(a, seq, j), a.V, w.p.ref, sm);
            w.q.sum = sum_again<DT>(draft_row<DT>(a, seq, j), a.V, w.q.ref, sm);
            left = u * qe * w.p.sum;
            right = pe * w.q.sum;
          }
          if (left < right) taken = j;
          else if (w.q.sum > 0.0) w.kind = kResidual;
        } else {
          for (int turn = 0; turn < 2; ++turn) {
            const double at = u * w.p.sum;
            double upto = 0.0;
            bool close = false;
            taken = -1;
#pragma unroll
            for (int i = 0; i < kMaxRows / kWave; ++i)
              for (uint64_t m = kids[i]; m != 0; m &= m - 1) {
                const int j = i * kWave + __builtin_ctzll(m);
                upto += exp_from(sm.x[j], w.p.ref);
                close |= upto > at * (1.0 - kClose) && upto < at * (1.0 + kClose);
                if (at < upto && taken < 0) taken = j;
              }
            if (!close || turn == 1) break;
            w.p.sum = sum_again<DT>(target_row<DT>(a, seq, w.node), a.V, w.p.ref, sm);
          }
          if (taken < 0) w.kind = kWithout;
        }
      }
    }
    if (taken < 0) break;
    if (tid == 0) sm.path[w.count] = taken;
    ++w.count;
    w.node = taken + 1;
  }
  __syncthreads();
  return w;
}

// One chunk of one row: its sum of exp, or its largest element. Blocks of a
// sequence: its target rows, then its draft rows.
template <class DT, bool GREEDY>
__global__ __launch_bounds__(kT) void verify_rows_kernel(VerifyArgs a, int chunks, int blocks, int64_t seq0,
                                                         RowChunk* __restrict__ stats, uint32_t* __restrict__ arrived) {
  using raw_t = typename DT::raw_t;
  __shared__ double sum_of[kW];
  __shared__ uint32_t top_of[kW];
  __shared__ uint64_t best_of[kW];
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int rows = a.D + 1 + (a.draft_logits != nullptr ? a.D : 0);
  const unsigned b = blockIdx.x;
  const int ch = static_cast<int>(b % static_cast<unsigned>(chunks));
  const unsigned item = b / static_cast<unsigned>(chunks);
  const int r = static_cast<int>(item % static_cast<unsigned>(rows));
  const int64_t seq = seq0 + item / static_cast<unsigned>(rows);
  if (r == 0 && ch == 0 && tid == 0) arrived[seq] = 0;
  const bool target = r <= a.D;
  const int w = target ? r : r - a.D - 1;
  const int n = draft_count(a, seq);
  if (target ? w > n : w >= n) return;
  const raw_t* row = target ? target_row<DT>(a, seq, w) : draft_row<DT>(a, seq, w);
  RowChunk* out = const_cast<RowChunk*>(target ? target_stats(a, stats, chunks, seq, w)
                                               : draft_stats(a, stats, chunks, seq, w)) + ch;
  const int first = ch * blocks * kT * kBlock;

  auto key_or_nan = [](float x) -> uint32_t {
    if (__builtin_isnan(x)) return 0xFFFFFFFFu;
    return F32T::key(__float_as_uint(x));
  };
  uint32_t top = 0;
  uint64_t best = 0;
  for (int i = 0; i < blocks; ++i) {
    const int v = first + (i * kT + tid) * kBlock;
    if (v >= a.V) break;
    float x[kBlock];
    load_block<DT>(row, v, a.V, x);
#pragma unroll
    for (int j = 0; j < kBlock; ++j) {
      const uint32_t k = key_or_nan(x[j]);
      top = top > k ? top : k;
      if constexpr (GREEDY) {
        const uint64_t one = (static_cast<uint64_t>(k) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(v + j));
        if (x[j] > -INFINITY && one > best) best = one;
      }
    }
  }
  top = wave_max_u32(top);
  if constexpr (GREEDY)
    best = wave_reduce_u64(best, 0ull, [](uint64_t p, uint64_t q) { return p > q ? p : q; });
  if (lane == 0) {
    top_of[wave] = top;
    best_of[wave] = best;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kW; ++i) {
    top = top > top_of[i] ? top : top_of[i];
    best = best > best_of[i] ? best : best_of[i];
  }
  const int bad = top >= F32T::key(0x7F800000u) ? 1 : 0;
  if constexpr (GREEDY) {
    if (tid == 0) {
      out->best = best;
      out->ref = 0.0f;
      out->bad = bad;
    }
    return;
  }
  const float ref = __uint_as_float(F32T::raw_of_key(top));
  double sum = 0.0;
  if (!bad && top > F32T::key(0xFF800000u)) {
    for (int i = 0; i < blocks; ++i) {
      const int v = first + (i * kT + tid) * kBlock;
      if (v >= a.V) break;
      float x[kBlock];
      load_block<DT>(row, v, a.V, x);
#pragma unroll
      for (int j = 0; j < kBlock; ++j) sum += exp_from(x[j], ref);
    }
  }
  sum = wave_sum_f64(sum);
  if (lane == 0) sum_of[wave] = sum;
  __syncthreads();
  if (tid == 0) {
    sum = 0.0;
    for (int i = 0; i < kW; ++i) sum += sum_of[i];
    out->sum = sum;
    out->ref = ref;
    out->bad = bad;
  }
}

struct FinalSmem {
  WalkSmem walk;
  int32_t out[kMaxRows];  // rejected tokens within the chunk
  int outs;
  double sum[5][kW];
  double parts[kMaxParts];  // of chunks, where summed again
  int last;
  int found;
  double below;
};

// The terms of eight neighbouring elements: p's, and q's.
template <class DT>
struct Terms {
  double p[kBlock], q[kBlock];
};
template <class DT>
__device__ __forceinline__ void terms_at(const typename DT::raw_t* prow, const typename DT::raw_t* qrow, int v, int V,
                                         const Walk& w, bool two, Terms<DT>& t) {
  float x[kBlock];
  load_block<DT>(prow, v, V, x);
#pragma unroll
  for (int j = 0; j < kBlock; ++j) t.p[j] = x[j] == -INFINITY ? 0.0 : exp_from(x[j], w.p.ref);
  if (two) {
    load_block<DT>(qrow, v, V, x);
#pragma unroll
    for (int j = 0; j < kBlock; ++j) t.q[j] = x[j] == -INFINITY ? 0.0 : exp_from(x[j], w.q.ref);
  }
}

// The rejected tokens within [first, end).
__device__ __forceinline__ void list_out(const VerifyArgs& a, const Walk& w, int first, int end, FinalSmem& sm) {
  const int tid = threadIdx.x;
  __syncthreads();
  if (tid == 0) sm.outs = 0;
  __syncthreads();
  if (w.kind == kWithout && tid < a.D && sm.walk.node[tid] == w.node) {
    const int t = sm.walk.token[tid];
    if (t >= first && t < end) sm.out[atomicAdd(&sm.outs, 1)] = t;
  }
  __syncthreads();
}
__device__ __forceinline__ bool is_out(int v, const FinalSmem& sm) {
  bool out = false;
  for (int i = 0; i < sm.outs; ++i) out |= sm.out[i] == v;
  return out;
}

// The workgroup's sum of v, in all threads.
__device__ __forceinline__ double block_sum(double v, double (&at)[kW]) {
  v = wave_sum_f64(v);
  __syncthreads();
  if (threadIdx.x % kWave == 0) at[threadIdx.x / kWave] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int i = 0; i < kW; ++i) v += at[i];
  return v;
}
// The sum of v over the threads below, and of all.
__device__ __forceinline__ double block_below(double v, double& all, double (&at)[kW]) {
  const int wave = threadIdx.x / kWave;
  const double upto = wave_incl_scan_f64(v);
  __syncthreads();
  if (threadIdx.x % kWave == kWave - 1) at[wave] = upto;
  __syncthreads();
  double below = 0.0;
  all = 0.0;
#pragma unroll
  for (int i = 0; i < kW; ++i) {
    if (i < wave) below += at[i];
    all += at[i];
  }
  return below + (upto - v);
}

template <class DT>
__global__ __launch_bounds__(kT) void verify_final_kernel(VerifyArgs a, int chunks, int parts, int blocks, int64_t seq0,
                                                          const RowChunk* __restrict__ stats,
                                                          FinalPart* __restrict__ finals,
                                                          uint32_t* __restrict__ arrived) {
  using raw_t = typename DT::raw_t;
  __shared__ FinalSmem sm;
  const int tid = threadIdx.x;
  const int ch = static_cast<int>(blockIdx.x % static_cast<unsigned>(parts));
  const int64_t seq = seq0 + blockIdx.x / static_cast<unsigned>(parts);
  const Walk w = walk<DT>(a, stats, chunks, seq, sm.walk);
  int32_t* tokens = a.out_tokens + seq * (a.D + 1);
  const bool greedy = a.uniforms == nullptr;
  const bool draws = !greedy && w.kind != kNone;
  if (ch == 0) {
    if (tid <= a.D && !(tid == w.count && draws))
      tokens[tid] = tid < w.count ? a.drafts[seq * a.D + sm.walk.path[tid]]
                                  : (tid == w.count && greedy ? best_token(w.best) : -1);
    if (a.out_path != nullptr && tid < a.D) a.out_path[seq * a.D + tid] = tid < w.count ? sm.walk.path[tid] : -1;
    if (tid == 0) a.out_accepted[seq] = w.count;
  }
  if (!draws) return;

  const raw_t* prow = target_row<DT>(a, seq, w.node);
  const bool two = w.kind == kResidual;
  const raw_t* qrow = two ? draft_row<DT>(a, seq, w.node) : prow;
  const int span = blocks * kT * kBlock;
  // p > q where scale * p's term > q's
  const double near = two ? w.q.sum / w.p.sum : 0.0;
  FinalPart mine{0.0, 0.0, 0.0, 0.0, 0.0};
  {
    const int first = ch * span;
    list_out(a, w, first, first + span, sm);
    for (int i = 0; i < blocks; ++i) {
      const int v = first + (i * kT + tid) * kBlock;
      if (v >= a.V) break;
      Terms<DT> t;
      terms_at<DT>(prow, qrow, v, a.V, w, two, t);
#pragma unroll
      for (int j = 0; j < kBlock; ++j) {
        mine.all += t.p[j];
        if (two) {
          const double more = near * t.p[j] - t.q[j];
          mine.draft += t.q[j];
          if (more > 0.0) {
            mine.kept += t.p[j];
            mine.other += t.q[j];
          }
          if (__builtin_fabs(more) <= 2.0 * kClose * t.q[j]) mine.close += t.p[j];
        } else if (!is_out(v + j, sm)) {
          mine.kept += t.p[j];
        }
      }
    }
  }
  mine.all = block_sum(mine.all, sm.sum[0]);
  mine.kept = block_sum(mine.kept, sm.sum[1]);
  mine.other = block_sum(mine.other, sm.sum[2]);
  mine.draft = block_sum(mine.draft, sm.sum[3]);
  mine.close = block_sum(mine.close, sm.sum[4]);
  FinalPart* slots = finals + seq * parts;
  if (tid == 0) {
    auto put = [](double* to, double v) { __hip_atomic_store(to, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); };
    put(&slots[ch].all, mine.all);
    put(&slots[ch].kept, mine.kept);
    put(&slots[ch].other, mine.other);
    put(&slots[ch].draft, mine.draft);
    put(&slots[ch].close, mine.close);
    const uint32_t before =
        __hip_atomic_fetch_add(&arrived[seq], 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    sm.last = before == static_cast<uint32_t>(parts) - 1u ? 1 : 0;
    sm.found = 0x7FFFFFFF;
  }
  __syncthreads();
  if (!sm.last) return;

  // The sequence's last workgroup: all sums are there.
  __threadfence();
  auto get = [](const double* from) { return __hip_atomic_load(from, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); };
  FinalPart p[2];
  FinalPart total{0.0, 0.0, 0.0, 0.0, 0.0};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int c = 2 * tid + i;
    p[i] = FinalPart{0.0, 0.0, 0.0, 0.0, 0.0};
    if (c < parts) p[i] = FinalPart{get(&slots[c].all), get(&slots[c].kept), get(&slots[c].other), get(&slots[c].draft),
                                    get(&slots[c].close)};
    total.all += p[i].all;
    total.draft += p[i].draft;
    total.close += p[i].close;
  }
  total.all = block_sum(total.all, sm.sum[0]);
  total.draft = block_sum(total.draft, sm.sum[1]);
  total.close = block_sum(total.close, sm.sum[2]);
  // what an element weighs: scale * p's term, less q's term or nothing if left out
  double scale = two ? total.draft / total.all : 1.0;
  bool residual = two, without = w.kind == kWithout;
  auto weight = [&](const Terms<DT>& t, int j, int v) -> double {
    if (residual) {
      const double more = scale * t.p[j] - t.q[j];
      return more > 0.0 ? more : 0.0;
    }
    return without && is_out(v, sm) ? 0.0 : t.p[j];
  };
  double part[2];
  if (two && total.close > 0x1p-20 * total.all) {
    // too much lies where the first ratio of the sums does not tell which is larger
    for (int c = 0; c < parts; ++c) {
      double sum = 0.0;
      for (int i = 0; i < blocks; ++i) {
        const int v = c * span + (i * kT + tid) * kBlock;
        if (v >= a.V) break;
        Terms<DT> t;
        terms_at<DT>(prow, qrow, v, a.V, w, true, t);
#pragma unroll
        for (int j = 0; j < kBlock; ++j) sum += weight(t, j, v + j);
      }
      sum = block_sum(sum, sm.sum[0]);
      if (tid == 0) sm.parts[c] = sum;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) part[i] = 2 * tid + i < parts ? sm.parts[2 * tid + i] : 0.0;
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const double left = two ? scale * p[i].kept - p[i].other : p[i].kept;
      part[i] = left > 0.0 ? left : 0.0;
    }
  }
  const double rest = block_sum(part[0] + part[1], sm.sum[0]);
  if (w.kind != kPlain && !(rest > kLeast * (two ? total.draft : total.all))) {
    residual = without = false;
#pragma unroll
    for (int i = 0; i < 2; ++i) part[i] = p[i].all;
  }
  double all;
  const double below = block_below(part[0] + part[1], all, sm.sum[1]);
  const double at = static_cast<double>(sm.walk.u[a.D]) * all;
  // the first chunk that reaches past `at`; if none does, the last one with any weight
  int mine_c = -1;
  if (part[0] > 0.0 && below + part[0] > at) mine_c = 2 * tid;
  else if (part[1] > 0.0 && below + part[0] + part[1] > at) mine_c = 2 * tid + 1;
  if (mine_c >= 0) atomicMin(&sm.found, mine_c);
  __syncthreads();
  const bool past = sm.found == 0x7FFFFFFF;
  __syncthreads();
  if (past) {
    if (tid == 0) sm.found = -1;
    __syncthreads();
    if (part[1] > 0.0) atomicMax(&sm.found, 2 * tid + 1);
    else if (part[0] > 0.0) atomicMax(&sm.found, 2 * tid);
    __syncthreads();
  }
  const int c = sm.found;
  if (c >= 0 && c / 2 == tid) sm.below = below + (c % 2 != 0 ? part[0] : 0.0);
  list_out(a, w, c * span, (c + 1) * span, sm);
  if (tid == 0) {
    sm.found = 0x7FFFFFFF;
    sm.last = -1;
  }
  double base = sm.below;
  __syncthreads();
  if (c < 0) {  // nothing weighs anything
    if (tid == 0) tokens[w.count] = -1;
    return;
  }
  for (int i = 0; i < blocks; ++i) {
    const int v = c * span + (i * kT + tid) * kBlock;
    double wt[kBlock], sum = 0.0;
    int some = -1;  // the last element with any weight
    if (v < a.V) {
      Terms<DT> t;
      terms_at<DT>(prow, qrow, v, a.V, w, two, t);
#pragma unroll
      for (int j = 0; j < kBlock; ++j) {
        wt[j] = weight(t, j, v + j);
        sum += wt[j];
        if (wt[j] > 0.0) some = v + j;
      }
    }
    double here;
    double upto = base + block_below(sum, here, sm.sum[2]);
    if (some >= 0) {
      atomicMax(&sm.last, some);
      int token = 0x7FFFFFFF;
      if (upto + sum > at) {
        token = some;
#pragma unroll
        for (int j = 0; j < kBlock; ++j) {
          upto += wt[j];
          if (wt[j] > 0.0 && upto > at) {
            token = token < v + j ? token : v + j;
          }
        }
        atomicMin(&sm.found, token);
      }
    }
    base += here;
    __syncthreads();
    if (sm.found != 0x7FFFFFFF) break;
  }
  if (tid == 0) tokens[w.count] = sm.found != 0x7FFFFFFF ? sm.found : sm.last;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Chunks that a row is cut into, of whole layers of a workgroup.
struct Cut {
  int chunks, blocks;
};
Cut cut_of(int64_t rows, int V, int most) {
  const int64_t layers = V > 0 ? ceil_div(V, kT * kBlock) : 1;
  int64_t blocks = rows * layers / 1024;
  blocks = blocks < 1 ? 1 : (blocks > most ? most : blocks);
  return Cut{static_cast<int>(ceil_div(layers, blocks)), static_cast<int>(blocks)};
}
Cut rows_cut(int64_t N, int D, int V, bool draft) { return cut_of(N * (D + 1 + (draft ? D : 0)), V, 8); }
Cut final_cut(int64_t N, int V) { return cut_of(N, V, 4); }

struct Layout {
  int64_t stats, finals, arrived, bytes;
};
Layout layout_of(int64_t N, int D, int V, bool draft) {
  const int64_t rows = N * (D + 1 + (draft ? D : 0));
  Layout l;
  l.stats = 0;
  l.finals = l.stats + rows * rows_cut(N, D, V, draft).chunks * static_cast<int64_t>(sizeof(RowChunk));
  l.arrived = l.finals + N * final_cut(N, V).chunks * static_cast<int64_t>(sizeof(FinalPart));
  l.bytes = l.arrived + N * 4;
  return l;
}

template <class DT>
hipError_t launch_typed(const VerifyArgs& a, hipStream_t stream) {
  const bool draft = a.draft_logits != nullptr;
  const int rows = a.D + 1 + (draft ? a.D : 0);
  const Cut rc = rows_cut(a.N, a.D, a.V, draft), fc = final_cut(a.N, a.V);
  const Layout l = layout_of(a.N, a.D, a.V, draft);
  char* ws = static_cast<char*>(a.workspace);
  RowChunk* stats = reinterpret_cast<RowChunk*>(ws + l.stats);
  FinalPart* finals = reinterpret_cast<FinalPart*>(ws + l.finals);
  uint32_t* arrived = reinterpret_cast<uint32_t*>(ws + l.arrived);
  const bool greedy = a.uniforms == nullptr;
  // a launch holds at most 2^22 workgroups of 256 threads
  const int64_t per = static_cast<int64_t>(rows) * rc.chunks > fc.chunks ? static_cast<int64_t>(rows) * rc.chunks
                                                                           : fc.chunks;
  const int64_t step = (int64_t{1} << 22) / per > 0 ? (int64_t{1} << 22) / per : 1;
  for (int64_t i = 0; i < a.N; i += step) {
    const int64_t n = a.N - i < step ? a.N - i : step;
    const dim3 g1(static_cast<unsigned>(n * rows * rc.chunks)), g2(static_cast<unsigned>(n * (greedy ? 1 : fc.chunks)));
    if (greedy)
      hipLaunchKernelGGL((verify_rows_kernel<DT, true>), g1, dim3(kT), 0, stream, a, rc.chunks, rc.blocks, i, stats,
                         arrived);
    else
      hipLaunchKernelGGL((verify_rows_kernel<DT, false>), g1, dim3(kT), 0, stream, a, rc.chunks, rc.blocks, i, stats,
                         arrived);
    if (const hipError_t e = hipGetLastError()) return e;
    hipLaunchKernelGGL((verify_final_kernel<DT>), g2, dim3(kT), 0, stream, a, rc.chunks, greedy ? 1 : fc.chunks,
                       fc.blocks, i, stats, finals, arrived);
    if (const hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

}  // namespace

int64_t verify_workspace(int dtype, int64_t N, int D, int V, bool draft_logits) {
  (void)dtype;
  return layout_of(N, D, V, draft_logits).bytes;
}

hipError_t launch_verify(int dtype, const VerifyArgs& a, hipStream_t stream) {
  if (dtype == 0) return launch_typed<F32T>(a, stream);
  if (dtype == 1) return launch_typed<F16T>(a, stream);
  return launch_typed<BF16T>(a, stream);
}

}  // namespace tkp
