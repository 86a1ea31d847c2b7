// Verification of drafted tokens.
//
// With p_w the softmax of row w of a sequence's target logits (row 0 follows the
// last token, row j + 1 draft j) and q_j that of draft row j, a draft d = drafts[j]
// behind an accepted one stands if u_j q_j(d) < p_j(d) (q = 1 where the draft
// came from no distribution). The token behind the accepted ones is drawn with
// the last uniform, by its place in the cumulative sum, from max(p - q, 0) where
// a draft was rejected (from p without the rejected tokens if there is no q) and
// from p where none was. Several drafts behind one token share its uniform: they
// cut [0, 1) into pieces of p(token).
//
//   1. verify_rows_kernel: sums of exp of chunks of the rows; of large trees only of
//      their first rows, and then
//      verify_behind_kernel: of the rows where each path goes on.
//   2. verify_final_kernel: every workgroup goes down the path by those sums, then
//      sums its range of the row where the path ends; the last workgroup of a
//      sequence finds the token.
//
// What bounds it: the rows are read once at the rate of the memory (64 sequences of 4
// drafts with draft logits, V 151936 bf16, 175 MB: 33 us, 5.3 TB/s; 128 of 3, V 128256
// fp32, 460 MB: 71 us, 6.5 TB/s), and the row where a path ends, with its draft row, a
// second time (22 and 45 us), as max(p - q, 0) needs both sums first. About 12 us of
// the last kernel are steps that hang on one another, which a single sequence takes as
// well: sums, the path, the row, what the workgroups tell each other, the token.
//
// Tokens are whole numbers, so decisions are those of 64-bit sums. An acceptance
// has one border, which sums in 32 bits with a known error (exp_sum.h) miss about
// once in a million; then both rows are summed again in 64 bits. A token that is
// drawn has a border beside every other one: that row's terms are in 64 bits.

#include <float.h>

#include <type_traits>

#include "device_common.h"
#include "draft_tree.h"
#include "exp64.h"
#include "exp_sum.h"
#include "reg_tile.h"
#include "speculative.h"
#include "verify_plan.h"

namespace tkp {
namespace {

using namespace verify;

constexpr int kW = kT / kWave;
constexpr int kMaxRows = 256;  // D + 1 at most
static_assert(kPiece == kWave * kBlock && kWaveLanes == kWave);
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
static_assert(sizeof(RowChunk) == 16);

// Sums over a chunk of the row where the path ends.
struct FinalPart {
  double all;    // of p's terms
  double left;   // of what is left: p's terms without the rejected tokens', or ratio * p's less q's where that is above 0
  double kept;   // of p's terms where it is
  double draft;  // of q's terms
  double close;  // of q's terms where they are too close to p's to tell which is larger: not in left and kept
};
constexpr int kSums = sizeof(FinalPart) / sizeof(double);
// Where workgroups of a sequence meet. Each one's counter has 64 bytes of its own:
// counters side by side wait for one another (8 sequences of 4 proposals, V 151936 bf16,
// 18.0 us instead of 15.9).
constexpr int kApart = 16;
struct Meeting {
  double* sums;       // [kSums][parts], those of all workgroups' waves as in FinalPart
  uint32_t* arrived;  // workgroups that are done, kApart counters apart
};

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

// What workgroups of one kernel tell each other goes past the caches of their dies:
// stores and loads of device scope, in order by waiting for the stores. (A fence
// of device scope writes back a die's whole cache: with one in every wave the last
// kernel took ten times as long.)
__device__ __forceinline__ void put_far(double* to, double v) {
  __hip_atomic_store(to, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ double get_far(const double* from) {
  return __hip_atomic_load(from, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// Whether this workgroup is the last of `count` that come here, which then sees
// what all of them have put. `told`: in shared memory.
__device__ __forceinline__ bool last_of(uint32_t* arrived, int count, int& told) {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (threadIdx.x == 0)
    told = __hip_atomic_fetch_add(arrived, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                   static_cast<uint32_t>(count) - 1u
               ? 1
               : 0;
  asm volatile("" ::: "memory");
  __syncthreads();
  return told != 0;
}

// A row's sum out of its chunks, by LANES neighbouring lanes (16 or a wave), which all
// get it; first: the first chunk of each lane, if there is one. sum = 0: no distribution.
struct RowSum {
  double sum;
  float ref;
};
template <int LANES, class T, class Op>
__device__ __forceinline__ T over_lanes(T v, Op op) {
  auto step = [&](uint64_t moved) { v = op(v, __builtin_bit_cast(T, moved)); };
  auto bits = [&]() { return __builtin_bit_cast(uint64_t, v); };
  step(dpp_u64<dpp::kQuad1032>(bits(), 0ull));
  step(dpp_u64<dpp::kQuad2301>(bits(), 0ull));
  step(dpp_u64<dpp::kRowHalfMirror>(bits(), 0ull));
  step(dpp_u64<dpp::kRowMirror>(bits(), 0ull));
  if constexpr (LANES == kWave) {
    T all = __builtin_bit_cast(T, readlane_u64(bits(), 0));
#pragma unroll
    for (int i = 16; i < kWave; i += 16) all = op(all, __builtin_bit_cast(T, readlane_u64(bits(), i)));
    v = all;
  }
  return v;
}
template <int LANES>
__device__ __forceinline__ RowSum row_sum(const RowChunk* __restrict__ s, int chunks, const RowChunk& first) {
  const int lane = threadIdx.x % LANES;
  // references and bad chunks as one number: those of 0 need no exp
  double sum = 0.0;
  float top = -INFINITY;
  bool bad = false, moved = false;
  for (int c = lane; c < chunks; c += LANES) {
    const RowChunk t = c == lane ? first : s[c];
    bad |= t.bad != 0;
    if (t.sum > 0.0) {
      top = fmaxf(top, t.ref);
      moved |= t.ref != 0.0f;
      sum += t.sum;
    }
  }
  if (__ballot(moved) != 0) {  // some chunk of the wave's rows has a reference of its own
    top = static_cast<float>(over_lanes<LANES>(static_cast<double>(top), [](double a, double b) { return fmax(a, b); }));
    sum = 0.0;
    for (int c = lane; c < chunks; c += LANES) {
      const RowChunk t = c == lane ? first : s[c];
      if (t.sum > 0.0) sum += t.sum * exp_from(t.ref, top);
    }
  } else {
    top = 0.0f;
  }
  sum = over_lanes<LANES>(sum, [](double a, double b) { return a + b; });
  const uint64_t any = over_lanes<LANES>(static_cast<uint64_t>(bad ? 1 : 0), [](uint64_t a, uint64_t b) { return a | b; });
  return any != 0 ? RowSum{0.0, 0.0f} : RowSum{sum, top};
}
// In the same way the largest (logit, token) as one number: 0 for none.
template <int LANES>
__device__ __forceinline__ uint64_t row_best(const RowChunk* __restrict__ s, int chunks, const RowChunk& first) {
  const int lane = threadIdx.x % LANES;
  uint64_t best = 0;
  for (int c = lane; c < chunks; c += LANES) {
    const RowChunk t = c == lane ? first : s[c];
    const uint64_t one = t.bad != 0 ? ~0ull : t.best;
    best = best > one ? best : one;
  }
  best = over_lanes<LANES>(best, [](uint64_t a, uint64_t b) { return a > b ? a : b; });
  return best == ~0ull ? 0ull : best;
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

// sum exp(x - ref) of a whole row in 64 bits, by the workgroup's first kT threads, so
// that every kernel gets the same. Rarely taken, so the elements of a block go
// through one exp in turn.
template <class DT>
__device__ __forceinline__ double sum_again(const typename DT::raw_t* row, int V, float ref, double (&at)[kW]) {
  double sum = 0.0;
  if (threadIdx.x < kT) {
#pragma unroll 1
    for (int v = threadIdx.x * kBlock; v < V; v += kT * kBlock) {
      float x[kBlock];
      load_block<DT>(row, v, V, x);
#pragma unroll 1
      for (int j = 0; j < kBlock; ++j) {
        sum += exp_from(x[0], ref);
#pragma unroll
        for (int k = 0; k + 1 < kBlock; ++k) x[k] = x[k + 1];
      }
    }
    sum = wave_sum_f64(sum);
  }
  __syncthreads();
  if (threadIdx.x < kT && threadIdx.x % kWave == 0) at[threadIdx.x / kWave] = sum;
  __syncthreads();
  sum = 0.0;
#pragma unroll
  for (int w = 0; w < kW; ++w) sum += at[w];
  return sum;
}

// What the drafts are, as kernels of their own: the code of one that does
// everything is 43 KB, which every compute unit would have to fetch.
enum Mode : int { kGreedy = 0, kProposed = 1, kDrawn = 2 };

// Where the path of a sequence ends.
enum Kind : int { kNone = 0, kPlain = 1, kWithout = 2, kResidual = 3 };
struct Walk {
  int node;    // row
  int count;   // accepted drafts, in sm.path
  Kind kind;   // what the token is drawn from: nothing, p, p without rejected tokens, max(p - q, 0)
  bool open;   // it goes on at rows that are not summed yet
  RowSum p, q;
  uint64_t best;
};

struct WalkSmem {
  int32_t token[kMaxRows];   // -1: the draft counts as not there
  int32_t node[kMaxRows];    // the row that it follows, -1 if it is not there
  float u[kMaxRows];
  double term[kMaxRows];     // its term in that row
  union {
    double sum[2][kMaxRows];  // of the rows: target, draft
    uint64_t best[kMaxRows];
  };
  float ref[2][kMaxRows];
  int32_t path[kMaxRows];
  uint64_t ends[kMaxRows / kWave];   // drafts of a chain that are rejected, are not there or cannot be told
  uint64_t close[kMaxRows / kWave];  // those that cannot be told
  double part[kW];
  Walk state;
  int again;
  float last_u;  // the one that the token is drawn with
};
// Relative error of a row's sum out of its chunks, and what decisions closer than
// that take: both sums again in 64 bits.
constexpr double kClose = 1e-6;
// Elements whose terms of p and q, by the ratio of such sums, differ by no more.
constexpr double kBand = 1e-6;

__device__ __forceinline__ DraftPlace draft_of(const VerifyArgs& a, int64_t seq, int j, int n) {
  if (j >= n) return DraftPlace{-1, -1};
  return draft_place(j, a.drafts[seq * a.D + j], a.parents == nullptr ? j - 1 : a.parents[seq * a.D + j], a.V);
}

// Goes down a sequence's path, in a tree `limit` drafts far at most: so many of its
// rows are summed. All threads of the workgroup take part and get the same result;
// what is one thing after the other is left to the first wave.
constexpr int kSets = kMaxRows / kWave;
template <class DT, Mode MODE>
__device__ __forceinline__ Walk walk(const VerifyArgs& a, const RowChunk* stats, int chunks, int limit, int64_t seq, WalkSmem& sm) {
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int D = a.D, n = draft_count(a, seq);
  constexpr bool greedy = MODE == kGreedy, drawn = MODE == kDrawn;
  const bool chain = drawn || a.parents == nullptr;
  const bool mine = wave * kWave <= n;  // waves that have drafts to look at: the first kSets at most
  int token = -1, node = -1;
  float x = -INFINITY, y = -INFINITY;
  if (mine) {
    const DraftPlace at = draft_of(a, seq, tid, n);
    token = at.token;
    node = at.node;
    if (token >= 0 && !greedy) x = DT::value(target_row<DT>(a, seq, node)[token]);
    if (token >= 0 && drawn) y = DT::value(draft_row<DT>(a, seq, tid)[token]);
    sm.u[tid] = !greedy && tid <= n ? a.uniforms[seq * (D + 1) + tid] : 0.0f;
  }
  if (tid < kMaxRows) {
    sm.token[tid] = token;
    sm.node[tid] = node;
    sm.path[tid] = tid;
  }
  if (tid == 0) sm.last_u = greedy ? 0.0f : a.uniforms[seq * (D + 1) + D];
  // 16 lanes a row: target rows, then draft rows (in a tree those that are not summed yet
  // are not looked at). Sums of kAtOnce rows are on their way at a time: 32 trees of 39
  // drafts 42.1 us, 43.3 one at a time. Draft logits leave no registers for that.
  constexpr int kRound = kT / 16, kAtOnce = drawn ? 1 : 4;
  const int targets = n + 1, rows = targets + (drawn ? n : 0), end = (rows + 3) / 4 * 4;
  auto row_stats = [&](int r) {
    return r < targets ? target_stats(a, stats, chunks, seq, r) : draft_stats(a, stats, chunks, seq, r - targets);
  };
  for (int i0 = tid < kT ? tid / 16 : end; i0 < end; i0 += kAtOnce * kRound) {
    RowChunk first[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int i = i0 + k * kRound;
      first[k] = RowChunk{};
      if (i < rows && tid % 16 < chunks) first[k] = row_stats(i)[tid % 16];
    }
#pragma unroll 1
    for (int k = 0; k < kAtOnce && i0 + k * kRound < end; ++k) {
      const int i = i0 + k * kRound, r = i < rows ? i : 0;
      if constexpr (greedy) {
        const uint64_t best = row_best<16>(row_stats(r), chunks, first[0]);
        if (tid % 16 == 0 && i < rows) sm.best[r] = best;
      } else {
        const RowSum t = row_sum<16>(row_stats(r), chunks, first[0]);
        if (tid % 16 == 0 && i < rows) {
          const bool target = r < targets;
          sm.sum[target ? 0 : 1][target ? r : r - targets] = t.sum;
          sm.ref[target ? 0 : 1][target ? r : r - targets] = t.ref;
        }
      }
#pragma unroll
      for (int j = 0; j + 1 < kAtOnce; ++j) first[j] = first[j + 1];
    }
  }
  __syncthreads();

  Walk w{0, 0, kNone, false, {0.0, 0.0f}, {0.0, 0.0f}, 0ull};
  if (chain) {
    // All drafts side by side. One that was drawn, or a proposal (then with 1 for q
    // and its sum), stands behind accepted ones if u q < p, with both sums on the
    // other side.
    bool stays = false, close = false;
    double pe = 0.0, qe = 1.0;
    auto stands = [&](double psum, double qsum) -> bool {
      const double left = sm.u[tid] * qe * psum, right = pe * qsum;
      close = right > 0.0 && left > right * (1.0 - kClose) && left < right * (1.0 + kClose);
      return left < right;
    };
    if (mine) {
      if (token >= 0) {
        if constexpr (greedy) {
          stays = token == best_token(sm.best[tid]);
        } else {
          const double psum = sm.sum[0][tid], qsum = drawn ? sm.sum[1][tid] : 1.0;
          pe = exp_from(x, sm.ref[0][tid]);
          if (drawn) qe = qsum > 0.0 ? exp_from(y, sm.ref[1][tid]) : 0.0;
          if (psum > 0.0) stays = stands(psum, qsum > 0.0 ? qsum : 1.0);
        }
      }
      const uint64_t ends = __ballot(!stays || close), closes = __ballot(close);
      if (lane == 0) {
        sm.ends[wave] = ends;
        sm.close[wave] = closes;
      }
    } else if (lane == 0 && wave < kSets) {
      sm.ends[wave] = ~0ull;
      sm.close[wave] = 0ull;
    }
    __syncthreads();
    int at;
    for (;;) {
      // the first draft that is rejected, is not there or cannot be told
      at = D;
      bool again = false;
#pragma unroll
      for (int i = kSets - 1; i >= 0; --i) {
        const uint64_t end = sm.ends[i];
        if (end != 0) {
          const int bit = __builtin_ctzll(end);
          at = i * kWave + bit;
          again = (sm.close[i] >> bit & 1u) != 0;
        }
      }
      at = at < D ? at : D;
      if (!again) break;
      double psum = 0.0, qsum = 1.0;
      const bool q = drawn && sm.sum[1][at] > 0.0;
#pragma unroll 1
      for (int i = 0; i < (q ? 2 : 1); ++i) {
        const double sum = sum_again<DT>(i == 0 ? target_row<DT>(a, seq, at) : draft_row<DT>(a, seq, at), a.V,
                                         sm.ref[i][at], sm.part);
        psum = i == 0 ? sum : psum;
        qsum = i == 1 ? sum : qsum;
      }
      __syncthreads();
      if (tid == at) {
        if (stands(psum, qsum)) sm.ends[wave] &= ~(1ull << lane);
        sm.close[wave] &= ~(1ull << lane);
      }
      __syncthreads();
    }
    w.node = w.count = at;
    if constexpr (greedy) {
      w.best = sm.best[at];
    } else {
      w.p = RowSum{sm.sum[0][at], sm.ref[0][at]};
      w.kind = w.p.sum > 0.0 ? kPlain : kNone;
      if (w.kind == kPlain && at < n && sm.token[at] >= 0) {  // a draft was rejected
        if constexpr (drawn) {
          w.q = RowSum{sm.sum[1][at], sm.ref[1][at]};
          if (w.q.sum > 0.0) w.kind = kResidual;
        } else {
          w.kind = kWithout;
        }
      }
    }
  } else if constexpr (!drawn) {
    // A tree: from node to node, out of the drafts' terms in their rows.
    if (mine && !greedy) sm.term[tid] = token >= 0 ? exp_from(x, sm.ref[0][node]) : 0.0;
    __syncthreads();
    bool exact = false;  // the sum of the node's row is in 64 bits
    for (;;) {
      if (wave == 0) {
        if (exact) w.p.sum = sm.state.p.sum;
        bool again = false;
        int tokens[kSets], nodes[kSets];
#pragma unroll
        for (int i = 0; i < kSets; ++i) {
          tokens[i] = sm.token[i * kWave + lane];
          nodes[i] = sm.node[i * kWave + lane];
        }
        for (;;) {
          uint64_t kids[kSets];  // the drafts behind this node: bits of the draft numbers
#pragma unroll
          for (int i = 0; i < kSets; ++i) kids[i] = __ballot(tokens[i] >= 0 && nodes[i] == w.node);
          int taken = -1;
          if constexpr (greedy) {
            w.best = sm.best[w.node];
            const int top = best_token(w.best);
#pragma unroll
            for (int i = kSets - 1; i >= 0; --i) {
              const uint64_t hit = __ballot(tokens[i] == top) & kids[i];
              if (hit != 0 && top >= 0) taken = i * kWave + __builtin_ctzll(hit);
            }
          } else {
            if (!exact) w.p = RowSum{sm.sum[0][w.node], sm.ref[0][w.node]};
            w.kind = w.p.sum > 0.0 ? kPlain : kNone;
            if (w.kind == kNone) break;
            const double at = sm.u[w.node] * w.p.sum;
            double upto = 0.0;
            bool close = false, any = false;
#pragma unroll
            for (int i = 0; i < kSets; ++i)
              for (uint64_t m = kids[i]; m != 0; m &= m - 1) {
                const int bit = __builtin_ctzll(m), j = i * kWave + bit;
                // a token that an earlier one of them has counts once
                const int same = __builtin_amdgcn_readlane(tokens[i], bit);
                uint64_t before = __ballot(tokens[i] == same) & kids[i] & ((1ull << bit) - 1);
#pragma unroll
                for (int k = 0; k < i; ++k) before |= __ballot(tokens[k] == same) & kids[k];
                if (before != 0) continue;
                any = true;
                upto += sm.term[j];
                close |= upto > at * (1.0 - kClose) && upto < at * (1.0 + kClose);
                if (at < upto && taken < 0) taken = j;
              }
            if (close && !exact) {
              again = true;
              break;
            }
            if (taken < 0 && any) w.kind = kWithout;
          }
          if (taken < 0) break;
          if (lane == 0) sm.path[w.count] = taken;
          ++w.count;
          w.node = taken + 1;
          exact = false;
          w.open = w.count >= limit;
          if (w.open) break;
        }
        if (lane == 0) {
          sm.state.node = w.node;
          sm.state.count = w.count;
          sm.state.kind = w.kind;
          sm.state.open = w.open;
          sm.state.p.sum = w.p.sum;
          sm.state.p.ref = w.p.ref;
          sm.state.best = w.best;
          sm.again = again ? 1 : 0;
        }
      }
      __syncthreads();
      if (sm.again == 0) break;
      const double sum = sum_again<DT>(target_row<DT>(a, seq, sm.state.node), a.V, sm.state.p.ref, sm.part);
      if (tid == 0) sm.state.p.sum = sum;
      exact = true;
      __syncthreads();
    }
    w.node = sm.state.node;
    w.count = sm.state.count;
    w.kind = sm.state.kind;
    w.open = sm.state.open;
    w.p.sum = sm.state.p.sum;
    w.p.ref = sm.state.p.ref;
    w.best = sm.state.best;
  }
  return w;
}

struct ChunkSmem {
  double sum[kW];
  uint32_t top[kW];
  uint64_t best[kW];
};

// One chunk of a row, of split.vecs vectors of 16 bytes: its sum of exp, or its
// largest element. The vectors of one group are on their way while the ones before
// are summed; the few elements before the row's first 16-byte boundary and behind
// its last one belong to the first and the last chunk. Returned to all threads.
template <class DT, bool GREEDY, bool KEEP>
__device__ __forceinline__ RowChunk chunk_of(const typename DT::raw_t* row, int V, int ch, Split split, ChunkSmem& sm) {
  using raw_t = typename DT::raw_t;
  constexpr int P = DT::kPerVec, kGroup = 32 / P;
  constexpr uint32_t kNeg = P == 4 ? static_cast<uint32_t>(DT::kNegInf)
                                   : static_cast<uint32_t>(DT::kNegInf) * 0x00010001u;
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int head = head_of(row, V);
  const int nfull = (V - head) / P;
  const int tail0 = head + nfull * P;
  const int v0 = ch * split.vecs;
  int cnt = nfull - v0;
  cnt = cnt < 0 ? 0 : (cnt < split.vecs ? cnt : split.vecs);
  const int first = head + v0 * P;
  const __amdgpu_buffer_rsrc_t rs = row_rsrc(row + (cnt > 0 ? first : 0), cnt * P);
  auto load = [&](int i) __attribute__((always_inline)) -> vec_t {
    return __builtin_amdgcn_raw_buffer_load_b128(rs, (i * kT + tid) * 16, 0, KEEP ? 0 : kLoadPolicy);
  };
  vec_t next[kGroup];
#pragma unroll
  for (int g = 0; g < kGroup; ++g) next[g] = load(g);
  int te = -1;
  if (ch == 0 && tid < head) te = tid;
  if (ch == split.chunks - 1 && tid >= 16 && tid - 16 < V - tail0) te = tail0 + tid - 16;
  raw_t re = DT::kNegInf;
  if (te >= 0) re = row[te];

  double sum = 0.0, sum_rest = 0.0;
  float top = -INFINITY;  // maximum() keeps a NaN
  float most = -INFINITY;
  int most_at = 0;        // the first element that is as large
  const int layers = (cnt + kT - 1) / kT;
#pragma unroll 1
  for (int i0 = 0; i0 < layers; i0 += kGroup) {
    vec_t now[kGroup];
#pragma unroll
    for (int g = 0; g < kGroup; ++g) now[g] = next[g];
    if (i0 + kGroup < layers) {
#pragma unroll
      for (int g = 0; g < kGroup; ++g) next[g] = load(i0 + kGroup + g);
    }
    if ((i0 + kGroup) * kT > cnt) {  // the last group
#pragma unroll
      for (int g = 0; g < kGroup; ++g)
        if ((i0 + g) * kT + tid >= cnt) now[g] = vec_t{kNeg, kNeg, kNeg, kNeg};
    }
#pragma unroll
    for (int g = 0; g < kGroup; ++g) {
      float e[P], rest = 0.0f;
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const float x = DT::value(lane_of<raw_t>(now[g], j));
        top = __builtin_elementwise_maximum(top, x);
        if constexpr (GREEDY) {
          const bool more = x > most;
          most = more ? x : most;
          most_at = more ? ((i0 + g) * kT + tid) * P + j : most_at;
        } else {
          e[j] = exp_parts<DT>(x, rest);
        }
      }
      if constexpr (!GREEDY) {
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
    }
  }
  const float xe = DT::value(re);
  top = __builtin_elementwise_maximum(top, xe);
  auto key_or_nan = [](float x) -> uint32_t {
    return __builtin_isnan(x) ? 0xFFFFFFFFu : F32T::key(__float_as_uint(x));
  };
  uint32_t top_key = wave_max_u32(key_or_nan(top));
  uint64_t best = 0;
  if constexpr (GREEDY) {
    auto pack = [](float x, int at) -> uint64_t {
      return x > -INFINITY ? (static_cast<uint64_t>(F32T::key(__float_as_uint(x))) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(at))
                           : 0ull;
    };
    best = pack(most, first + most_at);
    const uint64_t one = pack(xe, te);
    best = best > one ? best : one;
    best = over_lanes<kWave>(best, [](uint64_t a, uint64_t b) { return a > b ? a : b; });
  } else {
    float rest = 0.0f;
    sum += static_cast<double>(exp_parts<DT>(xe, rest));
    sum_rest += static_cast<double>(rest);
    sum = wave_sum_f64(sum_of<DT>(sum, sum_rest));  // (fp32: rest is that of this element alone)
  }
  __syncthreads();
  if (lane == 0) {
    sm.sum[wave] = sum;
    sm.top[wave] = top_key;
    sm.best[wave] = best;
  }
  __syncthreads();
  sum = 0.0;
#pragma unroll
  for (int i = 0; i < kW; ++i) {
    sum += sm.sum[i];
    top_key = top_key > sm.top[i] ? top_key : sm.top[i];
    best = best > sm.best[i] ? best : sm.best[i];
  }
  RowChunk out;
  out.ref = 0.0f;
  out.bad = top_key >= F32T::key(0x7F800000u) ? 1 : 0;
  if constexpr (GREEDY) {
    out.best = best;
    return out;
  }
  if (out.bad || top_key <= F32T::key(0xFF800000u)) {
    sum = 0.0;  // nothing but -inf, or a row that does not count
  } else {
    const float all = __uint_as_float(F32T::raw_of_key(top_key));
    if (all > kHighMax || all < kLowMax) {  // read again, in 64 bits and less the maximum
      out.ref = all;
      double part = te >= 0 ? exp_from(xe, all) : 0.0;
#pragma unroll 1
      for (int i = tid; i < cnt; i += kT) {
        const vec_t q = __builtin_amdgcn_raw_buffer_load_b128(rs, i * 16, 0, 0);
#pragma unroll
        for (int j = 0; j < P; ++j) part += exp_from(DT::value(lane_of<raw_t>(q, j)), all);
      }
      part = wave_sum_f64(part);
      __syncthreads();
      if (lane == 0) sm.sum[wave] = part;
      __syncthreads();
      sum = 0.0;
#pragma unroll
      for (int i = 0; i < kW; ++i) sum += sm.sum[i];
    }
  }
  out.sum = sum;
  return out;
}

template <class DT, bool GREEDY, bool KEEP>
__device__ __forceinline__ void put_chunk(const VerifyArgs& a, int64_t seq, bool target, int w, int ch, Split split,
                                          RowChunk* stats, ChunkSmem& sm) {
  const RowChunk c = chunk_of<DT, GREEDY, KEEP>(target ? target_row<DT>(a, seq, w) : draft_row<DT>(a, seq, w), a.V, ch, split, sm);
  RowChunk* out = const_cast<RowChunk*>(target ? target_stats(a, stats, split.chunks, seq, w)
                                               : draft_stats(a, stats, split.chunks, seq, w)) + ch;
  if (threadIdx.x == 0) *out = c;
}

// Chunks of rows. Workgroups of a sequence: its first `targets` target rows, then its
// draft rows, if there are any. KEEP: rows may stay in the caches, where the last
// kernel finds them.
template <class DT, bool GREEDY, bool KEEP>
__global__ __launch_bounds__(kT) void verify_rows_kernel(VerifyArgs a, Split split, int targets, int64_t seq0,
                                                         RowChunk* __restrict__ stats, uint32_t* __restrict__ arrived) {
  __shared__ ChunkSmem sm;
  const int rows = targets + (a.draft_logits == nullptr ? 0 : a.D);
  const unsigned b = blockIdx.x;
  const int ch = static_cast<int>(b % static_cast<unsigned>(split.chunks));
  const unsigned item = b / static_cast<unsigned>(split.chunks);
  const int r = static_cast<int>(item % static_cast<unsigned>(rows));
  const int64_t seq = seq0 + item / static_cast<unsigned>(rows);
  if (r == 0 && ch == 0 && threadIdx.x == 0) arrived[kApart * seq] = 0;
  const bool target = r < targets;
  const int w = target ? r : r - targets;
  const int n = draft_count(a, seq);
  if (target ? w > n : w >= n) return;
  put_chunk<DT, GREEDY, KEEP>(a, seq, target, w, ch, split, stats, sm);
}

template <class DT, int THREADS>
constexpr bool kTabled = THREADS == kMany && DT::kPerVec == 8 && DT::kNegInf == 0xFF80u;
struct NoTable {};
struct Table {
  double table[kTable];
};
template <class DT, int THREADS, Mode MODE>
struct FinalSmem : std::conditional_t<kTabled<DT, THREADS> && MODE != kGreedy, Table, NoTable> {
  static constexpr int kWaves = kFew / kWave;  // that find the token
  WalkSmem walk;
  int32_t out[kMaxRows];  // rejected tokens within the range
  int outs;
  double sum[4][kWaves];
  double parts[2][kFew];  // sums of the parts: of what is left, where summed again, and of p
  uint64_t is[kWaves], may[kWaves];
  double below;
  int last;
  int found, sure;
};

// The terms of eight neighbouring elements: p's, and q's.
struct Terms {
  double p[kBlock], q[kBlock];
};
// Elements of less than exp(-70) of the row are left out where a whole wave has none but
// them: rows that were filtered. All together they are below kFarShare of the row an
// element, and only a uniform closer than that to a token's border, as 0 is to the first
// one's, has the row summed again with them.
// The least that count: where the logits are so large that 70 less is the same number,
// that of the largest.
constexpr float kFar = 70.0f;
constexpr double kFarShare = 0x1p-100;  // exp(-70) is 2^-100.99
struct Rows {
  float p_least, q_least;
};
__device__ __forceinline__ float log_below(double sum) {  // no more than ln 2 below the logarithm
  return static_cast<float>(static_cast<int>(__builtin_bit_cast(uint64_t, sum) >> 52) - 1023) * kLn2;
}
__device__ __forceinline__ Rows least_of(const Walk& w) {
  Rows r;
  r.p_least = w.p.ref + (log_below(w.p.sum) - kFar);
  r.q_least = w.kind == kResidual ? w.q.ref + (log_below(w.q.sum) - kFar) : INFINITY;
  return r;
}
__device__ __forceinline__ float largest(const float (&x)[kBlock]) {
  return fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
}
// False if they are all left out, for the whole wave; all: none are.
template <class DT>
__device__ __forceinline__ bool terms_at(const typename DT::raw_t* prow, const typename DT::raw_t* qrow, int v, int V,
                                         const Walk& w, const Rows& least, bool all, bool two, Terms& t) {
  float x[kBlock], y[kBlock];
  load_block<DT>(prow, v, V, x);
  bool some = all || largest(x) >= least.p_least;
  if (two) {
    load_block<DT>(qrow, v, V, y);
    some |= largest(y) >= least.q_least;
  }
  if (__ballot(some) == 0) return false;
#pragma unroll
  for (int j = 0; j < kBlock; ++j) t.p[j] = exp_from(x[j], w.p.ref);
  if (two) {
#pragma unroll
    for (int j = 0; j < kBlock; ++j) t.q[j] = exp_from(y[j], w.q.ref);
  }
  return true;
}

// The rejected tokens within [first, end).
template <class Smem>
__device__ __forceinline__ void list_out(const VerifyArgs& a, const Walk& w, int first, int end, Smem& sm) {
  if (w.kind != kWithout) return;
  const int tid = threadIdx.x;
  __syncthreads();
  if (tid == 0) sm.outs = 0;
  __syncthreads();
  if (tid < a.D && sm.walk.node[tid] == w.node) {
    const int t = sm.walk.token[tid];
    if (t >= first && t < end) sm.out[atomicAdd(&sm.outs, 1)] = t;
  }
  __syncthreads();
}
// Which of the elements v .. v + 7 are among them: bits.
template <class Smem>
__device__ __forceinline__ uint32_t outs_at(int v, const Smem& sm) {
  uint32_t mask = 0;
  const int n = sm.outs;
  for (int i = 0; i < n; ++i) {
    const uint32_t at = static_cast<uint32_t>(sm.out[i] - v);
    if (at < kBlock) mask |= 1u << at;
  }
  return mask;
}

// The workgroup's sums of v[0 .. COUNT), in all threads.
template <int COUNT, int WAVES>
__device__ __forceinline__ void block_sums(double (&v)[COUNT], double (&at)[4][WAVES]) {
#pragma unroll
  for (int i = 0; i < COUNT; ++i) v[i] = wave_sum_f64(v[i]);
  __syncthreads();
  if (threadIdx.x % kWave == 0) {
#pragma unroll
    for (int i = 0; i < COUNT; ++i) at[i][threadIdx.x / kWave] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < COUNT; ++i) {
    v[i] = 0.0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) v[i] += at[i][w];
  }
}
// The sums of v over the threads below, up to this one, and over all. What one
// thread gets as its end is what the next one gets as its beginning.
template <int WAVES>
__device__ __forceinline__ void block_scan(double v, double& below, double& upto, double& all, double (&at)[4][WAVES]) {
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  const double end = wave_incl_scan_f64(v);
  const double begin = __shfl_up(end, 1);
  __syncthreads();
  if (lane == kWave - 1) at[0][wave] = end;
  __syncthreads();
  double base = 0.0;
  all = 0.0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    if (w == wave) base = all;
    all += at[0][w];
  }
  below = lane == 0 ? base : base + begin;
  upto = base + end;
}

// v, or next to 0 (below 2^-1022): one instruction, where a choice of both halves takes two.
__device__ __forceinline__ double if_or_none(bool is, double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t high = is ? static_cast<uint32_t>(u >> 32) : 0u;
  return __builtin_bit_cast(double, (static_cast<uint64_t>(high) << 32) | static_cast<uint32_t>(u));
}

// Eight elements' share of a part's sums; p > q where near * p's term > q's.
__device__ __forceinline__ void add_terms(FinalPart& mine, const Terms& t, double near) {
  bool close = false;
#pragma unroll
  for (int j = 0; j < kBlock; ++j) {
    const double more = __builtin_fma(near, t.p[j], -t.q[j]);
    mine.all += t.p[j];
    mine.draft += t.q[j];
    mine.left += __builtin_fmax(more, 0.0);
    mine.kept += if_or_none(more > 0.0, t.p[j]);
    close |= __builtin_fabs(more) < kBand * t.q[j];
  }
  if (__ballot(close) != 0) {
#pragma unroll
    for (int j = 0; j < kBlock; ++j) {
      const double more = __builtin_fma(near, t.p[j], -t.q[j]);
      const bool is = __builtin_fabs(more) < kBand * t.q[j];
      mine.left -= if_or_none(is && more > 0.0, more);
      mine.kept -= if_or_none(is && more > 0.0, t.p[j]);
      mine.close += if_or_none(is, t.q[j]);
    }
  }
}

// Sums over a wave's part of the row, of every lane's elements.
template <class DT, Mode MODE, class Smem>
__device__ __forceinline__ FinalPart part_of(const typename DT::raw_t* prow, const typename DT::raw_t* qrow, int first,
                                             int pieces, int V, const Walk& w, const Smem& sm) {
  FinalPart mine{};
  const Rows least = least_of(w);
  const int lane = threadIdx.x % kWave;
  if (MODE == kDrawn && w.kind == kResidual) {
    const double near = w.q.sum / w.p.sum;
#pragma unroll 1
    for (int i = 0; i < pieces; ++i) {
      const int v = first + i * kPiece + lane * kBlock;
      Terms t;
      if (!terms_at<DT>(prow, qrow, v, V, w, least, false, true, t)) continue;
      add_terms(mine, t, near);
    }
  } else {
    const bool outs = MODE != kDrawn && w.kind == kWithout && sm.outs != 0;
#pragma unroll 1
    for (int i = 0; i < pieces; ++i) {
      const int v = first + i * kPiece + lane * kBlock;
      Terms t;
      if (!terms_at<DT>(prow, qrow, v, V, w, least, false, false, t)) continue;
      double sum = 0.0;
#pragma unroll
      for (int j = 0; j < kBlock; ++j) sum += t.p[j];
      mine.all += sum;
      if (outs) {
        const uint32_t gone = outs_at(v, sm);
        sum = 0.0;
#pragma unroll
        for (int j = 0; j < kBlock; ++j) sum += (gone >> j & 1u) != 0 ? 0.0 : t.p[j];
      }
      mine.left += sum;
    }
  }
  return mine;
}

// bf16 rows whose references are 0, as a model's logits have: there are so few
// values that exp of all of them fits shared memory. A look-up takes 5 instructions
// and 10 or so cycles of shared memory, where the polynomial takes 17: 52 us and 61 for
// 64 sequences of 4 drafts with draft logits, V 151936. (Workgroups of kFew threads have
// too little room and time to fill it.)
template <int FIRST, int THREADS>
__device__ __forceinline__ void fill_table(double (&table)[kTable]) {  // by threads FIRST and up
  for (int m = kTableLow + threadIdx.x - FIRST; m <= kTableHigh; m += THREADS - FIRST)
    table_pair(m, table[m - kTableLow], table[kTableSign + m - kTableLow]);
}
using pair_t = uint16_t __attribute__((ext_vector_type(2)));
// The terms of two elements of a row.
__device__ __forceinline__ void look_up(const double (&table)[kTable], uint32_t word, double& first, double& second) {
  const uint32_t size = word & 0x7FFF7FFFu;
  pair_t m = __builtin_bit_cast(pair_t, size);
  m = __builtin_elementwise_max(m, pair_t{kTableLow, kTableLow});
  m = __builtin_elementwise_min(m, pair_t{kTableHigh, kTableHigh});
  m = m - pair_t{kTableLow, kTableLow};
  const uint32_t at = __builtin_bit_cast(uint32_t, m) | (word >> 2 & (kTableSign * 0x10001u));
  first = table[at & 0xFFFFu];
  second = table[at >> 16];
}
__device__ __forceinline__ vec_t load_words(const uint16_t* row, int v, int V) {
  vec_t q;
  if (v + kBlock <= V) {
    __builtin_memcpy(&q, row + v, 16);
  } else {
    q = vec_t{0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u};
#pragma unroll
    for (int j = 0; j < kBlock; ++j)
      if (v + j < V) set_lane<uint16_t>(q, j, row[v + j]);
  }
  return q;
}
__device__ __forceinline__ bool all_masked(const vec_t& q) {
  return (q.x & q.y & q.z & q.w) == 0xFF80FF80u && (q.x | q.y | q.z | q.w) == 0xFF80FF80u;
}
template <Mode MODE, class Smem>
__device__ __forceinline__ FinalPart part_by_table(const uint16_t* prow, const uint16_t* qrow, int first, int pieces, int V,
                                                   const Walk& w, const Smem& sm, const double (&table)[kTable]) {
  FinalPart mine{};
  const int lane = threadIdx.x % kWave;
  const bool two = MODE == kDrawn && w.kind == kResidual;
  const bool outs = MODE != kDrawn && w.kind == kWithout && sm.outs != 0;
  const double near = two ? w.q.sum / w.p.sum : 0.0;
  vec_t x = load_words(prow, first + lane * kBlock, V), y = x;
  if (two) y = load_words(qrow, first + lane * kBlock, V);
#pragma unroll 1
  for (int i = 0; i < pieces; ++i) {
    const int v = first + i * kPiece + lane * kBlock;
    const vec_t xn = x, yn = y;
    if (i + 1 < pieces) {  // the next ones are on their way
      x = load_words(prow, v + kPiece, V);
      if (two) y = load_words(qrow, v + kPiece, V);
    }
    if (__ballot(!(all_masked(xn) && (!two || all_masked(yn)))) == 0) continue;
    Terms t;
#pragma unroll
    for (int j = 0; j < kBlock; j += 2) look_up(table, vword(xn, j / 2), t.p[j], t.p[j + 1]);
    if (two) {
#pragma unroll
      for (int j = 0; j < kBlock; j += 2) look_up(table, vword(yn, j / 2), t.q[j], t.q[j + 1]);
      add_terms(mine, t, near);
    } else {
      double sum = 0.0;
#pragma unroll
      for (int j = 0; j < kBlock; ++j) sum += t.p[j];
      mine.all += sum;
      if (outs) {
        const uint32_t gone = outs_at(v, sm);
        sum = 0.0;
#pragma unroll
        for (int j = 0; j < kBlock; ++j) sum += (gone >> j & 1u) != 0 ? 0.0 : t.p[j];
      }
      mine.left += sum;
    }
  }
  return mine;
}

// What the row's elements weigh: scale * p's term less q's, or p's term, or nothing.
struct Weights {
  double scale;
  bool residual, without;
  template <class Smem>
  __device__ __forceinline__ void of(const Terms& t, int v, const Smem& sm, double (&wt)[kBlock]) const {
    uint32_t gone = 0;
    if (without) gone = outs_at(v, sm);
#pragma unroll
    for (int j = 0; j < kBlock; ++j) {
      const double more = residual ? __builtin_fma(scale, t.p[j], -t.q[j]) : t.p[j];
      wt[j] = more > 0.0 && (gone >> j & 1u) == 0 ? more : 0.0;
    }
  }
};

// The first thread for which `is` holds, or else the last one for which `may` does; -1 for none.
template <class Smem>
__device__ __forceinline__ int first_or_last(bool is, bool may, Smem& sm) {
  constexpr int THREADS = kFew;
  const int wave = threadIdx.x / kWave;
  const uint64_t a = __ballot(is), b = __ballot(may);
  if (threadIdx.x % kWave == 0) {
    sm.is[wave] = a;
    sm.may[wave] = b;
  }
  __syncthreads();
  int first = -1, last = -1;
#pragma unroll
  for (int i = THREADS / kWave - 1; i >= 0; --i)
    if (sm.is[i] != 0) first = i * kWave + __builtin_ctzll(sm.is[i]);
#pragma unroll
  for (int i = 0; i < THREADS / kWave; ++i)
    if (sm.may[i] != 0) last = i * kWave + 63 - __builtin_clzll(sm.may[i]);
  __syncthreads();
  return first >= 0 ? first : last;
}

// Finds the token out of the parts' sums, by the first kFew threads (the other waves
// have ended, and barriers wait for none of them).
//
// Parts were summed with near, the ratio of q's sum and p's out of the chunks; scale is
// that ratio in 64 bits. For elements that are not close both tell the same one of p
// and q to be larger, and left + (scale - near) kept is what they add up to. The close
// ones and those that are too far below the row's largest add up to at most `more`:
// where that could move the token, and where scale is not as near as that, the parts
// are summed again, with scale and of all elements.
template <class DT, Mode MODE, class Smem>
__device__ __forceinline__ int token_of(const VerifyArgs& a, const Walk& w, const Meeting& meet, int parts, int pieces,
                                        const typename DT::raw_t* prow, const typename DT::raw_t* qrow,
                                        Smem& sm) {
  constexpr int THREADS = kFew, kWaves = THREADS / kWave;
  const int tid = threadIdx.x, span = pieces * kPiece;
  const bool two = MODE == kDrawn && w.kind == kResidual;
  const Rows least = least_of(w);
  FinalPart p{};
  if (tid < parts) {
    const double* from = meet.sums + tid;
    p.all = get_far(from);
    p.left = get_far(from + parts);
    if (two) {
      p.kept = get_far(from + 2 * parts);
      p.draft = get_far(from + 3 * parts);
      p.close = get_far(from + 4 * parts);
    }
  }
  double total[MODE == kDrawn ? 3 : 1];
  total[0] = p.all;
  if constexpr (MODE == kDrawn) {
    total[1] = p.draft;
    total[2] = p.close;
  }
  sm.parts[1][tid] = p.all;
  block_sums(total, sm.sum);
  double part = p.left, scale = 1.0, more = 0.0, least_mass = kLeast * total[0];
  bool again = false;
  if constexpr (MODE == kDrawn) {
    more = a.V * kFarShare * total[0];
    if (two) {
      scale = total[1] / total[0];
      const double near = w.q.sum / w.p.sum, off = scale - near;
      part = __builtin_fmax(__builtin_fma(off, p.kept, part), 0.0);
      more = 2.0 * kBand * total[2] + a.V * kFarShare * total[1];
      least_mass = kLeast * total[1];
      again = __builtin_fabs(off) > 0.5 * kBand * near;
    }
  }
  for (;;) {
    if (again) {
      if constexpr (MODE == kProposed) list_out(a, w, 0, a.V, sm);
      const bool outs = MODE != kDrawn && w.kind == kWithout;
      for (int c0 = 0; c0 < parts; c0 += kWaves) {
        const int c = c0 + tid / kWave;
        double sum = 0.0, whole = 0.0;
#pragma unroll 1
        for (int i = 0; i < pieces; ++i) {
          const int v = c * span + i * kPiece + tid % kWave * kBlock;
          float x[kBlock], y[kBlock];
          load_block<DT>(prow, v, a.V, x);
          if constexpr (MODE == kDrawn) load_block<DT>(qrow, v, a.V, y);
          const uint32_t gone = outs ? outs_at(v, sm) : 0u;
#pragma unroll 1
          for (int j = 0; j < kBlock; ++j) {  // one after the other: rarely taken
            const double one = exp_from(x[0], w.p.ref);
            double left = (gone >> j & 1u) != 0 ? 0.0 : one;
            if constexpr (MODE == kDrawn) {
              const double more_than_q = __builtin_fmax(__builtin_fma(scale, one, -exp_from(y[0], w.q.ref)), 0.0);
              left = two ? more_than_q : one;
            }
            whole += one;
            sum += left;
#pragma unroll
            for (int k = 0; k + 1 < kBlock; ++k) {
              x[k] = x[k + 1];
              if constexpr (MODE == kDrawn) y[k] = y[k + 1];
            }
          }
        }
        sum = wave_sum_f64(sum);
        whole = wave_sum_f64(whole);
        if (tid % kWave == 0) {
          sm.parts[0][c] = sum;
          sm.parts[1][c] = whole;
        }
      }
      __syncthreads();
      part = tid < parts ? sm.parts[0][tid] : 0.0;
      more = 0.0;
    }
    Weights weights{scale, two, MODE != kDrawn && w.kind == kWithout};
    double below, upto, all;
    block_scan(part, below, upto, all, sm.sum);
    if (w.kind != kPlain && !(all > least_mass)) {
      if (!again) {
        again = true;
        continue;
      }
      weights.residual = weights.without = false;
      part = tid < parts ? sm.parts[1][tid] : 0.0;
      block_scan(part, below, upto, all, sm.sum);
    }
    // from a uniform of 1 on the last token of any weight, which roundings of the sums must not hide
    const double at = sm.walk.last_u < 1.0f ? static_cast<double>(sm.walk.last_u) * all : INFINITY;
    // Without q what is left out moves a border by less than the roundings of one at
    // 2^-26 of the row, so that only uniforms below that or from 1 on need all elements.
    if (MODE != kDrawn && !again && !(at >= 0x1p-26 * total[0] && at < all)) {
      again = true;
      continue;
    }
    // the part that `at` lies in, else the last one of any weight
    bool is = part > 0.0 && upto > at, may = part > 0.0;
    const double begin = below;
    int last_seen = -1;
    bool sure = more == 0.0;
    for (;;) {
      const int c = first_or_last(is, may, sm);
      if (c < 0) break;
      if (tid == c) sm.below = begin;
      __syncthreads();
      double base = sm.below;
      if constexpr (MODE == kProposed) list_out(a, w, c * span, (c + 1) * span, sm);
#pragma unroll 1
      for (int i = 0; i < span; i += THREADS * kBlock) {
        const int v = i + tid * kBlock < span ? c * span + i + tid * kBlock : a.V;
        double wt[kBlock], sum = 0.0;
        int last = -1;  // the last element of any weight
        Terms t;
        if (terms_at<DT>(prow, qrow, v, a.V, w, least, again, two, t)) {
          weights.of(t, v, sm, wt);
#pragma unroll
          for (int j = 0; j < kBlock; ++j) {
            sum += wt[j];
            if (wt[j] > 0.0) last = v + j;
          }
        }
        block_scan(sum, below, upto, all, sm.sum);
        const bool here = last >= 0 && base + upto > at;
        const int finder = first_or_last(here, last >= 0, sm);
        if (finder >= 0) {
          if (tid == finder) {
            int token = -1;
            double reach = base + below;
            bool clear = false;
#pragma unroll
            for (int j = 0; j < kBlock; ++j) {
              [[maybe_unused]] const double from = reach;
              reach += wt[j];
              if (token < 0 && wt[j] > 0.0 && reach > at) {
                token = v + j;
                if constexpr (MODE == kDrawn) clear = from + more <= at && at + more < reach;
              }
            }
            sm.found = token >= 0 ? token : last;
            sm.last = here ? 1 : 0;
            if constexpr (MODE == kDrawn) sm.sure = clear ? 1 : 0;
          }
          __syncthreads();
          last_seen = sm.found;
          if constexpr (MODE == kDrawn) sure = more == 0.0 || sm.sure != 0;
          const bool done = sm.last != 0;
          __syncthreads();
          if (done) break;
        }
        base += all;
      }
      if (last_seen >= 0) break;
      // its weight was but roundings, or elements that are left out
      if (tid == c) is = may = false;
    }
    if (sure) return last_seen;
    again = true;
  }
}

// A group's parts of the row where the path ends, one of each wave. Then the last
// of a sequence's `groups` workgroups finds the token; -2 for the others.
template <class DT, Mode MODE, int THREADS>
__device__ __forceinline__ int token_by_parts(const VerifyArgs& a, const Walk& w, int64_t seq, int group, int groups,
                                              int pieces, const Meeting& meet,
                                              FinalSmem<DT, THREADS, MODE>& sm) {
  using raw_t = typename DT::raw_t;
  constexpr int kWaves = THREADS / kWave;
  const int tid = threadIdx.x;
  const raw_t* prow = target_row<DT>(a, seq, w.node);
  const bool two = MODE == kDrawn && w.kind == kResidual;
  const raw_t* qrow = two ? draft_row<DT>(a, seq, w.node) : prow;
  const int span = pieces * kPiece, parts = groups * kWaves;
  if constexpr (MODE == kProposed) list_out(a, w, group * kWaves * span, (group + 1) * kWaves * span, sm);
  const int c = group * kWaves + tid / kWave;
  FinalPart mine;
  if constexpr (kTabled<DT, THREADS>) {
    if (w.p.ref == 0.0f && (!two || w.q.ref == 0.0f)) {
      mine = part_by_table<MODE>(prow, qrow, c * span, pieces, a.V, w, sm, sm.table);
    } else {
      mine = part_of<DT, MODE>(prow, qrow, c * span, pieces, a.V, w, sm);
    }
  } else {
    mine = part_of<DT, MODE>(prow, qrow, c * span, pieces, a.V, w, sm);
  }
  mine.all = wave_sum_f64(mine.all);
  mine.left = wave_sum_f64(mine.left);
  if (two) {
    mine.kept = wave_sum_f64(mine.kept);
    mine.draft = wave_sum_f64(mine.draft);
    if (__ballot(mine.close > 0.0) != 0) mine.close = wave_sum_f64(mine.close);
  }
  if (tid % kWave == 0) {
    double* to = meet.sums + c;
    put_far(to, mine.all);
    put_far(to + parts, mine.left);
    if (two) {
      put_far(to + 2 * parts, mine.kept);
      put_far(to + 3 * parts, mine.draft);
      put_far(to + 4 * parts, mine.close);
    }
  }
  if (!last_of(meet.arrived, groups, sm.last) || tid >= kFew) return -2;
  return token_of<DT, MODE>(a, w, meet, parts, pieces, prow, qrow, sm);
}

struct BehindSmem {
  WalkSmem walk;
  ChunkSmem chunk;
  int32_t rows[kMaxRows];
  uint64_t is[kW];
};
// The rows of a tree at and behind row `node`, in sm.rows; how many.
__device__ __forceinline__ int list_behind(int node, int n, BehindSmem& sm) {
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const bool in = tid <= n && row_behind(tid, node, sm.walk.token, sm.walk.node);
  const uint64_t mask = __ballot(in);
  if (lane == 0) sm.is[wave] = mask;
  __syncthreads();
  int below = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kW; ++i) {
    if (i < wave) below += __builtin_popcountll(sm.is[i]);
    all += __builtin_popcountll(sm.is[i]);
  }
  if (in) sm.rows[below + lanes_below(mask)] = tid;
  __syncthreads();
  return all;
}

// Of a tree whose path goes on after `limit` drafts, chunks of the row where it
// stands, or (all) of that and the rows behind it.
template <class DT, Mode MODE>
__global__ __launch_bounds__(kT, DT::kPerVec == 4 ? 4 : 5) void verify_behind_kernel(VerifyArgs a, Split split, int limit,
                                                                                     bool all, int groups, int64_t seq0,
                                                                                     RowChunk* stats) {
  __shared__ BehindSmem sm;
  const int group = static_cast<int>(blockIdx.x % static_cast<unsigned>(groups));
  const int64_t seq = seq0 + blockIdx.x / static_cast<unsigned>(groups);
  const Walk w = walk<DT, MODE>(a, stats, split.chunks, limit, seq, sm.walk);
  if (!w.open) return;
  const int rows = all ? list_behind(w.node, draft_count(a, seq), sm) : 1;
  for (int i = group; i < rows * split.chunks; i += groups) {
    const int k = i / split.chunks, ch = i - k * split.chunks;
    put_chunk<DT, MODE == kGreedy, true>(a, seq, true, all ? sm.rows[k] : w.node, ch, split, stats, sm.chunk);
  }
}

// The end of every path, and the row where it lies.
template <class DT, Mode MODE, int THREADS>
__global__ __launch_bounds__(THREADS) void verify_final_kernel(VerifyArgs a, int chunks, int groups, int pieces,
                                                               int64_t seq0, const RowChunk* __restrict__ stats,
                                                               Meeting all) {
  __shared__ FinalSmem<DT, THREADS, MODE> sm;
  constexpr bool greedy = MODE == kGreedy;
  const int tid = threadIdx.x;
  const int group = static_cast<int>(blockIdx.x % static_cast<unsigned>(groups));
  const int64_t seq = seq0 + blockIdx.x / static_cast<unsigned>(groups);
  if constexpr (kTabled<DT, THREADS> && MODE != kGreedy) {
    if (tid >= kT) fill_table<kT, THREADS>(sm.table);  // while the others go down the path
  }
  const Walk w = walk<DT, MODE>(a, stats, chunks, a.D + 1, seq, sm.walk);
  int32_t* tokens = a.out_tokens + seq * (a.D + 1);
  const bool draws = !greedy && w.kind != kNone;
  if (group == 0) {
    if (tid <= a.D && !(tid == w.count && draws))
      tokens[tid] = tid < w.count ? sm.walk.token[sm.walk.path[tid]]
                                  : (tid == w.count && greedy ? best_token(w.best) : -1);
    if (a.out_path != nullptr && tid < a.D) a.out_path[seq * a.D + tid] = tid < w.count ? sm.walk.path[tid] : -1;
    if (tid == 0) a.out_accepted[seq] = w.count;
  }
  if constexpr (!greedy) {
    if (!draws) return;
    const Meeting meet{all.sums + seq * groups * (THREADS / kWave) * kSums, all.arrived + kApart * seq};
    const int token = token_by_parts<DT, MODE, THREADS>(a, w, seq, group, groups, pieces, meet, sm);
    if (tid == 0 && token >= -1) tokens[w.count] = token;
  }
}

// Rows of no more than the last-level cache are left there: 64 sequences of 4 drafts,
// 175 MB, take 54.0 us so and 56.3 past it, 128 of 3 drafts, 460 MB, 113.4 and 111.7.
constexpr int64_t kKeptBytes = int64_t{256} << 20;

struct Layout {
  int64_t stats, finals, arrived, bytes;
};
Layout layout_of(const Plan& p, int64_t N, int D, bool draft) {
  const int64_t rows = N * (D + 1 + (draft ? D : 0));
  Layout l;
  l.stats = 0;
  l.finals = l.stats + rows * p.split.chunks * static_cast<int64_t>(sizeof(RowChunk));
  l.arrived = l.finals + N * p.cut.groups * (p.cut.threads / kWave) * static_cast<int64_t>(sizeof(FinalPart));
  l.bytes = l.arrived + N * kApart * 4;
  return l;
}

template <class DT, Mode MODE>
hipError_t launch_mode(int dtype, const VerifyArgs& a, hipStream_t stream) {
  const bool draft = MODE == kDrawn, greedy = MODE == kGreedy;
  const Plan p = plan_of(dtype, a.N, a.D, a.V, draft, a.parents != nullptr);
  const Layout l = layout_of(p, a.N, a.D, draft);
  char* ws = static_cast<char*>(a.workspace);
  RowChunk* stats = reinterpret_cast<RowChunk*>(ws + l.stats);
  const Meeting meet{reinterpret_cast<double*>(ws + l.finals), reinterpret_cast<uint32_t*>(ws + l.arrived)};
  const bool keep = a.N * (targets_of(p, a.D) + (draft ? a.D : 0)) * a.V * (dtype == 0 ? 4 : 2) <= kKeptBytes;
  const int targets = targets_of(p, a.D), groups = final_groups(p, greedy);
  const int64_t of_rows = rows_groups(p, a.D, draft);
  const int behind = p.steps > 0 ? behind_groups(a.N, a.D, p.split) : 0;
  const int64_t step = sequences_of_launch(p, a.N, a.D, draft, greedy);
  for (int64_t i = 0; i < a.N; i += step) {
    const int64_t n = a.N - i < step ? a.N - i : step;
    auto grid = [&](int64_t of) { return dim3(static_cast<unsigned>(n * of)); };
    if (keep)
      hipLaunchKernelGGL((verify_rows_kernel<DT, greedy, true>), grid(of_rows), dim3(kT), 0, stream, a, p.split, targets, i,
                         stats, meet.arrived);
    else
      hipLaunchKernelGGL((verify_rows_kernel<DT, greedy, false>), grid(of_rows), dim3(kT), 0, stream, a, p.split, targets,
                         i, stats, meet.arrived);
    if (const hipError_t e = hipGetLastError()) return e;
    if constexpr (!draft) {
      for (int limit = 1; limit <= p.steps; ++limit) {
        const bool all = limit == p.steps;
        const int of = all ? behind : p.split.chunks;
        hipLaunchKernelGGL((verify_behind_kernel<DT, MODE>), grid(of), dim3(kT), 0, stream, a, p.split, limit, all, of, i,
                           stats);
        if (const hipError_t e = hipGetLastError()) return e;
      }
    }
    if (final_threads(p, greedy) == kFew)
      hipLaunchKernelGGL((verify_final_kernel<DT, MODE, kFew>), grid(groups), dim3(kFew), 0, stream, a, p.split.chunks,
                         groups, p.cut.pieces, i, stats, meet);
    else if constexpr (!greedy)
      hipLaunchKernelGGL((verify_final_kernel<DT, MODE, kMany>), grid(groups), dim3(kMany), 0, stream, a, p.split.chunks,
                         groups, p.cut.pieces, i, stats, meet);
    if (const hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

template <class DT>
hipError_t launch_typed(int dtype, const VerifyArgs& a, hipStream_t stream) {
  if (a.uniforms == nullptr) return launch_mode<DT, kGreedy>(dtype, a, stream);
  if (a.draft_logits != nullptr) return launch_mode<DT, kDrawn>(dtype, a, stream);
  return launch_mode<DT, kProposed>(dtype, a, stream);
}

}  // namespace

int64_t verify_workspace(int dtype, int64_t N, int D, int V, bool draft_logits) {
  const int64_t chain = layout_of(plan_of(dtype, N, D, V, draft_logits, false), N, D, draft_logits).bytes;
  const int64_t tree = draft_logits ? 0 : layout_of(plan_of(dtype, N, D, V, false, true), N, D, false).bytes;
  return chain > tree ? chain : tree;
}

hipError_t launch_verify(int dtype, const VerifyArgs& a, hipStream_t stream) {
  if (dtype == 0) return launch_typed<F32T>(dtype, a, stream);
  if (dtype == 1) return launch_typed<F16T>(dtype, a, stream);
  return launch_typed<BF16T>(dtype, a, stream);
}

}  // namespace tkp
