// Caches kept in pages: rows of a page table that follow their beams, rows that
// grow and shrink, and entries that move within their row.
//
// A page's uses are how many entries of the table name it; one with no uses is
// free. So a fork only writes tables and uses, whatever the pages hold: rows share
// pages until one of them writes into one, which is when it grows and its last
// page is not full. Then the page is copied (all but the last row that shares it).
// Free pages are given out from the lowest number on, so results do not depend on
// the order in which threads run.

#include "cache_pages.h"
#include "device_common.h"

namespace tkp {
namespace {

constexpr int kForkThreads = 256;
constexpr int kForkWaves = kForkThreads / kWave;
constexpr int kForkCols = kWave;
constexpr int kMaxBeams = 128;

__device__ __forceinline__ int pages_of(int length, int S, int C) {
  const int n = length <= 0 ? 0 : (length - 1) / S + 1;
  return n < C ? n : C;
}
__device__ __forceinline__ bool is_page(int32_t page, int64_t P) { return page >= 0 && page < P; }

// 64 columns of one prompt's rows. They pass through shared memory, as any row may
// follow any other. It reads and writes whole pieces of 256 bytes and is bound by its
// steps that hang on one another: 64 prompts of 8 beams and 2048 columns, 5 MB, take
// 6.8 us, one prompt of 64 columns 2.1. The prompt's workgroups here begin at column
// tile0 * 64. LENGTHS: the prompt has no other workgroup, which would still have to read
// the lengths.
template <bool LENGTHS>
__global__ __launch_bounds__(kForkThreads) void pages_fork_kernel(PageTable t, const int32_t* __restrict__ parents, int K,
                                                                  int tiles, int tile0, int64_t item0) {
  __shared__ int32_t held[kMaxBeams][kForkCols];
  __shared__ int32_t parent[kMaxBeams];
  __shared__ int32_t pages[kMaxBeams];
  __shared__ int32_t length[kMaxBeams];
  __shared__ int32_t kids[kMaxBeams];
  __shared__ uint64_t apart[kForkWaves];  // columns whose entries are not all the same page
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int tile = tile0 + static_cast<int>(blockIdx.x % static_cast<unsigned>(tiles));
  const int64_t item = item0 + blockIdx.x / static_cast<unsigned>(tiles);
  if (tid < K) {
    const int p = parents[item * K + tid];
    parent[tid] = p >= 0 && p < K ? p : tid;
    length[tid] = t.lengths[item * K + tid];
    pages[tid] = pages_of(length[tid], t.S, t.C);
    kids[tid] = 0;
  }
  __syncthreads();
  if (tid < K) atomicAdd(&kids[parent[tid]], 1);
  if (LENGTHS && tid < K) t.lengths[item * K + tid] = length[parent[tid]];
  const int col = tile * kForkCols + lane;
  int32_t* table = t.tables + item * K * t.ld;
  for (int b = wave; b < K; b += kForkWaves) held[b][lane] = col < pages[b] ? table[b * t.ld + col] : -1;
  __syncthreads();
  bool same = true;
  for (int b = wave; b < K; b += kForkWaves) same = same && held[b][lane] == held[0][lane];
  const uint64_t mask = __ballot(!same);
  if (lane == 0) apart[wave] = mask;
  __syncthreads();
  uint64_t differ = 0;
#pragma unroll
  for (int w = 0; w < kForkWaves; ++w) differ |= apart[w];
  for (int b = wave; b < K; b += kForkWaves) {
    // entries that all rows share stay as many
    const int32_t page = held[b][lane];
    if (kids[b] != 1 && ((differ >> lane) & 1u) != 0 && is_page(page, t.P)) atomicAdd(&t.uses[page], kids[b] - 1);
    const int p = parent[b];
    if (p != b && (col < pages[p] || col < pages[b])) table[b * t.ld + col] = held[p][lane];
  }
}

__global__ __launch_bounds__(kMaxBeams) void pages_fork_lengths_kernel(PageTable t, const int32_t* __restrict__ parents,
                                                                      int K, int64_t item0) {
  const int64_t item = item0 + blockIdx.x;
  const int b = threadIdx.x;
  int32_t length = 0;
  if (b < K) {
    const int p = parents[item * K + b];
    length = t.lengths[item * K + (p >= 0 && p < K ? p : b)];
  }
  __syncthreads();
  if (b < K) t.lengths[item * K + b] = length;
}

// ------------------------------------------------------------------ resize ---

constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / kWave;
constexpr int kScan = 16;     // pages of a thread in a group, which a step through the pool has four of
constexpr int kScanGroups = 4;
static_assert(kPlanThreads * kScan < 1 << 16);
constexpr int kFewPages = 4;  // more pages of a row are handled by the whole workgroup

// One page copied: `slots` slots of page `from` to page `to`.
struct PageCopy {
  int32_t from, to, slots;
};
struct ResizePlan {
  int32_t copies;
  int32_t pad[3];
};

enum Tail : int32_t { kNoTail = 0, kOwn = 1, kKeeps = 2, kCopies = 3 };
struct RowPlan {
  int32_t old_len, new_len;
  int32_t old_pages, new_pages;
  int32_t page;   // the last page, if the row is going to write into it
  int32_t tail;   // kOwn: nobody else uses it; kKeeps: the others leave it to this row; kCopies: they do not
  int32_t first;  // place of its first new page among the free ones
  int32_t serve;  // 1: the row gets what it needs
};

struct PlanSmem {
  uint64_t scan[kPlanWaves];
  int32_t many[2][kPlanThreads];  // rows that give back or get many pages
  int32_t many_count[2];
  int32_t shared;   // 1: a row writes into a page that is not its own
  int32_t blocked;  // the first row that would have to copy where nothing can be
  int32_t copies;
};

// The sum of v over the threads below, and of all.
__device__ __forceinline__ uint64_t plan_below(uint64_t v, uint64_t& all, PlanSmem& sm) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const uint64_t upto = wave_incl_scan_u64(v);
  __syncthreads();
  if (lane == kWave - 1) sm.scan[wave] = upto;
  __syncthreads();
  const uint64_t of = lane < kPlanWaves ? sm.scan[lane] : 0ull;
  const uint64_t sums = wave_incl_scan_u64(of);
  all = readlane_u64(sums, kPlanWaves - 1);
  const uint64_t before = wave == 0 ? 0ull : readlane_u64(sums, wave - 1);
  return before + upto - v;
}

__device__ __forceinline__ int32_t load_now(const int32_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void store_now(int32_t* p, int32_t v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Everything but the copies, by one workgroup: releases, last pages, needs, free
// pages, tables. It is a chain of dependent steps: lengths, last page, its uses, the
// free pages: 5 us for 64 rows and 16384 pages, where several workgroups would have to
// wait for one another at each step. Large pools that are nearly full are read by one
// compute unit: 72 us for 2^20 pages, 26 for 2^18. ONE: a row for each thread, which
// keeps its plan in registers.
template <bool ONE>
__global__ __launch_bounds__(kPlanThreads) void pages_resize_kernel(PageTable t, const int32_t* __restrict__ new_lengths,
                                                                   bool can_copy, RowPlan* __restrict__ plans,
                                                                   PageCopy* __restrict__ copies,
                                                                   ResizePlan* __restrict__ out,
                                                                   int32_t* __restrict__ pool) {
  __shared__ PlanSmem sm;
  const int tid = threadIdx.x;
  RowPlan held{};
  // f(r, plan) for this thread's rows
  auto rows = [&](auto f) {
    if constexpr (ONE) {
      if (tid < t.R) f(static_cast<int64_t>(tid), held);
    } else {
      for (int64_t r = tid; r < t.R; r += kPlanThreads) f(r, plans[r]);
    }
  };
  // f(r, plan, i) for every page i below count(plan) of the rows: by their threads
  // where these are few, else by a wave or, of few such rows, all waves, which need
  // the plan in memory
  auto each_page = [&](int which, auto count, auto f) {
    rows([&](int64_t r, RowPlan& p) {
      const int n = count(p);
      int at = kPlanThreads;
      if (n > kFewPages) at = atomicAdd(&sm.many_count[which], 1);
      if (at < kPlanThreads) {
        if constexpr (ONE) plans[r] = p;
        sm.many[which][at] = static_cast<int32_t>(r);
      } else {
        for (int i = 0; i < n; ++i) f(r, p, i);
      }
    });
    __syncthreads();
    const int n = sm.many_count[which] < kPlanThreads ? sm.many_count[which] : kPlanThreads;
    const int lanes = n < kPlanWaves ? kPlanThreads : kWave;
    for (int k = tid / lanes; k < n; k += kPlanThreads / lanes) {
      const int64_t r = sm.many[which][k];
      const RowPlan p = plans[r];
      const int m = count(p);
#pragma unroll 4
      for (int i = tid % lanes; i < m; i += lanes) f(r, p, i);
    }
  };

  if (tid == 0) {
    sm.many_count[0] = sm.many_count[1] = 0;
    sm.shared = 0;
    sm.blocked = 0x7FFFFFFF;
    sm.copies = 0;
  }
  rows([&](int64_t r, RowPlan& p) {
    p = RowPlan{};
    p.old_len = t.lengths[r];
    p.new_len = new_lengths[r];
    const int64_t most = static_cast<int64_t>(t.C) * t.S;
    if (p.old_len < 0 || p.old_len > most || p.new_len < 0 || p.new_len > most) p.old_len = p.new_len = 0;
    p.old_pages = pages_of(p.old_len, t.S, t.C);
    p.new_pages = pages_of(p.new_len, t.S, t.C);
    p.page = -1;
    if (p.new_len > p.old_len && p.old_len % t.S != 0) p.page = t.tables[r * t.ld + p.old_pages - 1];
  });
  __syncthreads();
  // pages behind the rows' new ends
  each_page(
      0, [](const RowPlan& p) { return p.new_len < p.old_len ? p.old_pages - p.new_pages : 0; },
      [&](int64_t r, const RowPlan& p, int i) {
        int32_t* entry = t.tables + r * t.ld + p.new_pages + i;
        if (is_page(*entry, t.P)) atomicSub(&t.uses[*entry], 1);
        *entry = -1;
      });
  // Rows that write into a page leave it. Where none stays, the last of them takes it
  // again, marked by -1 - row. If every row was its page's only user that is all;
  // else the last one is found by the smallest of the marks.
  rows([&](int64_t, RowPlan& p) {
    if (!is_page(p.page, t.P)) return;
    p.tail = kCopies;
    if (atomicSub(&t.uses[p.page], 1) != 1) sm.shared = 1;
  });
  __syncthreads();
  const bool shared = sm.shared != 0;
  rows([&](int64_t r, RowPlan& p) {
    if (p.tail == kNoTail) return;
    if (!shared) {
      p.tail = kOwn;
      store_now(&t.uses[p.page], static_cast<int32_t>(-1 - r));
    } else if (load_now(&t.uses[p.page]) <= 0) {
      atomicMin(&t.uses[p.page], static_cast<int32_t>(-1 - r));
    }
  });
  if (shared) {
    __syncthreads();
    rows([&](int64_t r, RowPlan& p) {
      if (p.tail != kCopies) return;
      if (load_now(&t.uses[p.page]) == static_cast<int32_t>(-1 - r)) p.tail = kKeeps;
      else if (!can_copy) atomicMin(&sm.blocked, static_cast<int32_t>(r));
    });
  }
  // what the rows need, one behind the other
  const uint64_t cap = static_cast<uint64_t>(t.P) + 1;  // more than there can be
  uint64_t need_all = 0;
  const int64_t end = ONE ? kPlanThreads : (t.R + kPlanThreads - 1) / kPlanThreads * kPlanThreads;
  auto need_of = [](const RowPlan& p) -> uint32_t {
    return p.new_len > p.old_len ? static_cast<uint32_t>(p.new_pages - p.old_pages) + (p.tail == kCopies ? 1u : 0u) : 0u;
  };
  for (int64_t r0 = 0; r0 < end; r0 += kPlanThreads) {
    const int64_t r = r0 + tid;
    RowPlan* p = nullptr;
    if constexpr (ONE) p = &held;
    else if (r < t.R) p = &plans[r];
    const bool is = p != nullptr && r < t.R;
    uint64_t all;
    const uint64_t below = need_all + plan_below(is ? need_of(*p) : 0u, all, sm);
    if (is) p->first = static_cast<int32_t>(below < cap ? below : cap);
    need_all += all;
  }
  // the free pages, from the lowest on
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
  uint32_t found = 0;
  for (int64_t p0 = 0; p0 < t.P && found < need_all; p0 += int64_t{kScanGroups} * kPlanThreads * kScan) {
    uint32_t mask[kScanGroups];
    uint64_t counts = 0;  // of the groups, 16 bits each: a group has kPlanThreads * kScan pages
#pragma unroll
    for (int g = 0; g < kScanGroups; ++g) {
      const int64_t base = p0 + (static_cast<int64_t>(g) * kPlanThreads + tid) * kScan;
      mask[g] = 0;
      if (base + kScan <= t.P) {
        int32_t u[kScan];
        __builtin_memcpy(u, t.uses + base, sizeof(u));
#pragma unroll
        for (int i = 0; i < kScan; ++i) mask[g] |= (u[i] == 0 ? 1u : 0u) << i;
      } else {
        for (int i = 0; i < kScan; ++i)
          if (base + i < t.P && t.uses[base + i] == 0) mask[g] |= 1u << i;
      }
      counts |= static_cast<uint64_t>(__builtin_popcount(mask[g])) << (16 * g);
    }
    uint64_t all;
    const uint64_t below = plan_below(counts, all, sm);
#pragma unroll
    for (int g = 0; g < kScanGroups; ++g) {
      uint32_t at = found + static_cast<uint32_t>(below >> (16 * g) & 0xFFFFu);
      const int64_t base = p0 + (static_cast<int64_t>(g) * kPlanThreads + tid) * kScan;
      for (uint32_t m = mask[g]; m != 0 && at < need_all; m &= m - 1, ++at)
        pool[at] = static_cast<int32_t>(base + __builtin_ctz(m));
      found += static_cast<uint32_t>(all >> (16 * g) & 0xFFFFu);
    }
  }
  __syncthreads();
  const int64_t blocked = sm.blocked;
  if (shared) {
    rows([&](int64_t, RowPlan& p) {
      if (p.tail == kKeeps) store_now(&t.uses[p.page], 0);
    });
    __syncthreads();
  }
  rows([&](int64_t r, RowPlan& p) {
    p.serve = p.new_len > p.old_len && r < blocked && static_cast<uint64_t>(p.first) + need_of(p) <= found ? 1 : 0;
    if (p.tail == kOwn) store_now(&t.uses[p.page], 1);
    else if (p.tail == kKeeps || (p.tail == kCopies && !p.serve)) atomicAdd(&t.uses[p.page], 1);
    if (p.serve && p.tail == kCopies) {
      const int32_t page = pool[p.first++];
      t.tables[r * t.ld + p.old_pages - 1] = page;
      store_now(&t.uses[page], 1);
      copies[atomicAdd(&sm.copies, 1)] = PageCopy{p.page, page, p.old_len % t.S};
    }
    if (p.serve || p.new_len < p.old_len) t.lengths[r] = p.new_len;
  });
  each_page(
      1, [](const RowPlan& p) { return p.serve ? p.new_pages - p.old_pages : 0; },
      [&](int64_t r, const RowPlan& p, int i) {
        const int32_t page = pool[p.first + i];
        t.tables[r * t.ld + p.old_pages + i] = page;
        store_now(&t.uses[page], 1);
      });
  if (tid == 0) out->copies = sm.copies;
}

// ------------------------------------------------------------------- caches ---

constexpr int kMaxCaches = 128;  // of one shape, in one launch

// A cache of pages and slots, cut into columns: the same bytes of every slot.
struct PageShape {
  int64_t page_stride, slot_stride;
  int64_t stride[3];
  Div size1, size2;
  Div run;           // columns of a run
  uint32_t columns;  // of a slot: panels * columns of a run
};
struct PageCaches {
  PageShape shape;
  int count;
  char* data[kMaxCaches];
};

// The byte offset of a slot's column within a page.
template <int W>
__device__ __forceinline__ int64_t column_at(const PageShape& s, uint32_t c) {
  const uint32_t panel = quotient(c, s.run);
  const uint32_t j = c - panel * s.run.d;
  const uint32_t p2 = quotient(panel, s.size2), i2 = panel - p2 * s.size2.d;
  const uint32_t i0 = quotient(p2, s.size1), i1 = p2 - i0 * s.size1.d;
  return i0 * s.stride[0] + i1 * s.stride[1] + i2 * s.stride[2] + static_cast<int64_t>(j) * W;
}

template <int W>
struct Bytes;
template <>
struct Bytes<16> { using type = uint32_t __attribute__((ext_vector_type(4))); };
template <>
struct Bytes<4> { using type = uint32_t; };
template <>
struct Bytes<2> { using type = uint16_t; };
template <>
struct Bytes<1> { using type = uint8_t; };

constexpr int kCopyThreads = 256;

// The copies that the resize has listed: workgroups take (copy, cache) pairs in turn.
// How many there are is not known on the host: 2048 workgroups that find none end
// within 1 us; 16 prompts of 4 beams that grow into shared pages of 32 caches, 17 MB
// moved, take 7 to 10. One workgroup moves all of a page of a cache, so that few large
// caches are slow: the same pages in one tensor of all 32 layers take 40.
template <int W>
__global__ __launch_bounds__(kCopyThreads) void pages_copy_kernel(PageCaches c, const PageCopy* __restrict__ copies,
                                                                  const ResizePlan* __restrict__ plan) {
  using col_t = typename Bytes<W>::type;
  const uint32_t total = static_cast<uint32_t>(plan->copies), count = static_cast<uint32_t>(c.count);
  const uint32_t step = gridDim.x / count, step_cache = gridDim.x - step * count;
  uint32_t k = blockIdx.x / count, cache = blockIdx.x - k * count;
  for (; k < total; k += step, cache += step_cache) {
    if (cache >= count) {
      cache -= count;
      if (++k >= total) break;
    }
    const PageCopy one = copies[k];
    char* data = c.data[cache];
    const char* from = data + one.from * c.shape.page_stride;
    char* to = data + one.to * c.shape.page_stride;
    const uint32_t runs = c.shape.run.d, per = runs * static_cast<uint32_t>(one.slots);
    const uint32_t panels = c.shape.columns / runs;
    // columns of a panel follow each other slot by slot
    for (uint32_t panel = 0; panel < panels; ++panel) {
      const int64_t base = column_at<W>(c.shape, panel * runs);
      for (uint32_t j = threadIdx.x; j < per; j += kCopyThreads) {
        const uint32_t slot = quotient(j, c.shape.run);
        const int64_t off = base + slot * c.shape.slot_stride + static_cast<int64_t>(j - slot * runs) * W;
        *reinterpret_cast<col_t*>(to + off) = *reinterpret_cast<const col_t*>(from + off);
      }
    }
  }
}

constexpr int kCompactThreads = 64;
constexpr int kAhead = 8;  // entries of a column on their way at a time
constexpr int kMaxPath = 255;

// 64 columns of one cache and one sequence. Entries move towards the front, each
// to a place no further than where it lies, so a thread that takes them in order
// overwrites none that it still needs. 64 sequences of 39 drafts in 64 caches of 8
// heads of 128 bf16, 25 MB moved: 8.2 us, 3.1 TB/s; a workgroup's steps hang on one
// another (path, table, entries), and one sequence of 4 caches takes 3.
template <int W>
__global__ __launch_bounds__(kCompactThreads) void pages_compact_kernel(PageCaches c, CompactArgs a, int tiles,
                                                                       int64_t seq0) {
  using col_t = typename Bytes<W>::type;
  __shared__ int32_t from_page[kMaxPath + 1], to_page[kMaxPath + 1];
  __shared__ int32_t from_slot[kMaxPath + 1], to_slot[kMaxPath + 1];
  __shared__ int32_t stop;
  const int tid = threadIdx.x;
  const unsigned tile = blockIdx.x % static_cast<unsigned>(tiles), item = blockIdx.x / static_cast<unsigned>(tiles);
  char* data = c.data[item % static_cast<unsigned>(c.count)];
  const int64_t seq = seq0 + item / static_cast<unsigned>(c.count);
  // all that does not hang on one another at once
  int n = a.counts[seq];
  const int64_t start = a.starts[seq], most = static_cast<int64_t>(a.C) * a.S;
  int32_t at = tid < a.D ? a.path[seq * a.D + tid] : -1, before = tid > 0 && tid < a.D ? a.path[seq * a.D + tid - 1] : -1;
  n = n < a.D ? n : a.D;
  if (n <= 0) return;
  if (tid == 0) stop = n;
  __syncthreads();
  for (int j = tid; j < n; j += kCompactThreads) {
    if (j >= kCompactThreads) {
      at = a.path[seq * a.D + j];
      before = a.path[seq * a.D + j - 1];
    }
    const int64_t from = start + at, to = start + j;
    from_page[j] = to_page[j] = -1;
    if (at <= before || start < 0 || from >= most) {
      atomicMin(&stop, j);  // the path ends where it does not go on
    } else if (at != j) {
      const int fc = static_cast<int>(from / a.S), tc = static_cast<int>(to / a.S);
      const int32_t f = a.tables[seq * a.ld + fc], g = a.tables[seq * a.ld + tc];
      if (f >= 0 && f < a.P && g >= 0 && g < a.P) {
        from_page[j] = f;
        to_page[j] = g;
        from_slot[j] = static_cast<int32_t>(from - static_cast<int64_t>(fc) * a.S);
        to_slot[j] = static_cast<int32_t>(to - static_cast<int64_t>(tc) * a.S);
      }
    }
  }
  __syncthreads();
  n = stop;
  const uint32_t col = tile * kCompactThreads + tid;
  if (col >= c.shape.columns) return;
  data += column_at<W>(c.shape, col);
  for (int j0 = 0; j0 < n; j0 += kAhead) {
    col_t v[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (j0 + i < n && from_page[j0 + i] >= 0)
        v[i] = *reinterpret_cast<const col_t*>(data + from_page[j0 + i] * c.shape.page_stride +
                                               from_slot[j0 + i] * c.shape.slot_stride);
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (j0 + i < n && from_page[j0 + i] >= 0)
        *reinterpret_cast<col_t*>(data + to_page[j0 + i] * c.shape.page_stride +
                                  to_slot[j0 + i] * c.shape.slot_stride) = v[i];
  }
}

int64_t low_bit(int64_t x) { return x & -x; }

// Bytes of a column: what every address is aligned to, at most 16.
int column_bytes(const BeamState& s) {
  int64_t w = 16 | reinterpret_cast<int64_t>(s.data) | s.row_stride | s.run;
  if (s.positions > 1) w |= s.position_stride;
  for (int i = 0; i < 3; ++i)
    if (s.size[i] > 1) w |= s.stride[i];
  w = low_bit(w);
  return w >= 16 ? 16 : (w >= 4 ? 4 : static_cast<int>(w));
}

PageShape shape_of(const BeamState& s, int w) {
  PageShape p{};
  p.page_stride = s.row_stride;
  p.slot_stride = s.position_stride;
  for (int i = 0; i < 3; ++i) p.stride[i] = s.stride[i];
  p.size1 = make_div(static_cast<uint32_t>(s.size[1]));
  p.size2 = make_div(static_cast<uint32_t>(s.size[2]));
  p.run = make_div(static_cast<uint32_t>(s.run / w));
  p.columns = static_cast<uint32_t>(s.size[0] * s.size[1] * s.size[2] * (s.run / w));
  return p;
}

bool same_shape(const BeamState& a, const BeamState& b) {
  bool same = a.row_stride == b.row_stride && a.positions == b.positions && a.position_stride == b.position_stride &&
              a.run == b.run && column_bytes(a) == column_bytes(b);
  for (int i = 0; i < 3; ++i) same = same && a.size[i] == b.size[i] && a.stride[i] == b.stride[i];
  return same;
}

// f(caches, bytes of a column) for runs of caches of one shape, of no more than
// kMaxColumns columns together (or one cache).
constexpr uint64_t kMaxColumns = uint64_t{1} << 31;
template <class F>
hipError_t by_shape(const BeamState* caches, int64_t count, F f) {
  for (int64_t i = 0; i < count;) {
    const int w = column_bytes(caches[i]);
    PageCaches c{};
    c.shape = shape_of(caches[i], w);
    int64_t j = i;
    for (; j < count && c.count < kMaxCaches && same_shape(caches[i], caches[j]) &&
           (c.count == 0 || (static_cast<uint64_t>(c.count) + 1) * c.shape.columns <= kMaxColumns);
         ++j)
      c.data[c.count++] = caches[j].data;
    if (const hipError_t e = f(c, w)) return e;
    i = j;
  }
  return hipSuccess;
}

}  // namespace

bool page_state_fits(const BeamState& s) {
  if (s.run > INT32_MAX || s.positions > INT32_MAX) return false;
  // columns of a page
  uint64_t n = static_cast<uint64_t>(s.run / column_bytes(s));
  for (int64_t f : {s.size[0], s.size[1], s.size[2], s.positions}) {
    n *= static_cast<uint64_t>(f);
    if (n >= (uint64_t{1} << 31) || f >= (int64_t{1} << 31)) return false;
  }
  return true;
}

hipError_t launch_pages_fork(const PageTable& t, const int32_t* parents, int64_t N, int K, hipStream_t stream) {
  // a launch holds at most 2^22 workgroups
  constexpr int64_t kMost = int64_t{1} << 22;
  const int64_t tiles = t.C > 0 ? (static_cast<int64_t>(t.C) + kForkCols - 1) / kForkCols : 1;
  const int64_t step = kMost / tiles > 0 ? kMost / tiles : 1;
  for (int64_t i = 0; i < N; i += step) {
    const int64_t n = N - i < step ? N - i : step;
    if (tiles == 1) {
      hipLaunchKernelGGL((pages_fork_kernel<true>), dim3(static_cast<unsigned>(n)), dim3(kForkThreads), 0, stream, t,
                         parents, K, 1, 0, i);
    } else {
      for (int64_t j = 0; j < tiles; j += kMost) {
        const int64_t of = tiles - j < kMost ? tiles - j : kMost;
        hipLaunchKernelGGL((pages_fork_kernel<false>), dim3(static_cast<unsigned>(n * of)), dim3(kForkThreads), 0, stream,
                           t, parents, K, static_cast<int>(of), static_cast<int>(j), i);
        if (const hipError_t e = hipGetLastError()) return e;
      }
      hipLaunchKernelGGL(pages_fork_lengths_kernel, dim3(static_cast<unsigned>(n)), dim3(kMaxBeams), 0, stream, t,
                         parents, K, i);
    }
    if (const hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

int64_t pages_resize_workspace(int64_t R, int64_t P) {
  return static_cast<int64_t>(sizeof(ResizePlan)) + R * static_cast<int64_t>(sizeof(RowPlan) + sizeof(PageCopy)) +
         (P + 2) * 4;
}

hipError_t launch_pages_resize(const PageTable& t, const int32_t* new_lengths, const BeamState* caches, int64_t count,
                               bool can_copy, void* workspace, hipStream_t stream) {
  ResizePlan* plan = static_cast<ResizePlan*>(workspace);
  RowPlan* rows = reinterpret_cast<RowPlan*>(plan + 1);
  PageCopy* copies = reinterpret_cast<PageCopy*>(rows + t.R);
  int32_t* pool = reinterpret_cast<int32_t*>(copies + t.R);
  if (t.R <= kPlanThreads)
    hipLaunchKernelGGL((pages_resize_kernel<true>), dim3(1), dim3(kPlanThreads), 0, stream, t, new_lengths, can_copy,
                       rows, copies, plan, pool);
  else
    hipLaunchKernelGGL((pages_resize_kernel<false>), dim3(1), dim3(kPlanThreads), 0, stream, t, new_lengths, can_copy,
                       rows, copies, plan, pool);
  if (const hipError_t e = hipGetLastError()) return e;
  return by_shape(caches, count, [&](const PageCaches& c, int w) -> hipError_t {
    const int64_t most = t.R * c.count;
    const dim3 grid(static_cast<unsigned>(most < 2048 ? most : 2048));
    if (w == 16) hipLaunchKernelGGL((pages_copy_kernel<16>), grid, dim3(kCopyThreads), 0, stream, c, copies, plan);
    else if (w == 4) hipLaunchKernelGGL((pages_copy_kernel<4>), grid, dim3(kCopyThreads), 0, stream, c, copies, plan);
    else if (w == 2) hipLaunchKernelGGL((pages_copy_kernel<2>), grid, dim3(kCopyThreads), 0, stream, c, copies, plan);
    else hipLaunchKernelGGL((pages_copy_kernel<1>), grid, dim3(kCopyThreads), 0, stream, c, copies, plan);
    return hipGetLastError();
  });
}

hipError_t launch_pages_compact(const BeamState* caches, int64_t count, const CompactArgs& a, hipStream_t stream) {
  return by_shape(caches, count, [&](const PageCaches& c, int w) -> hipError_t {
    const int64_t tiles = (static_cast<int64_t>(c.shape.columns) + kCompactThreads - 1) / kCompactThreads;
    const int64_t per = tiles * c.count;
    const int64_t step = (int64_t{1} << 25) / per > 0 ? (int64_t{1} << 25) / per : 1;
    for (int64_t i = 0; i < a.N; i += step) {
      const int64_t n = a.N - i < step ? a.N - i : step;
      const dim3 grid(static_cast<unsigned>(n * per)), block(kCompactThreads);
      const int ti = static_cast<int>(tiles);
      if (w == 16) hipLaunchKernelGGL((pages_compact_kernel<16>), grid, block, 0, stream, c, a, ti, i);
      else if (w == 4) hipLaunchKernelGGL((pages_compact_kernel<4>), grid, block, 0, stream, c, a, ti, i);
      else if (w == 2) hipLaunchKernelGGL((pages_compact_kernel<2>), grid, block, 0, stream, c, a, ti, i);
      else hipLaunchKernelGGL((pages_compact_kernel<1>), grid, block, 0, stream, c, a, ti, i);
      if (const hipError_t e = hipGetLastError()) return e;
    }
    return hipSuccess;
  });
}

}  // namespace tkp
