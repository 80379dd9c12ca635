// page_kernel.cu -- the pages of the paged cache: given to sequences, taken
// back, passed on to the children of a beam step, compacted, and copied.
//
// An entry >= 0 of a block table is a reference to a page, and ref_counts[p]
// counts them (and any that the caller holds besides); a page is free where that
// is 0.  Which pages a call gives is a function of its input alone: the lowest
// free ones in order, to the rows in order.  Counts change by integer atomics,
// whose order does not matter.
//
// Giving pages out needs two scans, of the free pages and of the rows' needs,
// that meet: the k-th page needed is the k-th free one.  One cluster of 8 or 16 CTAs
// does both: the rows' needs are scanned by runs of rows, their totals exchanged
// through distributed shared memory; the pool is counted in segments that are dealt
// out to all warps, and the segments' counts and the free pages' numbers go through
// the caller's workspace, with cluster barriers between.  A small pool takes one CTA
// and its own barriers; of a large one the counts and needs are found and the pages
// written by kernels of the whole GPU, the cluster's between.  What touches whole tables (a release, the rows of a fork,
// the new numbers of a compaction) is a kernel with a CTA per row, but for the rows
// of a small fork; it is set up while the plan before it ends.
//
// Bound: latency (dependent passes and barriers) for small pools; the cluster's reads
// of low segments for large ones; HBM for the copies.  Measured (device time, the calls
// replayed): 32 of 512 rows of up to 2048 entries replaced, 690000 pages: free and
// alloc 13.4 us; a fork of 512 rows of 263 entries with its copies 16.5 us; 2100 pages of
// 64 KB moved: plan, tables and copies 57 us, the copies at 6.8 TB/s.  The first
// by the cluster alone 22 us, each CTA of which had a share of consecutive pages and its
// warps a row each 27 us.
#include <cooperative_groups.h>
#include <limits.h>

#include <algorithm>

#include "tv_device.cuh"
#include "tv_launch.h"

namespace cg = cooperative_groups;

namespace tv {
namespace {

constexpr int kNoPage = 7;
constexpr int kPage = 16;
constexpr int kCluster = 16;         // CTAs of a cluster, most
constexpr int kThreads = 1024;       // of a CTA of the cluster
constexpr int kWarps = kThreads / 32;
constexpr int kRowThreads = 256;     // of a CTA of the kernels over tables
constexpr int kAhead = 8;            // entries of a row that a lane has in flight
constexpr int kMaxRows = 65536;      // of a table
constexpr int kNeeds = 8192;         // pieces' needs that a CTA holds
constexpr int kFewEntries = 16384;   // table entries that a CTA writes beside its other work

__device__ __forceinline__ int pages_of(int tokens) { return tokens / kPage + (tokens % kPage > 0); }

// ---------------------------------------------------------------- scans of a cluster
// The C CTAs of a kernel: a cluster, or one.
template <int C>
struct Group {
  __device__ __forceinline__ static int rank() {
    if constexpr (C > 1) return static_cast<int>(cg::this_cluster().block_rank());
    return 0;
  }
  // every thread's writes before are seen after, in all C CTAs
  __device__ __forceinline__ static void sync() {
    if constexpr (C > 1) {
      cg::this_cluster().sync();
    } else {
      __syncthreads();
    }
  }
};
struct Totals {
  int before[2], all[2];  // of two numbers: the sum of the CTAs before this one, and of all
};
struct ScanSmem {
  int warp[2][kWarps];  // of this CTA's warps: exclusive sums of two numbers
  int total[2];         // of this CTA
  Totals sums;
};

__device__ __forceinline__ int warp_sum(int n) { return __reduce_add_sync(0xffffffffu, n); }
__device__ __forceinline__ int warp_before(int n) {  // exclusive sum over the lanes
  const int lane = threadIdx.x & 31;
  int x = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x - n;
}

// Exclusive sums over the CTA's warps of two numbers per warp into s.warp, the CTA's
// totals into s.total.  For all threads.
__device__ void scan_warps(ScanSmem& s, int n, int m) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane < 2) s.warp[lane][warp] = lane ? m : n;
  __syncthreads();
  if (warp < 2) {
    const int v = s.warp[warp][lane], x = warp_before(v);
    s.warp[warp][lane] = x;
    if (lane == 31) s.total[warp] = x + v;
  }
  __syncthreads();
}

// The CTAs' totals, after a barrier of the group.
template <int C>
__device__ Totals group_totals(ScanSmem& s) {
  Totals r;
  if constexpr (C == 1) {
    r.before[0] = r.before[1] = 0;
    r.all[0] = s.total[0];
    r.all[1] = s.total[1];
  } else {
    static_assert(2 * C <= 32, "a lane a number");
    if (threadIdx.x < 32) {
      const int which = threadIdx.x / C, cta = threadIdx.x % C;
      const int x = which < 2 ? *cg::this_cluster().map_shared_rank(&s.total[which], cta) : 0;
      const int low = cta < Group<C>::rank() ? x : 0;
      const int before0 = warp_sum(which == 0 ? low : 0), before1 = warp_sum(which == 1 ? low : 0);
      const int all0 = warp_sum(which == 0 ? x : 0), all1 = warp_sum(which == 1 ? x : 0);
      if (threadIdx.x == 0) s.sums = {{before0, before1}, {all0, all1}};
    }
    __syncthreads();
    r = s.sums;
  }
  return r;
}

// A warp's share of the pages: whole runs of 128 pages, four a lane.
constexpr int kRun = 128;
struct Share {
  int p0, p1;
};
template <int C>
__device__ __forceinline__ Share share_of(int pages, int rank) {
  const int runs = (pages + kRun - 1) / kRun;
  const int warps = C * kWarps, w = rank * kWarps + static_cast<int>(threadIdx.x >> 5);
  const int each = runs / warps, extra = runs % warps;
  Share s;
  s.p0 = (w * each + min(w, extra)) * kRun;
  s.p1 = min(s.p0 + (each + (w < extra)) * kRun, pages);
  s.p0 = min(s.p0, pages);
  return s;
}
// The counts of four pages from p on (past `end`: 1).
__device__ __forceinline__ int4 counts_of(const int32_t* refs, int p, int end) {
  if (p + 4 <= end) return *reinterpret_cast<const int4*>(refs + p);
  int4 r = make_int4(1, 1, 1, 1);
  if (p < end) r.x = refs[p];
  if (p + 1 < end) r.y = refs[p + 1];
  if (p + 2 < end) r.z = refs[p + 2];
  return r;
}
// A lane's pages of the four runs from q on.
struct Runs {
  int4 r[4];
  __device__ __forceinline__ void load(const int32_t* refs, int q, int end) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = counts_of(refs, page(q, i), end);
  }
  __device__ __forceinline__ static int page(int q, int i) { return q + i * kRun + (threadIdx.x & 31) * 4; }
  // a bit for each free page of the i-th four
  __device__ __forceinline__ unsigned free_mask(int i) const {
    return (r[i].x == 0) | (r[i].y == 0) << 1 | (r[i].z == 0) << 2 | (r[i].w == 0) << 3;
  }
  __device__ __forceinline__ int free_pages() const {
    return __popc(free_mask(0) | free_mask(1) << 4 | free_mask(2) << 8 | free_mask(3) << 12);
  }
};

// Free pages of a warp's share (of the pages below `end`).
__device__ int count_free(const int32_t* refs, const Share& sh, int end) {
  const int p1 = min(sh.p1, end);
  int n = 0;
  for (int q = sh.p0; q < p1; q += 8 * kRun) {  // (eight runs on their way)
    Runs x, y;
    x.load(refs, q, p1);
    y.load(refs, q + 4 * kRun, p1);
    n += x.free_pages() + y.free_pages();
  }
  return warp_sum(n);
}

// The pool in at most kSegments segments, whole runs, dealt out to the warps of all
// CTAs in turn: the pages that a call takes, the lowest, are then everybody's work
// (as consecutive shares they were that of the first CTAs: 13000 of 38000 clocks).
constexpr int kSegments = kPageSegments;
struct Segments {
  int pages;  // of a segment
  int count;
};
__device__ __forceinline__ Segments segments_of(int pages) {
  Segments s;
  const int runs = (pages + kRun - 1) / kRun, each = (runs + kSegments - 1) / kSegments;
  s.pages = each * kRun;
  s.count = (runs + each - 1) / each;
  return s;
}
// Free pages of every segment, into counts.
template <int C>
__device__ void count_segments(const PageArgs& a, const Segments& g) {
  constexpr int kAtOnce = 6;  // segments on their way
  const int lane = threadIdx.x & 31, step = C * kWarps;
  for (int i = static_cast<int>(threadIdx.x >> 5) * C + Group<C>::rank(); i < g.count; i += kAtOnce * step) {
    int n[kAtOnce] = {};
    for (int k = lane * 4; k < g.pages; k += kRun) {
      int4 r[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
        r[j] = i + j * step < g.count ? counts_of(a.ref_counts, (i + j * step) * g.pages + k, a.num_blocks) : make_int4(1, 1, 1, 1);
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) n[j] += (r[j].x == 0) + (r[j].y == 0) + (r[j].z == 0) + (r[j].w == 0);
    }
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int all = warp_sum(n[j]);
      if (lane == 0 && i + j * step < g.count) a.counts[i + j * step] = all;
    }
  }
}
// After a barrier of the group: the free pages before each segment into before;
// returns how many there are.
__device__ int scan_segments(const PageArgs& a, const Segments& g, ScanSmem& s, int* before) {
  static_assert(kSegments == 4 * kThreads, "four a thread");
  const int i = static_cast<int>(threadIdx.x) * 4;
  int n[4], sum = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    n[j] = i + j < g.count ? a.counts[i + j] : 0;
    sum += n[j];
  }
  const int lanes = warp_before(sum);
  scan_warps(s, __shfl_sync(0xffffffffu, lanes + sum, 31), 0);
  int at = s.warp[0][threadIdx.x >> 5] + lanes;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    before[i + j] = at;
    at += n[j];
  }
  __syncthreads();
  return s.total[0];
}

// The first `want` free pages of a share, in order, into list; `rank` is that of its
// first free page.
__device__ void list_free(const int32_t* refs, const Share& sh, int rank, int want, int32_t* list) {
  for (int q = sh.p0; q < sh.p1 && rank < want; q += kRun) {
    const int p = q + (threadIdx.x & 31) * 4;
    const int4 r = counts_of(refs, p, sh.p1);
    const int c[4] = {r.x, r.y, r.z, r.w}, n = (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0);
    int at = rank + warp_before(n);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c[j] == 0) {
        if (at < want) list[at] = p + j;
        ++at;
      }
    rank += warp_sum(n);
  }
}

// The first `want` free pages of the pool, in order, into a.list.
template <int C>
__device__ void list_segments(const PageArgs& a, const Segments& g, const int* before, int want) {
  for (int i = static_cast<int>(threadIdx.x >> 5) * C + Group<C>::rank(); i < g.count && before[i] < want; i += C * kWarps)
    list_free(a.ref_counts, {i * g.pages, min((i + 1) * g.pages, a.num_blocks)}, before[i], want, a.list);
}

// ---------------------------------------------------------------- alloc
struct Range {
  int t0, t1, code;  // entries of a row that have to name pages
};
__device__ __forceinline__ Range range_of(const PageArgs& a, int b) {
  const int begin = a.begin ? a.begin[b] : 0, end = a.end[b];
  Range r;
  r.code = begin < 0 || end < 0 || end > static_cast<long long>(a.width) * kPage ? kBadTree : kOk;
  r.t0 = r.code == kOk ? begin / kPage : 0;
  r.t1 = r.code == kOk ? pages_of(end) : 0;
  return r;
}

// How many of a row's entries [q0, q1) lack a page (-1: one names nothing), by a warp.
__device__ int piece_needs(const PageArgs& a, const int32_t* row, int q0, int q1) {
  const int lane = threadIdx.x & 31;
  int lack = 0;
  bool bad = false;
  for (int t = q0 + lane; t < q1; t += 32 * kAhead) {
    int e[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) e[j] = t + j * 32 < q1 ? row[t + j * 32] : 0;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      lack += e[j] < 0;
      bad |= e[j] >= a.num_blocks;
    }
  }
  lack = warp_sum(lack);
  return __any_sync(0xffffffffu, bad) ? -1 : lack;
}
// Which of a lane's entries from q on lack one, a bit each.
__device__ __forceinline__ unsigned lacking(const int32_t* row, int q, int q1) {
  unsigned r = 0;
#pragma unroll
  for (int j = 0; j < kAhead; ++j) {
    const int t = q + j * 32 + static_cast<int>(threadIdx.x & 31);
    r |= static_cast<unsigned>(t < q1 && row[t] < 0) << j;
  }
  return r;
}
// Gives those of [q0, q1) the list's pages from `from` on; `lacks` is lacking(row, q0, q1).
__device__ __forceinline__ void fill_piece(const PageArgs& a, int32_t* row, int q0, int q1, int from, unsigned lacks) {
  const int lane = threadIdx.x & 31;
  for (int q = q0; q < q1; q += 32 * kAhead) {
    if (q > q0) lacks = lacking(row, q, q1);
    int at_list[kAhead], page[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const unsigned m = __ballot_sync(0xffffffffu, lacks >> j & 1u);
      at_list[j] = from + __popc(m & ((1u << lane) - 1));
      from += __popc(m);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) page[j] = lacks >> j & 1u ? a.list[at_list[j]] : 0;
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (lacks >> j & 1u) {
        row[q + j * 32 + lane] = page[j];
        a.ref_counts[page[j]] = 1;
      }
  }
}

// A row is cut into a.cuts pieces of a.piece entries from its range's first on, a
// warp a piece.  Dynamic shared memory: the pieces' needs (-1: an entry that names
// nothing), the rows' places in the list (-1: refused, -2: without a page) and ranges.
template <int C, bool SPLIT>
__global__ void __launch_bounds__(kThreads) alloc_kernel(const PageArgs a) {
  extern __shared__ int need[];
  __shared__ ScanSmem s, of_segments;
  __shared__ int free_before[kSegments];
  const int rank = Group<C>::rank(), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Segments g = segments_of(a.num_blocks);
  const int each = (a.rows + C - 1) / C;
  const int b0 = min(rank * each, a.rows), n = min(each, a.rows - b0), pieces = n * a.cuts;
  int* place = need + each * a.cuts;
  int* first = place + each;
  int* last = first + each;
  if constexpr (SPLIT) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int i = threadIdx.x; i < pieces; i += kThreads) need[i] = a.needs[b0 * a.cuts + i];
  } else {
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const Range r = range_of(a, b0 + i);
      first[i] = r.code == kOk ? r.t0 : -1;
      last[i] = r.t1;
    }
    count_segments<C>(a, g);
    __syncthreads();
    // how many entries of each piece lack a page
    for (int i = warp; i < pieces; i += kWarps) {
      const int b = i / a.cuts, q0 = first[b] + (i - b * a.cuts) * a.piece, q1 = min(q0 + a.piece, last[b]);
      const int lack = first[b] < 0 ? -1 : piece_needs(a, a.block_table + static_cast<size_t>(b0 + b) * a.width, q0, q1);
      if (lane == 0) need[i] = lack;
    }
  }
  __syncthreads();
  // exclusive sums of the rows' needs: a run of rows per thread
  const int run = (n + kThreads - 1) / kThreads, i0 = min(static_cast<int>(threadIdx.x) * run, n), i1 = min(i0 + run, n);
  int sum = 0;
  for (int i = i0; i < i1; ++i) {
    int lack = 0;
    bool bad = false;
    for (int k = 0; k < a.cuts; ++k) {
      const int x = need[i * a.cuts + k];
      bad |= x < 0;
      lack += x;
    }
    place[i] = bad ? -1 : lack;
    sum += bad ? 0 : lack;
  }
  const int before = warp_before(sum);
  scan_warps(s, 0, warp_sum(sum));
  Group<C>::sync();
  const Totals needs = group_totals<C>(s);
  const int wanted = needs.all[1], own = needs.before[1] + s.warp[1][warp] + before;
  int frees = 0;
  if (wanted > 0) {  // (a decode step mostly finds nothing lacking)
    frees = scan_segments(a, g, of_segments, free_before);
    list_segments<C>(a, g, free_before, min(wanted, frees));
  }
  int at = own;
  for (int i = i0; i < i1; ++i) {
    const int lack = place[i];
    place[i] = lack < 0 ? -1 : lack > 0 && lack > frees - at ? -2 : at;
    at += max(lack, 0);
  }
  Group<C>::sync();  // the list is written, and no CTA reads another's shared memory any more
  for (int i = threadIdx.x; i < n; i += kThreads) {
    a.status[b0 + i] = place[i] == -1 ? kBadTree : place[i] == -2 ? kNoPage : kOk;
    if (SPLIT) a.first[b0 + i] = place[i];
  }
  if (SPLIT || wanted == 0) return;
  for (int i = warp; i < pieces; i += kWarps) {
    const int k = i % a.cuts, b = b0 + i / a.cuts;
    int from = place[i / a.cuts];
    if (from < 0 || need[i] == 0) continue;
    for (int j = 0; j < k; ++j) from += need[i - k + j];
    const int q0 = first[i / a.cuts] + k * a.piece, q1 = min(q0 + a.piece, last[i / a.cuts]);
    int32_t* row = a.block_table + static_cast<size_t>(b) * a.width;
    fill_piece(a, row, q0, q1, from, lacking(row, q0, q1));
  }
}

// The same of a large pool in three kernels, the second and third set up while the one
// before ends.  First, all over the GPU, a warp for each segment's free pages and each
// piece's needs (8.6 of the cluster's 19 us at 690000 pages and 512 rows); then the plan
// by the cluster (alloc_kernel with SPLIT); and again a warp a piece (its 5 us).
__global__ void __launch_bounds__(kRowThreads) survey_kernel(const PageArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, w = static_cast<int>(blockIdx.x) * (kRowThreads / 32) + static_cast<int>(threadIdx.x >> 5);
  const Segments g = segments_of(a.num_blocks);
  if (w < g.count) {
    const int end = min((w + 1) * g.pages, a.num_blocks);
    int n = 0;
    for (int q = w * g.pages; q < end; q += 4 * kRun) {
      Runs x;
      x.load(a.ref_counts, q, end);
      n += x.free_pages();
    }
    n = warp_sum(n);
    if (lane == 0) a.counts[w] = n;
  } else if (w - g.count < a.rows * a.cuts) {
    const int i = w - g.count, b = i / a.cuts;
    const Range r = range_of(a, b);
    const int q0 = r.t0 + (i - b * a.cuts) * a.piece;
    const int lack = r.code != kOk ? -1 : piece_needs(a, a.block_table + static_cast<size_t>(b) * a.width, q0, min(q0 + a.piece, r.t1));
    if (lane == 0) a.needs[i] = lack;
  }
}
__global__ void __launch_bounds__(kRowThreads) fill_kernel(const PageArgs a) {
  const int lane = threadIdx.x & 31, i = static_cast<int>(blockIdx.x) * (kRowThreads / 32) + static_cast<int>(threadIdx.x >> 5);
  const bool here = i < a.rows * a.cuts;
  const int b = here ? i / a.cuts : 0, k = here ? i - b * a.cuts : 0;
  // (what the kernels before do not write)
  const Range r = range_of(a, b);
  const int q0 = r.t0 + k * a.piece, q1 = min(q0 + a.piece, r.t1);
  int32_t* row = a.block_table + static_cast<size_t>(b) * a.width;
  const unsigned lacks = r.code == kOk ? lacking(row, q0, q1) : 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!here) return;
  const int place = a.first[b], need = lane <= k ? a.needs[i - k + lane] : 0;
  if (place < 0 || __shfl_sync(0xffffffffu, need, k) == 0) return;
  fill_piece(a, row, q0, q1, place + warp_sum(lane < k ? need : 0), lacks);
}

// ---------------------------------------------------------------- free
__global__ void __launch_bounds__(kRowThreads) free_kernel(const PageArgs a) {
  const int b = blockIdx.x;
  const int begin = a.keep_begin ? a.keep_begin[b] : 0, end = a.keep_end ? a.keep_end[b] : INT_MAX;
  bool bad = begin < 0 || end < 0;
  if (!bad) {
    // entries below `low` but for the first tokens', and from `high` on
    const int low = begin / kPage, high = pages_of(end), first = pages_of(a.sinks);
    int32_t* row = a.block_table + static_cast<size_t>(b) * a.width;
    for (int t0 = threadIdx.x; t0 < a.width; t0 += kRowThreads * kAhead) {
      int e[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int t = t0 + j * kRowThreads;
        e[j] = t < a.width && ((t < low && t >= first) || t >= high) ? row[t] : -1;
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (e[j] < 0) continue;
        row[t0 + j * kRowThreads] = -1;
        if (e[j] < a.num_blocks) {
          atomicSub(a.ref_counts + e[j], 1);
        } else {
          bad = true;
        }
      }
    }
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) a.status[b] = bad ? kBadTree : kOk;
}

// ---------------------------------------------------------------- fork
struct Child {
  int parent, len, code;
};
__device__ __forceinline__ Child child_of(const PageArgs& a, int i) {
  Child c;
  c.parent = a.parents[i];
  c.len = 0;
  c.code = c.parent < -1 || c.parent >= a.rows ? kBadTree : kOk;
  if (c.code == kOk && c.parent >= 0) {
    c.len = a.seq_lens[c.parent];
    if (c.len < 0 || c.len > static_cast<long long>(a.width) * kPage) c.code = kBadTree;
  }
  return c;
}

// New row i of a fork, and what becomes of old row i, by the threads from `first`
// on in steps of `step`.  Returns whether an entry that a child continues names
// nothing.
__device__ bool fork_row(const PageArgs& a, int i, int first, int step) {
  bool bad = false;
  if (i < a.new_rows) {
    const int code = a.status[i], p = a.parents[i];
    int32_t* out = a.table_out + static_cast<size_t>(i) * a.width;
    if (code != kOk || p < 0) {
      for (int t = first; t < a.width; t += step) out[t] = -1;
    } else {
      const bool takes = a.first[p] == i;
      const int len = a.seq_lens[p], whole = len / kPage, part = len % kPage > 0;
      const int src = a.copies[3 * static_cast<size_t>(i)], dst = a.copies[3 * static_cast<size_t>(i) + 1];
      const int32_t* in = a.block_table + static_cast<size_t>(p) * a.width;
      for (int t0 = first; t0 < a.width; t0 += step * kAhead) {
        int entry[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) entry[j] = t0 + j * step < a.width ? in[t0 + j * step] : -1;
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const int t = t0 + j * step;
          if (t >= a.width) break;
          int e = entry[j];
          if (t >= whole + part && !takes) e = -1;  // the first child has the spare ones
          if (e >= a.num_blocks) bad = true, e = -1;
          if (t == whole && part && dst >= 0) {
            if (takes) atomicSub(a.ref_counts + src, 1);
            e = dst;
          } else if (e >= 0 && !takes) {
            atomicAdd(a.ref_counts + e, 1);
          }
          out[t] = max(e, -1);
        }
      }
    }
  }
  // nobody takes over the references of a row without a (first) child
  if (i < a.rows && a.first[i] == INT_MAX) {
    const int32_t* in = a.block_table + static_cast<size_t>(i) * a.width;
    for (int t0 = first; t0 < a.width; t0 += step * kAhead) {
      int entry[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) entry[j] = t0 + j * step < a.width ? in[t0 + j * step] : -1;
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (entry[j] >= 0 && entry[j] < a.num_blocks) atomicSub(a.ref_counts + entry[j], 1);
    }
  }
  return bad;
}

// Who takes over a parent's last page, and the pages and copies of the others;
// with ROWS the rows too.
template <int C, bool ROWS>
__global__ void __launch_bounds__(kThreads) fork_plan_kernel(const PageArgs a) {
  __shared__ ScanSmem s, of_segments;
  __shared__ int free_before[kSegments];
  const int rank = Group<C>::rank(), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int i = rank * kThreads + threadIdx.x; i < a.rows; i += C * kThreads) a.first[i] = INT_MAX;
  const Segments g = segments_of(a.num_blocks);
  count_segments<C>(a, g);
  Group<C>::sync();
  for (int i = rank * kThreads + threadIdx.x; i < a.new_rows; i += C * kThreads) {
    const Child c = child_of(a, i);
    if (c.code == kOk && c.parent >= 0) atomicMin(a.first + c.parent, i);
  }
  Group<C>::sync();
  // a run of children per thread: how many of them need a page
  const int each = (a.new_rows + C - 1) / C;
  const int b0 = min(rank * each, a.new_rows), n = min(each, a.new_rows - b0);
  const int run = (n + kThreads - 1) / kThreads, i0 = min(static_cast<int>(threadIdx.x) * run, n), i1 = min(i0 + run, n);
  // the page that a child has to copy, -1: none, -2: it should have one but there is none
  const auto source = [&](int i, const Child& c) {
    if (c.code != kOk || c.len % kPage == 0) return -1;
    const int e = a.block_table[static_cast<size_t>(c.parent) * a.width + c.len / kPage];
    if (e < 0 || e >= a.num_blocks) return -2;
    const int refs = a.ref_counts[e];
    if (refs < 1) return -2;
    return a.first[c.parent] != i || refs > 1 ? e : -1;
  };
  int sum = 0;
  for (int i = i0; i < i1; ++i) {
    const int src = source(b0 + i, child_of(a, b0 + i));
    a.copies[3 * static_cast<size_t>(b0 + i)] = src;  // (decided once: counts change below)
    sum += src >= 0;
  }
  const int before = warp_before(sum);
  scan_warps(s, 0, warp_sum(sum));
  Group<C>::sync();
  const Totals needs = group_totals<C>(s);
  int at = needs.before[1] + s.warp[1][warp] + before, frees = 0;
  if (needs.all[1] > 0) {
    frees = scan_segments(a, g, of_segments, free_before);
    list_segments<C>(a, g, free_before, min(needs.all[1], frees));
  }
  Group<C>::sync();  // the list is written, and no CTA reads another's shared memory any more
  for (int i = i0; i < i1; ++i) {
    const int b = b0 + i;
    const Child c = child_of(a, b);
    int32_t* copy = a.copies + 3 * static_cast<size_t>(b);
    const int src = copy[0];
    int code = src == -2 ? kBadTree : c.code, dst = -1;
    if (src >= 0) {
      if (at < frees) {
        dst = a.list[at];
        a.ref_counts[dst] = 1;
      } else {
        code = kNoPage;
      }
      ++at;
    }
    // a first child without its page takes nothing over
    if (code != kOk && c.code == kOk && c.parent >= 0 && a.first[c.parent] == b) a.first[c.parent] = INT_MAX;
    a.status[b] = code;
    a.lens_out[b] = code == kOk ? c.len : 0;
    copy[0] = dst >= 0 ? src : -1;
    copy[1] = dst;
    copy[2] = dst >= 0 ? c.len % kPage : 0;
  }
  if (!ROWS) return;
  Group<C>::sync();
  for (int i = rank * kWarps + warp; i < max(a.rows, a.new_rows); i += C * kWarps) {
    const bool bad = fork_row(a, i, lane, 32);
    if (__any_sync(0xffffffffu, bad) && lane == 0) a.status[i] = kBadTree;
  }
}

__global__ void __launch_bounds__(kRowThreads) fork_rows_kernel(const PageArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const bool bad = fork_row(a, blockIdx.x, threadIdx.x, kRowThreads);
  if (__syncthreads_or(bad) && threadIdx.x == 0) a.status[blockIdx.x] = kBadTree;
}

// ---------------------------------------------------------------- compact
template <int C>
__global__ void __launch_bounds__(kThreads) compact_plan_kernel(const PageArgs a) {
  __shared__ ScanSmem s;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int rank = Group<C>::rank(), warp = threadIdx.x >> 5;
  const Share sh = share_of<C>(a.num_blocks, rank);
  const int mine = count_free(a.ref_counts, sh, a.num_blocks);
  scan_warps(s, mine, 0);
  Group<C>::sync();
  const Totals free_pages = group_totals<C>(s);
  const int live = a.num_blocks - free_pages.all[0], first = free_pages.before[0] + s.warp[0][warp];
  // the holes: free pages below `live`, as many as pages in use from there on
  scan_warps(s, mine, count_free(a.ref_counts, sh, live));  // (another CTA may read the first total still: it stays)
  Group<C>::sync();
  const int holes = group_totals<C>(s).all[1];
  int frees = first;
  for (int q = sh.p0; q < sh.p1; q += kRun) {
    const int p = q + static_cast<int>(threadIdx.x & 31) * 4;
    const int4 r = counts_of(a.ref_counts, p, sh.p1);
    const int c[4] = {r.x, r.y, r.z, r.w}, n = (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0);
    int f = frees + warp_before(n);  // free pages before this one
    int to[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int page = p + j;
      const bool is_free = c[j] == 0;
      // (a page in use from `live` on gets its number below, past a barrier)
      to[j] = !is_free && page < live ? page : -1;
      if (is_free && page < live) {
        a.copies[3 * static_cast<size_t>(f) + 1] = page;
        a.copies[3 * static_cast<size_t>(f) + 2] = kPage;
      } else if (!is_free && page >= live && page < sh.p1) {
        a.copies[3 * static_cast<size_t>(page - live - (f - holes))] = page;
      }
      f += is_free;
    }
    if (p + 4 <= sh.p1) {
      *reinterpret_cast<int4*>(a.page_map + p) = make_int4(to[0], to[1], to[2], to[3]);
      *reinterpret_cast<int4*>(a.refs_out + p) = r;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (p + j < sh.p1) a.page_map[p + j] = to[j], a.refs_out[p + j] = c[j];
    }
    frees += warp_sum(n);
  }
  if (rank == 0 && threadIdx.x == 0) {
    a.count[0] = live;
    a.count[1] = holes;
  }
  Group<C>::sync();
  for (int i = rank * kThreads + threadIdx.x; i < holes; i += C * kThreads) {
    const int src = a.copies[3 * static_cast<size_t>(i)], dst = a.copies[3 * static_cast<size_t>(i) + 1];
    a.page_map[src] = dst;
    a.refs_out[dst] = a.ref_counts[src];
    a.refs_out[src] = 0;
  }
}

__global__ void __launch_bounds__(kRowThreads) renumber_kernel(const PageArgs a) {
  const int b = blockIdx.x;
  const int32_t* in = a.block_table + static_cast<size_t>(b) * a.width;
  int32_t* out = a.table_out + static_cast<size_t>(b) * a.width;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  bool bad = false;
  for (int t0 = threadIdx.x; t0 < a.width; t0 += kRowThreads * kAhead) {
    int e[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) e[j] = t0 + j * kRowThreads < a.width ? in[t0 + j * kRowThreads] : -1;
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (e[j] >= 0) {
        e[j] = e[j] < a.num_blocks ? a.page_map[e[j]] : -1;
        bad |= e[j] < 0;
      }
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (t0 + j * kRowThreads < a.width) out[t0 + j * kRowThreads] = max(e[j], -1);
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) a.status[b] = bad ? kBadTree : kOk;
}

// ---------------------------------------------------------------- copies
constexpr int kCopyThreads = 256;
constexpr int kInFlight = 8;  // 16-byte words of a thread

// A CTA takes a slice of the K or V page of an entry in a layer.
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const CopyArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int entries = a.count ? max(0, min(a.count[0], a.entries)) : a.entries;
  const int per = 2 * a.layers * a.slices;  // of an entry
  const long long all = static_cast<long long>(entries) * per;
  const int heads = a.hkv, row_words = a.row_bytes / 16, shift = 31 - __clz(row_words);
  const int words = heads * kPage * row_words, slice_words = (words + a.slices - 1) / a.slices;
  for (long long w = blockIdx.x; w < all; w += gridDim.x) {
    const int i = static_cast<int>(w / per), which = static_cast<int>(w - static_cast<long long>(i) * per);
    const int slice = which % a.slices, kv = which / a.slices & 1, layer = which / a.slices >> 1;
    const int src = a.copies[3 * static_cast<size_t>(i)], dst = a.copies[3 * static_cast<size_t>(i) + 1];
    const int tokens = a.copies[3 * static_cast<size_t>(i) + 2];
    const bool none = src < 0 && dst < 0;
    const bool good = src >= 0 && dst >= 0 && src < a.num_blocks && dst < a.num_blocks && tokens >= 0 && tokens <= kPage;
    if (a.status && which == 0 && threadIdx.x == 0) a.status[i] = none || good ? kOk : kNoPage;
    if (!good || src == dst) continue;
    uint8_t* pool = static_cast<uint8_t*>(kv ? a.pool[1] : a.pool[0]) + layer * a.layer_stride;
    const uint4* from = reinterpret_cast<const uint4*>(pool) + static_cast<size_t>(src) * words;
    uint4* to = reinterpret_cast<uint4*>(pool) + static_cast<size_t>(dst) * words;
    const int j0 = slice * slice_words, j1 = min(j0 + slice_words, words);
    for (int q = j0 + threadIdx.x; q < j1; q += kCopyThreads * kInFlight) {
      uint4 x[kInFlight];
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        const int j = q + u * kCopyThreads;
        if (j < j1 && (j >> shift) % kPage < tokens) x[u] = from[j];
      }
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        const int j = q + u * kCopyThreads;
        if (j < j1 && (j >> shift) % kPage < tokens) to[j] = x[u];
      }
    }
    if (a.scale[0] && slice == 0) {
      float* scales = (kv ? a.scale[1] : a.scale[0]) + layer * a.scale_stride;
      const float* sf = scales + static_cast<size_t>(src) * heads * kPage;
      float* st = scales + static_cast<size_t>(dst) * heads * kPage;
      for (int j = threadIdx.x; j < heads * kPage; j += kCopyThreads)
        if (j % kPage < tokens) st[j] = sf[j];
    }
  }
}

int launched() { return cudaGetLastError() == cudaSuccess ? 0 : -1; }

// A kernel of C CTAs of a cluster; `behind`: as launch_behind's.
template <int C>
int launch_group(void (*kernel)(PageArgs), const PageArgs& a, size_t smem, cudaStream_t stream, bool behind = false) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(C);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = C == 1 ? 0 : behind ? 2 : 1;
  if (C > 8 && cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) return -1;
  return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? 0 : -1;
}

// A kernel that may be set up while the one before it in the stream ends, for
// whose results it waits.
template <typename Args>
int launch_behind(void (*kernel)(Args), const Args& a, unsigned grid, unsigned threads, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? 0 : -1;
}

// How many CTAs: one for a pool of at most `most` pages (it spares the cluster
// barriers), 8 below 2^17 pages, then 16.  Device times with 1, 8 and 16 CTAs, us:
// free and alloc, 3550 pages 8.2, 9.3, 10.3; 9900 11.3, 10.2, 10.3; 141000 -, 15.4,
// 13.3 (now in three kernels, 11.3); 690000 -, 32.8, 22.6 (13.4).  Compaction and copies, 1600 pages 11.3, 13.3, 13.4; 8780
// 57.1, 57.1, 57.4; 13800 27.7, 25.6, 25.7 (smaller pages); 198000 -, 224, 218.  Fork and
// copies (its children do not divide as well), 1360 pages 12.1, 15.4, 16.4;
// 17400 16.5, 17.9, 20.9; 25900 17.7, 17.5, 24.4.
int ctas_for(const PageArgs& a, int most) {
  if (a.num_blocks <= most && a.rows <= kThreads && a.new_rows <= kThreads) return 1;
  return a.num_blocks < kManyPages ? 8 : kCluster;
}

}  // namespace

int launch_alloc_pages(PageArgs a, cudaStream_t stream) {
  const int ctas = ctas_for(a, 6144), each = (a.rows + ctas - 1) / ctas;
  // pieces of a row: of 256 entries (what a warp has in flight) at least, as many as a
  // CTA has room for
  int cuts = (a.width + 255) / 256;
  cuts = cuts < kMaxCuts ? cuts : kMaxCuts;
  a.cuts = cuts < kNeeds / each ? cuts : (kNeeds / each > 1 ? kNeeds / each : 1);
  a.piece = (a.width + a.cuts - 1) / a.cuts;
  const size_t smem = static_cast<size_t>(each) * (a.cuts + 3) * 4;  // (65536 rows are 8192 for each of 8 CTAs: 128 KB)
  const auto kernel = ctas == 1 ? alloc_kernel<1, false> : ctas == 8 ? alloc_kernel<8, false> : alloc_kernel<kCluster, true>;
  // (the kernel's limit is all host threads': always that of the most rows)
  const int most = ctas == 1 ? kThreads : kMaxRows / ctas, limit = (std::max(kNeeds, most) + 3 * most) * 4;
  if (smem > 24 * 1024 && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, limit) != cudaSuccess)
    return -1;
  if (ctas <= 8) return ctas == 1 ? launch_group<1>(kernel, a, smem, stream) : launch_group<8>(kernel, a, smem, stream);
  const int warps = kRowThreads / 32, pieces = a.rows * a.cuts;
  survey_kernel<<<static_cast<unsigned>((kSegments + pieces + warps - 1) / warps), kRowThreads, 0, stream>>>(a);
  if (launched() || launch_group<kCluster>(kernel, a, smem, stream, true)) return -1;
  return launch_behind(fill_kernel, a, static_cast<unsigned>((pieces + warps - 1) / warps), kRowThreads, stream);
}

int launch_free_pages(const PageArgs& a, cudaStream_t stream) {
  free_kernel<<<a.rows, kRowThreads, 0, stream>>>(a);
  return launched();
}

namespace {

template <bool ROWS>
int launch_fork_plan(const PageArgs& a, int ctas, cudaStream_t stream) {
  return ctas == 1   ? launch_group<1>(fork_plan_kernel<1, ROWS>, a, 0, stream)
         : ctas == 8 ? launch_group<8>(fork_plan_kernel<8, ROWS>, a, 0, stream)
                     : launch_group<kCluster>(fork_plan_kernel<kCluster, ROWS>, a, 0, stream);
}

}  // namespace

int launch_fork_pages(const PageArgs& a, cudaStream_t stream) {
  const int rows = a.rows > a.new_rows ? a.rows : a.new_rows, ctas = ctas_for(a, 24576);
  // few entries are done by the same CTAs: 32 rows of 253 entries take 0.8 us more on
  // the device (12.1, with copies), but the host spends 2 us less on a call (18.3)
  if (static_cast<long long>(rows) * a.width <= static_cast<long long>(ctas) * kFewEntries)
    return launch_fork_plan<true>(a, ctas, stream);
  if (launch_fork_plan<false>(a, ctas, stream)) return -1;
  return launch_behind(fork_rows_kernel, a, static_cast<unsigned>(rows), kRowThreads, stream);
}

int launch_compact_pages(const PageArgs& a, cudaStream_t stream) {
  const int ctas = ctas_for(a, 6144);
  if (ctas == 1   ? launch_group<1>(compact_plan_kernel<1>, a, 0, stream)
      : ctas == 8 ? launch_group<8>(compact_plan_kernel<8>, a, 0, stream)
                  : launch_group<kCluster>(compact_plan_kernel<kCluster>, a, 0, stream))
    return -1;
  return launch_behind(renumber_kernel, a, static_cast<unsigned>(a.rows), kRowThreads, stream);
}

int launch_copy_pages(CopyArgs a, int sms, cudaStream_t stream) {
  // few entries: several CTAs a page, so that every SM has four
  const long long pages = 2ll * a.entries * a.layers, want = 4ll * sms / pages;
  a.slices = static_cast<int>(want < 1 ? 1 : want < 8 ? want : 8);
  const long long all = pages * a.slices, most = 8ll * sms;
  return launch_behind(copy_kernel, a, static_cast<unsigned>(all < most ? all : most), kCopyThreads, stream);
}

}  // namespace tv
