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
// does both: every CTA counts a slice of the pages and of the rows, the totals go
// through distributed shared memory, the free pages' numbers through the caller's
// workspace, with a cluster barrier between; one launch, and the slices are
// read from the same L2.  A small pool takes one CTA and its own barriers.  What
// touches whole tables (a release, the rows of a fork, the new numbers of a
// compaction) is a kernel with a CTA per row, but for the rows of a small fork.
//
// Bound: latency (three dependent passes and two cluster barriers) for small
// pools; the cluster's reads of the counts for large ones; HBM for the copies.
#include <cooperative_groups.h>
#include <limits.h>

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
struct ScanSmem {
  int warp[2][kWarps];     // of this CTA's warps: exclusive sums
  int total[2];            // of this CTA
  int mine[2][kCluster];   // the CTAs' totals
  int more;
};

// Exclusive sums over the CTA's warps of a number per warp (lane 0's), into
// s.warp[which], the CTA's total into s.total[which].  For all threads.
__device__ void scan_warps(ScanSmem& s, int which, int n) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) s.warp[which][warp] = n;
  __syncthreads();
  if (warp == 0) {
    const int v = s.warp[which][lane];
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    s.warp[which][lane] = x - v;
    if (lane == 31) s.total[which] = x;
  }
  __syncthreads();
}

// The CTAs' totals, after a barrier of the group: (those of the CTAs before this one, all).
template <int C>
__device__ int2 group_totals(ScanSmem& s, int which) {
  if constexpr (C == 1) return make_int2(0, s.total[which]);
  if (threadIdx.x < C) s.mine[which][threadIdx.x] = *cg::this_cluster().map_shared_rank(&s.total[which], threadIdx.x);
  __syncthreads();
  int before = 0, all = 0;
  for (int i = 0; i < C; ++i) {
    if (i < Group<C>::rank()) before += s.mine[which][i];
    all += s.mine[which][i];
  }
  return make_int2(before, all);
}

// A warp's share of the pages: whole runs of 128 pages.
struct Share {
  int p0, p1;
};
template <int C>
__device__ __forceinline__ Share share_of(int pages, int rank) {
  const int runs = (pages + 127) / 128;
  const int warps = C * kWarps, w = rank * kWarps + static_cast<int>(threadIdx.x >> 5);
  const int each = runs / warps, extra = runs % warps;
  Share s;
  s.p0 = (w * each + min(w, extra)) * 128;
  s.p1 = min(s.p0 + (each + (w < extra)) * 128, pages);
  s.p0 = min(s.p0, pages);
  return s;
}
// The counts of a lane's four pages from p on (past `end`: `fill`).
__device__ __forceinline__ int4 counts_of(const int32_t* refs, int p, int end, int fill) {
  if (p + 4 <= end) return *reinterpret_cast<const int4*>(refs + p);
  int4 r = make_int4(fill, fill, fill, fill);
  if (p < end) r.x = refs[p];
  if (p + 1 < end) r.y = refs[p + 1];
  if (p + 2 < end) r.z = refs[p + 2];
  return r;
}
__device__ __forceinline__ int free_mask(int4 r) {
  return (r.x == 0) | (r.y == 0) << 1 | (r.z == 0) << 2 | (r.w == 0) << 3;
}
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

// Free pages of a warp's share (of the pages below `end`).
__device__ int count_free(const int32_t* refs, const Share& sh, int end) {
  const int lane = threadIdx.x & 31;
  int n = 0;
#pragma unroll 4
  for (int p = sh.p0 + lane * 4; p < min(sh.p1, end); p += 128)
    n += __popc(free_mask(counts_of(refs, p, min(sh.p1, end), 1)));
  return warp_sum(n);
}

// The first `want` free pages of the pool, in order, into list; `rank` is that of
// the warp's first free page.
__device__ void list_free(const int32_t* refs, const Share& sh, int rank, int want, int32_t* list) {
  const int lane = threadIdx.x & 31;
  for (int q0 = sh.p0; q0 < sh.p1 && rank < want; q0 += 4 * 128) {
    int m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = free_mask(counts_of(refs, q0 + i * 128 + lane * 4, sh.p1, 1));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int p = q0 + i * 128 + lane * 4, n = __popc(m[i]);
      int at = rank + warp_before(n);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (m[i] >> j & 1) {
          if (at < want) list[at] = p + j;
          ++at;
        }
      rank += warp_sum(n);
    }
  }
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

// (dynamic shared memory: the needs of the CTA's rows, then their exclusive sums;
// -1: a row that is refused)
template <int C>
__global__ void __launch_bounds__(kThreads) alloc_kernel(const PageArgs a) {
  extern __shared__ int need[];
  __shared__ ScanSmem s;
  const int rank = Group<C>::rank(), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Share sh = share_of<C>(a.num_blocks, rank);
  const int mine = count_free(a.ref_counts, sh, a.num_blocks);
  const int each = (a.rows + C - 1) / C;
  const int b0 = min(rank * each, a.rows), n = min(each, a.rows - b0);
  // how many entries of each row lack a page
  for (int i = warp; i < n; i += kWarps) {
    const Range r = range_of(a, b0 + i);
    const int32_t* row = a.block_table + static_cast<size_t>(b0 + i) * a.width;
    int lack = 0;
    bool bad = r.code != kOk;
#pragma unroll 8
    for (int t = r.t0 + lane; t < r.t1; t += 32) {
      const int e = row[t];
      lack += e < 0;
      bad |= e >= a.num_blocks;
    }
    lack = warp_sum(lack);
    if (__any_sync(0xffffffffu, bad)) lack = -1;
    if (lane == 0) need[i] = lack;
  }
  scan_warps(s, 0, mine);
  // exclusive sums of the rows' needs: a run of rows per thread
  const int run = (n + kThreads - 1) / kThreads, i0 = min(static_cast<int>(threadIdx.x) * run, n), i1 = min(i0 + run, n);
  int sum = 0;
  for (int i = i0; i < i1; ++i) sum += max(need[i], 0);
  const int before = warp_before(sum);
  scan_warps(s, 1, __shfl_sync(0xffffffffu, before + sum, 31));
  Group<C>::sync();
  const int2 free_pages = group_totals<C>(s, 0), needed = group_totals<C>(s, 1);
  if (needed.y > 0) list_free(a.ref_counts, sh, free_pages.x + s.warp[0][warp], min(needed.y, free_pages.y), a.list);
  // rows in order, each with its place in the list
  int at = needed.x + s.warp[1][warp] + before;
  for (int i = i0; i < i1; ++i) {
    const int lack = need[i];
    // as its place: refused -1, without a page -2
    need[i] = lack < 0 ? -1 : lack > 0 && lack > free_pages.y - at ? -2 : at;
    at += max(lack, 0);
  }
  Group<C>::sync();  // the list is written, and no CTA reads another's shared memory any more
  for (int i = warp; i < n; i += kWarps) {
    const int b = b0 + i;
    int place = need[i];
    if (lane == 0) a.status[b] = place == -1 ? kBadTree : place == -2 ? kNoPage : kOk;
    if (place < 0 || needed.y == 0) continue;
    const Range r = range_of(a, b);
    int32_t* row = a.block_table + static_cast<size_t>(b) * a.width;
    for (int q = r.t0; q < r.t1; q += 32 * kAhead) {
      bool lacks[kAhead];
      int from[kAhead], page[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int t = q + j * 32 + lane;
        lacks[j] = t < r.t1 && row[t] < 0;
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const unsigned m = __ballot_sync(0xffffffffu, lacks[j]);
        from[j] = place + __popc(m & ((1u << lane) - 1));
        place += __popc(m);
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) page[j] = lacks[j] ? a.list[from[j]] : 0;
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (lacks[j]) {
          row[q + j * 32 + lane] = page[j];
          a.ref_counts[page[j]] = 1;
        }
    }
  }
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
  __shared__ ScanSmem s;
  const int rank = Group<C>::rank(), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int i = rank * kThreads + threadIdx.x; i < a.rows; i += C * kThreads) a.first[i] = INT_MAX;
  const Share sh = share_of<C>(a.num_blocks, rank);
  const int mine = count_free(a.ref_counts, sh, a.num_blocks);
  Group<C>::sync();
  for (int i = rank * kThreads + threadIdx.x; i < a.new_rows; i += C * kThreads) {
    const Child c = child_of(a, i);
    if (c.code == kOk && c.parent >= 0) atomicMin(a.first + c.parent, i);
  }
  scan_warps(s, 0, mine);
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
  scan_warps(s, 1, __shfl_sync(0xffffffffu, before + sum, 31));
  Group<C>::sync();
  const int2 free_pages = group_totals<C>(s, 0), needed = group_totals<C>(s, 1);
  if (needed.y > 0) list_free(a.ref_counts, sh, free_pages.x + s.warp[0][warp], min(needed.y, free_pages.y), a.list);
  Group<C>::sync();
  int at = needed.x + s.warp[1][warp] + before;
  for (int i = i0; i < i1; ++i) {
    const int b = b0 + i;
    const Child c = child_of(a, b);
    int32_t* copy = a.copies + 3 * static_cast<size_t>(b);
    const int src = copy[0];
    int code = src == -2 ? kBadTree : c.code, dst = -1;
    if (src >= 0) {
      if (at < free_pages.y) {
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
  const int rank = Group<C>::rank(), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Share sh = share_of<C>(a.num_blocks, rank);
  scan_warps(s, 0, count_free(a.ref_counts, sh, a.num_blocks));
  Group<C>::sync();
  const int2 free_pages = group_totals<C>(s, 0);
  const int live = a.num_blocks - free_pages.y;
  // the holes: free pages below `live`, as many as pages in use from there on
  scan_warps(s, 1, count_free(a.ref_counts, sh, live));
  Group<C>::sync();
  const int holes = group_totals<C>(s, 1).y;
  int frees = free_pages.x + s.warp[0][warp];
  for (int q = sh.p0; q < sh.p1; q += 128) {
    const int p = q + lane * 4;
    const int4 r = counts_of(a.ref_counts, p, sh.p1, 1);
    const int m = free_mask(r), n = __popc(m);
    int f = frees + warp_before(n);  // free pages before this one
    const int count[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int page = p + j;
      if (page >= sh.p1) break;
      const bool is_free = m >> j & 1;
      if (page < live) {
        a.page_map[page] = is_free ? -1 : page;
        if (is_free) {
          a.copies[3 * static_cast<size_t>(f) + 1] = page;
          a.copies[3 * static_cast<size_t>(f) + 2] = kPage;
        } else {
          a.refs_out[page] = count[j];
        }
      } else {
        if (is_free) {
          a.page_map[page] = -1;
          a.refs_out[page] = 0;
        } else {
          // pages in use from `live` on, before this one
          a.copies[3 * static_cast<size_t>(page - live - (f - holes))] = page;
        }
      }
      f += is_free;
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

// A kernel of C CTAs of a cluster.
template <int C>
int launch_group(void (*kernel)(PageArgs), const PageArgs& a, size_t smem, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(C);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = C > 1 ? 1 : 0;
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

// How many CTAs: one for a pool that it reads in a few loads a thread, `most` pages
// (which spares two cluster barriers, about 2 us; its work behind the counts differs
// by kernel), 8 up to 2^18 pages, then 16 (512 rows over 650000 pages: alloc 31 us
// with 8, 23 with 16; 8 rows over 4000 pages: 10 us with 8, 12 with 16).
int ctas_for(const PageArgs& a, int most) {
  if (a.num_blocks <= most && a.rows <= kThreads && a.new_rows <= kThreads) return 1;
  return a.num_blocks < (1 << 18) ? 8 : kCluster;
}

}  // namespace

int launch_alloc_pages(const PageArgs& a, cudaStream_t stream) {
  static_assert(65536 / 8 * 4 <= 40 * 1024, "no opt-in");
  const int ctas = ctas_for(a, 16384);
  const size_t smem = static_cast<size_t>((a.rows + ctas - 1) / ctas) * 4;
  return ctas == 1   ? launch_group<1>(alloc_kernel<1>, a, smem, stream)
         : ctas == 8 ? launch_group<8>(alloc_kernel<8>, a, smem, stream)
                     : launch_group<kCluster>(alloc_kernel<kCluster>, a, smem, stream);
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
  const int rows = a.rows > a.new_rows ? a.rows : a.new_rows, ctas = ctas_for(a, 32768);
  // few entries are done by the same CTAs
  if (static_cast<long long>(rows) * a.width <= static_cast<long long>(ctas) * kFewEntries)
    return launch_fork_plan<true>(a, ctas, stream);
  if (launch_fork_plan<false>(a, ctas, stream)) return -1;
  return launch_behind(fork_rows_kernel, a, static_cast<unsigned>(rows), kRowThreads, stream);
}

int launch_compact_pages(const PageArgs& a, cudaStream_t stream) {
  const int ctas = ctas_for(a, 4096);
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
