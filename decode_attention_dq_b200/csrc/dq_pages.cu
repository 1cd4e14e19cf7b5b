// dq_pages.cu -- the pages of a paged cache: advancing every sequence by a
// step, forking sequences, compacting a pool, and copying pages.
//
// The state is three arrays of whole numbers: refs[p], how many references
// page p has (0: free), the page table T[b][j] (-1: no page) and the lengths
// L[b]. Each bookkeeping call reads one state and writes the next one:
//   advance  gives back what a sequence no longer needs and hands out the
//            pages of its next tokens
//   fork     row c of the new table is row parent[c] of the old one; full
//            pages are shared, a partly filled last page is copied, pages past
//            the length go to the first child
//   compact  moves the live pages to the lowest numbers
// Pages are handed out lowest first, in the order of the rows, and holes are
// filled in ascending order, so every result is determined by the state:
// nothing depends on the order of the atomics (sums of whole numbers).
//
// One launch each: a cluster of 16 CTAs goes through the phases with
// hardware cluster barriers in between and exchanges its counts through
// distributed shared memory. What bounds such a call at serving sizes is the
// chain of phases (releases before the free pages are known, these before a
// page is handed out), not bytes, and a barrier of one cluster costs less
// than a kernel boundary.
//
// Free pages and holes are found in two passes over refs: each warp counts in
// its own contiguous part, the counts are summed over the warps before it
// (block scan) and the CTAs before (distributed shared memory), then the
// warp goes through its part again and knows the rank of each page it finds.
#include <cooperative_groups.h>

#include <algorithm>

#include "dq_device.cuh"

namespace cg = cooperative_groups;

namespace dqi {
namespace {

// (Measured with 1, 2, 4, 8 and 16: 16 is the fastest from 777 pages up, 13.2 against 13.9 us for the smallest case, 39
// against 357 us for 600011 pages.)
constexpr int kCluster = 16;
constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kPage = 32;   // tokens per page
// A lane holds kQuads groups of four consecutive values at a time: four
// 16-byte loads in flight per lane, 64 KB per SM (with 32 bytes per lane the
// few SMs of a cluster waited for latency).
constexpr int kQuads = 4;
constexpr int kSeg = 32 * 4 * kQuads;  // table entries that a warp handles at a time (a work item)

// A CTA's part of the counts that the cluster exchanges.
struct Totals {
  long long free_pages, need;
  int released, bad, clamped;
};

struct Shared {
  Totals totals, before, all;
  long long scan[kWarps];
};

__device__ __forceinline__ long long warp_total(long long v) {
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// Sum of v (one per warp) over the warps of the CTA below this one and, in
// `total`, over all of them. Two barriers.
__device__ __forceinline__ long long block_exclusive(long long v, long long *sh, long long &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();
  if (lane == 0) sh[warp] = v;
  __syncthreads();
  const long long x = sh[lane];
  total = warp_total(x);
  return warp_total(lane < warp ? x : 0);
}

// Exclusive sum over the lanes of a small count; `total` over all of them.
__device__ __forceinline__ int lane_exclusive(int v, int &total) {
  int x = v;
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, x, o);
    if (static_cast<int>(threadIdx.x & 31) >= o) x += y;
  }
  total = __shfl_sync(kFull, x, 31);
  return x - v;
}

// [lo, hi) of part i out of n of [0, size).
__device__ __forceinline__ void part(long long size, long long i, long long n, long long &lo, long long &hi) {
  lo = size * i / n;
  hi = size * (i + 1) / n;
}

// This warp's part of num_pages, in whole groups of four.
__device__ __forceinline__ void warp_part(long long P, long long rank, long long &lo, long long &hi) {
  part((P + 3) / 4, rank * kWarps + (threadIdx.x >> 5), kCluster * kWarps, lo, hi);
  lo *= 4;
  hi = hi * 4 < P ? hi * 4 : P;
}

__device__ __forceinline__ bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// x[i .. i + 3], `other` from `end` on; past L1, which other CTAs' stores do
// not reach. vec: x is 16-byte aligned and i a multiple of 4.
__device__ __forceinline__ int4 load4(const int32_t *x, long long i, long long end, bool vec, int other) {
  if (vec && i + 3 < end) return __ldcg(reinterpret_cast<const int4 *>(x + i));
  return make_int4(i < end ? __ldcg(x + i) : other, i + 1 < end ? __ldcg(x + i + 1) : other,
                   i + 2 < end ? __ldcg(x + i + 2) : other, i + 3 < end ? __ldcg(x + i + 3) : other);
}
__device__ __forceinline__ void store4(int32_t *x, long long i, long long end, bool vec, const int (&v)[4]) {
  if (vec && i + 3 < end) {
    *reinterpret_cast<int4 *>(x + i) = make_int4(v[0], v[1], v[2], v[3]);
    return;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (i + k < end) x[i + k] = v[k];
}

// Calls f(index of the first, values) for this lane's groups of four of
// x[lo, hi), in ascending order over the calls and the lanes; all lanes call
// it together. lo is a multiple of 4 or vec is false.
template <class F>
__device__ __forceinline__ void for_quads(const int32_t *x, long long lo, long long hi, bool vec, int other, F f) {
  const int lane = threadIdx.x & 31;
  for (long long i0 = lo; i0 < hi; i0 += 128 * kQuads) {
    int4 v[kQuads];
#pragma unroll
    for (int k = 0; k < kQuads; ++k) v[k] = load4(x, i0 + 128 * k + 4 * lane, hi, vec, other);
#pragma unroll
    for (int k = 0; k < kQuads; ++k)
      if (i0 + 128 * k < hi) {
        const int q[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
        f(i0 + 128 * k + 4 * lane, q);
      }
  }
}

__device__ __forceinline__ int ballot_rank(unsigned mask) {
  return __popc(mask & ((1u << (threadIdx.x & 31)) - 1u));
}

__device__ __forceinline__ long long clamp_tokens(int len, long long cap) {
  return len < 0 ? 0 : (len > cap ? cap : len);
}

// Adds a thread's counts to the CTA's.
__device__ __forceinline__ void add_counts(Totals *mine, int released, int bad, int clamped) {
  released = __reduce_add_sync(kFull, released);
  bad = __reduce_add_sync(kFull, bad);
  clamped = __reduce_add_sync(kFull, clamped);
  if ((threadIdx.x & 31) == 0) {
    if (released) atomicAdd(&mine->released, released);
    if (bad) atomicAdd(&mine->bad, bad);
    if (clamped) atomicAdd(&mine->clamped, clamped);
  }
}

// After a cluster barrier: the counts of the CTAs before this one (free pages
// and needs) and of all. The first warp reads them, a CTA per lane.
__device__ __forceinline__ void exchange(cg::cluster_group &cl, Shared &sh, Totals &before, Totals &all) {
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x, rank = static_cast<int>(cl.block_rank());
    Totals t{};
    if (lane < kCluster) t = *cl.map_shared_rank(&sh.totals, lane);
    Totals b{};
    b.free_pages = warp_total(lane < rank ? t.free_pages : 0);
    b.need = warp_total(lane < rank ? t.need : 0);
    t.free_pages = warp_total(t.free_pages);
    t.need = warp_total(t.need);
    t.released = __reduce_add_sync(kFull, t.released);
    t.bad = __reduce_add_sync(kFull, t.bad);
    t.clamped = __reduce_add_sync(kFull, t.clamped);
    if (lane == 0) {
      sh.before = b;
      sh.all = t;
    }
  }
  __syncthreads();
  before = sh.before;
  all = sh.all;
}

// d_counts: see dq_page_counts in dq.h.
__device__ __forceinline__ void write_counts(int32_t *c, long long free_pages, long long taken, int released,
                                             long long short_of, int bad, int clamped, long long pairs) {
  c[0] = static_cast<int32_t>(free_pages);
  c[1] = static_cast<int32_t>(taken);
  c[2] = released;
  c[3] = static_cast<int32_t>(short_of);
  c[4] = bad;
  c[5] = clamped;
  c[6] = static_cast<int32_t>(pairs);
  c[7] = 0;
}

// The free pages (0 in `refs`) of this warp's part get their ranks; those
// below `take` go into list[rank] and are taken in refs_out.
__device__ __forceinline__ void list_free(const int32_t *refs, long long lo, long long hi, bool vec, long long rank,
                                          long long take, int32_t *list, int32_t *refs_out) {
  if (rank >= take) return;
  for_quads(refs, lo, hi, vec, 1, [&](long long p, const int (&v)[4]) {
    const int n = (v[0] == 0) + (v[1] == 0) + (v[2] == 0) + (v[3] == 0);
    if (rank >= take || !__any_sync(kFull, n)) return;
    int total;
    long long r = rank + lane_exclusive(n, total);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (v[k] == 0) {
        if (r < take) {
          list[r] = static_cast<int32_t>(p + k);
          atomicAdd(refs_out + p + k, 1);
        }
        ++r;
      }
    rank += total;
  });
}

__device__ __forceinline__ long long count_free(const int32_t *refs, long long lo, long long hi, bool vec) {
  int n = 0;
  for_quads(refs, lo, hi, vec, 1, [&](long long, const int (&v)[4]) {
    n += (v[0] == 0) + (v[1] == 0) + (v[2] == 0) + (v[3] == 0);
  });
  return warp_total(n);
}

__device__ __forceinline__ void copy_refs(const PagesArgs &a, long long lo, long long hi, bool vec) {
  for_quads(a.refs_in, lo, hi, vec, 0, [&](long long p, const int (&v)[4]) { store4(a.refs_out, p, hi, vec, v); });
}

struct RowCounts {
  int released, bad, clamped;
};

// One work item of dq_pages_advance, by a warp: what is given back, and how
// many entries want a page.
__device__ __forceinline__ void advance_item(const PagesArgs &a, long long it, long long nseg, long long cap, bool vec,
                                             RowCounts &n_of) {
  const int lane = threadIdx.x & 31;
  const long long P = a.num_pages, mp = a.max_pages;
  const long long b = it / nseg, j0 = (it % nseg) * kSeg, j1 = j0 + kSeg < mp ? j0 + kSeg : mp;
  const int raw = a.lens_in[b], n = a.step[b];
  const long long len = clamp_tokens(raw, cap), want = n < 0 ? 0 : len + n;
  const long long len2 = want < cap ? want : cap;
  if (j0 == 0 && lane == 0) n_of.clamped += (raw != len || want != len2) ? 1 : 0;
  // Blocks [g_lo, g_hi) are given back; blocks [t_lo, t_hi) need a page.
  long long g_lo = 0, g_hi = n < 0 ? mp : 0;
  if (n > 0 && a.window > 0) {  // (a row that gets no token may attend from its last one again)
    g_lo = (a.sinks + kPage - 1) / kPage;
    const long long seen = len + 1 - a.window;  // the first token that a next one sees
    g_hi = seen > 0 ? seen / kPage : 0;
  }
  const bool grows = n > 0 && len2 > len;
  const long long t_lo = grows ? len / kPage : 0, t_hi = grows ? (len2 + kPage - 1) / kPage : 0;
  int32_t *out = a.table_out + b * mp;
  int need = 0;
  for_quads(a.table_in + b * mp, j0, j1, vec, -1, [&](long long j, const int (&e)[4]) {
    int v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool held = e[k] >= 0 && e[k] < P;
      const bool gone = j + k >= g_lo && j + k < g_hi;
      n_of.bad += (!held && e[k] != -1) ? 1 : 0;
      if (held && gone) {
        atomicSub(a.refs_out + e[k], 1);
        ++n_of.released;
      }
      v[k] = held && !gone ? e[k] : -1;
      need += (v[k] < 0 && j + k >= t_lo && j + k < t_hi) ? 1 : 0;
    }
    store4(out, j, j1, vec, v);
  });
  need = __reduce_add_sync(kFull, need);
  if (lane == 0) {
    a.item_need[it] = need;
    a.item_lo[it] = static_cast<int32_t>(t_lo > j0 ? t_lo : j0);
    a.item_hi[it] = static_cast<int32_t>(t_hi < j1 ? t_hi : j1);
  }
}

__device__ __forceinline__ long long max_tokens(const PagesArgs &a) {
  return kPage * a.max_pages < 0x7FFFFFFF ? kPage * a.max_pages : 0x7FFFFFFF;
}
__device__ __forceinline__ bool aligned_rows(const PagesArgs &a) {
  return aligned16(a.table_in) && aligned16(a.table_out) && a.max_pages % 4 == 0;
}

// Large states: the counts' copy and the rows on all SMs, in two launches of
// their own before advance_kernel<false>; the rows' counts gather in d_counts.
__global__ void __launch_bounds__(kThreads) advance_copy_kernel(const PagesArgs a) {
  const long long warps = static_cast<long long>(gridDim.x) * kWarps;
  if (blockIdx.x == 0 && threadIdx.x < 8) a.counts[threadIdx.x] = 0;
  if (a.refs_out == a.refs_in) return;
  long long lo, hi;
  part((a.num_pages + 3) / 4, static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5), warps, lo, hi);
  hi = hi * 4 < a.num_pages ? hi * 4 : a.num_pages;
  copy_refs(a, lo * 4, hi, aligned16(a.refs_in) && aligned16(a.refs_out));
}
__global__ void __launch_bounds__(kThreads) advance_rows_kernel(const PagesArgs a) {
  const long long nseg = (a.max_pages + kSeg - 1) / kSeg, items = a.B_in * nseg;
  RowCounts n{0, 0, 0};
  for (long long it = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5); it < items;
       it += static_cast<long long>(gridDim.x) * kWarps)
    advance_item(a, it, nseg, max_tokens(a), aligned_rows(a), n);
  n.released = __reduce_add_sync(kFull, n.released);
  n.bad = __reduce_add_sync(kFull, n.bad);
  n.clamped = __reduce_add_sync(kFull, n.clamped);
  if ((threadIdx.x & 31) == 0) {
    if (n.released) atomicAdd(a.counts + 2, n.released);
    if (n.bad) atomicAdd(a.counts + 4, n.bad);
    if (n.clamped) atomicAdd(a.counts + 5, n.clamped);
  }
}

// kRows: with the copy of the counts and the rows; else they have been done.
template <bool kRows>
__global__ void __launch_bounds__(kThreads, 1) advance_kernel(const PagesArgs a) {
  cg::cluster_group cl = cg::this_cluster();
  __shared__ Shared sh;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = static_cast<int>(cl.block_rank());
  const long long P = a.num_pages, mp = a.max_pages, cap = max_tokens(a);
  const long long nseg = (mp + kSeg - 1) / kSeg, items = a.B_in * nseg;
  const bool vec_refs = aligned16(a.refs_in) && aligned16(a.refs_out);
  if (threadIdx.x == 0) sh.totals = Totals{};
  long long w_lo, w_hi, i_lo, i_hi;
  warp_part(P, rank, w_lo, w_hi);
  part(items, rank, kCluster, i_lo, i_hi);
  if constexpr (kRows) {
    if (a.refs_out != a.refs_in) copy_refs(a, w_lo, w_hi, vec_refs);
    cl.sync();
    RowCounts n{0, 0, 0};
    for (long long it = i_lo + warp; it < i_hi; it += kWarps) advance_item(a, it, nseg, cap, aligned_rows(a), n);
    add_counts(&sh.totals, n.released, n.bad, n.clamped);
    cl.sync();
  } else {
    __syncthreads();
    if (rank == 0 && threadIdx.x == 0) {
      sh.totals.released = a.counts[2];
      sh.totals.bad = a.counts[4];
      sh.totals.clamped = a.counts[5];
    }
  }

  // Lengths (all have been read); needs of this CTA; free pages of its part.
  for (long long b = static_cast<long long>(rank) * kThreads + threadIdx.x; b < a.B_in; b += kCluster * kThreads) {
    const int n = a.step[b];
    const long long want = n < 0 ? 0 : clamp_tokens(a.lens_in[b], cap) + n;
    a.lens_out[b] = static_cast<int32_t>(want < cap ? want : cap);
  }
  long long need = 0, total;
  for (long long it = i_lo + threadIdx.x; it < i_hi; it += kThreads) need += a.item_need[it];
  const long long mine = count_free(a.refs_out, w_lo, w_hi, vec_refs);
  block_exclusive(warp_total(need), sh.scan, total);
  if (threadIdx.x == 0) sh.totals.need = total;
  const long long w_before = block_exclusive(mine, sh.scan, total);
  if (threadIdx.x == 0) sh.totals.free_pages = total;
  cl.sync();
  Totals before, all;
  exchange(cl, sh, before, all);
  const long long take = all.need < all.free_pages ? all.need : all.free_pages;
  if (rank == 0 && threadIdx.x == 0)
    write_counts(a.counts, all.free_pages - take, take, all.released, all.need - take, all.bad, all.clamped, 0);
  list_free(a.refs_out, w_lo, w_hi, vec_refs, before.free_pages + w_before, take, a.list, a.refs_out);
  cl.sync();

  // The items' entries, in their order: the rank of each item's first one,
  // then an item per warp.
  __shared__ long long first[kThreads];
  long long base = before.need;
  for (long long c0 = i_lo; c0 < i_hi; c0 += kThreads) {
    const long long it = c0 + threadIdx.x;
    int in_warp;
    const int before_lane = lane_exclusive(it < i_hi ? a.item_need[it] : 0, in_warp);
    first[threadIdx.x] = base + block_exclusive(in_warp, sh.scan, total) + before_lane;
    base += total;
    __syncthreads();
    for (long long id = c0 + warp; id < i_hi && id < c0 + kThreads; id += kWarps) {
      if (a.item_need[id] == 0) continue;
      long long r = first[id - c0];
      int32_t *out = a.table_out + (id / nseg) * mp;
      const int hi = a.item_hi[id];
      for (int j0 = a.item_lo[id]; j0 < hi; j0 += 32) {
        const int j = j0 + lane;
        const bool w = j < hi && __ldcg(out + j) < 0;
        const unsigned m = __ballot_sync(kFull, w);
        if (w) {
          const long long x = r + ballot_rank(m);
          if (x < take) out[j] = __ldcg(a.list + x);
        }
        r += __popc(m);
      }
    }
    __syncthreads();  // `first` is written again
  }
}

__global__ void __launch_bounds__(kThreads, 1) fork_kernel(const PagesArgs a) {
  cg::cluster_group cl = cg::this_cluster();
  __shared__ Shared sh;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = static_cast<int>(cl.block_rank());
  const long long P = a.num_pages, mp = a.max_pages, cap = kPage * mp < 0x7FFFFFFF ? kPage * mp : 0x7FFFFFFF;
  const long long nseg = (mp + kSeg - 1) / kSeg;
  const long long tid = static_cast<long long>(rank) * kThreads + threadIdx.x, threads = kCluster * kThreads;
  const bool vec_refs = aligned16(a.refs_in) && aligned16(a.refs_out);
  const bool vec_rows = aligned16(a.table_in) && aligned16(a.table_out) && mp % 4 == 0;
  if (threadIdx.x == 0) sh.totals = Totals{};
  long long w_lo, w_hi, c_lo, c_hi;
  warp_part(P, rank, w_lo, w_hi);
  part(a.B_out, rank, kCluster, c_lo, c_hi);  // the rows whose new pages this CTA hands out
  for (long long b = tid; b < a.B_in; b += threads) {
    a.children[b] = 0;
    a.first[b] = 0x7FFFFFFF;
  }
  copy_refs(a, w_lo, w_hi, vec_refs);
  cl.sync();

  int bad = 0, clamped = 0;
  for (long long c = tid; c < a.B_out; c += threads) {
    const int p = a.step[c];
    if (p >= 0 && p < a.B_in) {
      atomicAdd(a.children + p, 1);
      atomicMin(a.first + p, static_cast<int>(c));
    } else if (p >= 0) {
      ++bad;
    }
  }
  const long long mine = count_free(a.refs_in, w_lo, w_hi, vec_refs);
  cl.sync();

  // Whether a page t that the row will write to stays with its first child:
  // nobody else may hold it.
  auto stays = [&](int t) { return __ldcg(a.refs_in + t) == 1; };
  // The old rows' references go, the children's come (items of all rows, over
  // the cluster); then the new rows (those whose new pages this CTA hands out,
  // so that it knows how many they are).
  int need = 0;
  auto do_item = [&](bool is_new, long long it) {
    const long long row = it / nseg, seg = it % nseg;
    const long long j0 = seg * kSeg, j1 = j0 + kSeg < mp ? j0 + kSeg : mp;
    const int parent = is_new ? a.step[row] : static_cast<int>(row);
    const bool real = parent >= 0 && parent < a.B_in;
    const int raw = real ? a.lens_in[parent] : 0;
    const long long len = clamp_tokens(raw, cap);
    // Blocks from own_lo on are written to as the row grows: the partly filled
    // one (col), then those that lie past the length.
    const long long own_lo = len / kPage, col = len % kPage ? own_lo : -1;
    if (!is_new && seg == 0 && lane == 0 && raw != len) ++clamped;
    const int kids = real ? __ldcg(a.children + parent) : 0;
    if (!is_new && kids == 1 && j1 <= own_lo) return;  // its pages keep their references
    const bool is_first = is_new && real && __ldcg(a.first + parent) == row;
    int32_t *out = a.table_out + row * mp;
    if (!real) {  // a row without a parent (there may be no old table at all)
      for (long long j = j0 + lane; j < j1; j += 32) out[j] = -1;
      if (seg == 0 && lane == 0) {
        a.lens_out[row] = 0;
        a.item_need[row] = 0;
      }
      return;
    }
    for_quads(a.table_in + parent * mp, j0, j1, vec_rows, -1, [&](long long j, const int (&e)[4]) {
      int v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const bool held = e[k] >= 0 && e[k] < P, own = j + k >= own_lo;
        v[k] = held ? e[k] : -1;
        if (is_new) {
          bad += (!held && e[k] != -1) ? 1 : 0;
          const bool leave = held && own && !(is_first && stays(e[k]));
          if (j + k == col) {
            need += leave ? 1 : 0;
            a.item_need[row] = leave ? 1 : 0;
            a.item_lo[row] = v[k];  // the page to copy from
            a.item_hi[row] = static_cast<int32_t>(col);
          }
          if (leave) v[k] = -1;
        } else if (held) {
          const int d = own ? (kids > 0 && stays(e[k]) ? 0 : -1) : kids - 1;
          if (d) atomicAdd(a.refs_out + e[k], d);
        }
      }
      if (is_new) store4(out, j, j1, vec_rows, v);
    });
    if (is_new && seg == 0 && lane == 0) {
      a.lens_out[row] = static_cast<int32_t>(len);
      if (col < 0) a.item_need[row] = 0;
    }
  };
  for (long long it = static_cast<long long>(rank) * kWarps + warp; it < a.B_in * nseg; it += kCluster * kWarps)
    do_item(false, it);
  for (long long it = c_lo * nseg + warp; it < c_hi * nseg; it += kWarps) do_item(true, it);
  add_counts(&sh.totals, 0, bad, clamped);
  long long total;
  const long long w_before = block_exclusive(mine, sh.scan, total);
  if (threadIdx.x == 0) sh.totals.free_pages = total;
  block_exclusive(warp_total(need), sh.scan, total);
  if (threadIdx.x == 0) sh.totals.need = total;
  cl.sync();
  Totals before, all;
  exchange(cl, sh, before, all);
  const long long take = all.need < all.free_pages ? all.need : all.free_pages;
  if (rank == 0 && threadIdx.x == 0)
    write_counts(a.counts, 0, take, 0, all.need - take, all.bad, all.clamped, take);  // (the free pages are added below)
  list_free(a.refs_in, w_lo, w_hi, vec_refs, before.free_pages + w_before, take, a.list, a.refs_out);
  for (long long i = take + tid; i < a.B_out; i += threads) {
    a.pairs[2 * i] = -1;
    a.pairs[2 * i + 1] = -1;
  }
  cl.sync();

  long long base = before.need;
  for (long long c0 = c_lo; c0 < c_hi; c0 += kThreads) {
    const long long c = c0 + threadIdx.x;
    const bool w = c < c_hi && __ldcg(a.item_need + c) != 0;
    const unsigned m = __ballot_sync(kFull, w);
    const long long r = base + block_exclusive(__popc(m), sh.scan, total) + ballot_rank(m);
    base += total;
    if (w && r < take) {
      const int page = __ldcg(a.list + r);
      a.pairs[2 * r] = __ldcg(a.item_lo + c);
      a.pairs[2 * r + 1] = page;
      a.table_out[c * mp + __ldcg(a.item_hi + c)] = page;
    }
  }
  // (Counted at the end: atomics that return what a page had before would
  // each be waited for.)
  const long long left = count_free(a.refs_out, w_lo, w_hi, vec_refs);
  block_exclusive(left, sh.scan, total);
  if (threadIdx.x == 0 && total) atomicAdd(a.counts, static_cast<int>(total));
}

__global__ void __launch_bounds__(kThreads, 1) compact_kernel(const PagesArgs a) {
  cg::cluster_group cl = cg::this_cluster();
  __shared__ Shared sh;
  const int rank = static_cast<int>(cl.block_rank());
  const long long P = a.num_pages, entries = static_cast<long long>(a.B_in) * a.max_pages;
  const long long tid = static_cast<long long>(rank) * kThreads + threadIdx.x, threads = kCluster * kThreads;
  const bool vec_refs = aligned16(a.refs_in);
  if (threadIdx.x == 0) sh.totals = Totals{};
  long long w_lo, w_hi;
  warp_part(P, rank, w_lo, w_hi);
  int live = 0;
  for_quads(a.refs_in, w_lo, w_hi, vec_refs, 0, [&](long long, const int (&v)[4]) {
    live += (v[0] > 0) + (v[1] > 0) + (v[2] > 0) + (v[3] > 0);
  });
  long long total;
  const long long w_before = block_exclusive(warp_total(live), sh.scan, total);
  if (threadIdx.x == 0) sh.totals.need = total;
  cl.sync();
  Totals before, all;
  exchange(cl, sh, before, all);
  const long long n_live = all.need;

  // Live pages below n_live stay. A hole's index is the number of holes
  // before it; the movers are indexed from the last one down, which needs no
  // count of those that stay.
  long long lr = before.need + w_before;  // live pages before the next one
  int holes = 0;
  for_quads(a.refs_in, w_lo, w_hi, vec_refs, 0, [&](long long p0, const int (&v)[4]) {
    int in_warp;
    long long r = lr + lane_exclusive((v[0] > 0) + (v[1] > 0) + (v[2] > 0) + (v[3] > 0), in_warp);
    lr += in_warp;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const long long p = p0 + k;
      const bool lv = v[k] > 0;
      if (p < w_hi && p < n_live) {
        a.map[p] = lv ? static_cast<int32_t>(p) : -1;
        if (lv) {
          a.refs_out[p] = v[k];
        } else {
          a.list[p - r] = static_cast<int32_t>(p);
          ++holes;
        }
      } else if (p < w_hi) {
        if (lv) {
          a.movers[n_live - 1 - r] = static_cast<int32_t>(p);
        } else {
          a.map[p] = -1;
          a.refs_out[p] = 0;
        }
      }
      r += lv ? 1 : 0;
    }
  });
  block_exclusive(warp_total(holes), sh.scan, total);
  if (threadIdx.x == 0) sh.totals.free_pages = total;
  cl.sync();
  exchange(cl, sh, before, all);
  const long long moves = all.free_pages, cap = P / 2 > 1 ? P / 2 : 1;
  for (long long i = tid; i < cap; i += threads) {
    int src = -1, dst = -1;
    if (i < moves) {
      src = __ldcg(a.movers + (moves - 1 - i));
      dst = __ldcg(a.list + i);
      a.map[src] = dst;
      a.refs_out[dst] = __ldcg(a.refs_in + src);
      a.refs_out[src] = 0;
    }
    a.pairs[2 * i] = src;
    a.pairs[2 * i + 1] = dst;
  }
  cl.sync();

  int bad = 0;
  const bool vec = aligned16(a.table_in) && aligned16(a.table_out);
  long long e_lo, e_hi;
  part((entries + 3) / 4, static_cast<long long>(rank) * kWarps + (threadIdx.x >> 5), kCluster * kWarps, e_lo, e_hi);
  e_hi = e_hi * 4 < entries ? e_hi * 4 : entries;
  for_quads(a.table_in, e_lo * 4, e_hi, vec, -1, [&](long long i, const int (&e)[4]) {
    int v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool held = e[k] >= 0 && e[k] < P;
      bad += (!held && e[k] != -1) ? 1 : 0;
      v[k] = held ? __ldcg(a.map + e[k]) : -1;
    }
    store4(a.table_out, i, e_hi, vec, v);
  });
  add_counts(&sh.totals, 0, bad, 0);
  cl.sync();
  if (rank == 0) {
    exchange(cl, sh, before, all);
    if (threadIdx.x == 0) write_counts(a.counts, P - n_live, 0, 0, 0, all.bad, 0, moves);
  }
  cl.sync();  // the others' counts have been read before they leave
}

// Pages src -> dst of both pools in every layer. A warp copies pieces of
// kPiece bytes, eight 16-byte loads in flight per lane before the first store
// (two: 5 % slower, four: 2 %). 226 MB of pages take 73 us: 6.2 TB/s read and
// written, 0.96 of a measured copy.
constexpr int kLoads = 8;
constexpr int kPiece = 32 * 16 * kLoads;
constexpr int kCopyThreads = 256;
constexpr int kCopyBlocksPerSm = 8;

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const CopyArgs a) {
  long long n = a.max_pairs;
  if (a.counts) {
    const long long c = a.counts[6];
    n = c < 0 ? 0 : (c < n ? c : n);
  }
  const int lane = threadIdx.x & 31;
  const unsigned kp = static_cast<unsigned>((a.k_bytes + kPiece - 1) / kPiece);
  const unsigned pieces = kp + static_cast<unsigned>((a.v_bytes + kPiece - 1) / kPiece);  // of one page in one layer
  const long long units = n * a.n_layers * pieces;
  const long long warps = static_cast<long long>(gridDim.x) * (kCopyThreads / 32);
  unsigned bad = 0;
  for (long long u = (static_cast<long long>(blockIdx.x) * kCopyThreads + threadIdx.x) >> 5; u < units; u += warps) {
    const long long pl = u / pieces;
    const unsigned piece = static_cast<unsigned>(u - pl * pieces);
    const long long layer = pl / n, i = pl - layer * n;
    const int src = a.pairs[2 * i], dst = a.pairs[2 * i + 1];
    if (src < 0 && dst < 0) continue;
    if (src < 0 || dst < 0 || src >= a.num_pages || dst >= a.num_pages) {
      if (layer == 0 && piece == 0) ++bad;
      continue;
    }
    const bool is_k = piece < kp;
    const int64_t bytes = is_k ? a.k_bytes : a.v_bytes;
    uint8_t *pool = is_k ? a.kpool + layer * a.k_stride : a.vpool + layer * a.v_stride;
    const int64_t at = static_cast<int64_t>(is_k ? piece : piece - kp) * kPiece + lane * 16;
    const uint8_t *from = pool + src * bytes + at;
    uint8_t *to = pool + dst * bytes + at;
    uint4 x[kLoads];
#pragma unroll
    for (int k = 0; k < kLoads; ++k)
      if (at + 512 * k < bytes) x[k] = __ldcs(reinterpret_cast<const uint4 *>(from + 512 * k));
#pragma unroll
    for (int k = 0; k < kLoads; ++k)
      if (at + 512 * k < bytes) __stcs(reinterpret_cast<uint4 *>(to + 512 * k), x[k]);
  }
  if (a.stats && lane == 0 && bad) atomicAdd(&a.stats->bad_pages, static_cast<unsigned long long>(bad));
}

template <auto Kern>
int launch_cluster(const PagesArgs &a, cudaStream_t st) {
  const cudaError_t e = allow_wide_cluster<Kern>();
  if (e != cudaSuccess) return static_cast<int>(e);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kCluster);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = kCluster;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return static_cast<int>(cudaLaunchKernelEx(&cfg, Kern, a));
}

}  // namespace

// Counts and table entries up to which dq_pages_advance is one launch. (One
// launch and three: 12.8 and 15.1 us for 41 thousand, 17.5 and 18.4 us for 462
// thousand, 25.9 and 22.0 us for 924 thousand, 37.6 and 25.0 us for 1.6 million.)
constexpr int64_t kOneLaunch = int64_t(5) << 17;

PagesLayout pages_layout(int64_t num_pages, int64_t B, int64_t max_pages) {
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  PagesLayout l;
  const size_t rows = static_cast<size_t>(B), pages = static_cast<size_t>(num_pages);
  const size_t items = rows * ((max_pages + kSeg - 1) / kSeg);
  l.list = 0;  // the pages handed out, or a hole per move: never more than there are pages
  l.need = l.list + up(4 * pages);
  l.lo = l.need + up(4 * items);
  l.hi = l.lo + up(4 * items);
  l.map = l.hi + up(4 * items);                               // compact: new numbers; fork: children of each row
  l.movers = l.map + up(4 * std::max(pages, rows));           // compact: pages that move; fork: first children
  l.total = l.movers + up(4 * std::max(pages / 2 + 1, rows));
  return l;
}

int launch_pages_advance(const PagesArgs &a, int sm_count, void *stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (a.num_pages + a.B_in * a.max_pages <= kOneLaunch) return launch_cluster<advance_kernel<true>>(a, st);
  advance_copy_kernel<<<sm_count, kThreads, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return static_cast<int>(e);
  advance_rows_kernel<<<sm_count, kThreads, 0, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return static_cast<int>(e);
  return launch_cluster<advance_kernel<false>>(a, st);
}
int launch_pages_fork(const PagesArgs &a, void *stream) {
  return launch_cluster<fork_kernel>(a, static_cast<cudaStream_t>(stream));
}
int launch_pages_compact(const PagesArgs &a, void *stream) {
  return launch_cluster<compact_kernel>(a, static_cast<cudaStream_t>(stream));
}

int launch_pages_copy(const CopyArgs &a, int sm_count, void *stream) {
  const int64_t pieces = (a.k_bytes + kPiece - 1) / kPiece + (a.v_bytes + kPiece - 1) / kPiece;
  const int64_t most = a.max_pairs * a.n_layers * pieces;  // warps that could have work
  const int64_t blocks = (most + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
  const int64_t full = static_cast<int64_t>(sm_count) * kCopyBlocksPerSm;
  copy_kernel<<<static_cast<unsigned>(blocks < full ? blocks : full), kCopyThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return static_cast<int>(cudaGetLastError());
}

}  // namespace dqi
