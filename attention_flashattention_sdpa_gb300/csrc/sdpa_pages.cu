// sdpa_pages.cu — who owns which page of a cache, and pages and rows moved inside it.
//
// Every page has a count of its owners (rows of page tables, and what else the program counts); a page
// is free iff its count is 0, and free pages are given lowest first, so that results depend on nothing else.
//
//   fork     row i of the new table is row parents[i] of the old one; counts: + the new rows, - the old
//   grow     the columns between two lengths get free pages in the order of (row, column); a partly filled
//            page with other owners is replaced by a free one, and listed as a copy to make
//   free     the columns behind a shorter length are given back
//   compact  of n pages in use the k-th at or behind n moves to the k-th free one before n
//   copy     pages of K, V and their scales, by a list
//   keep     rows of the newest tokens move to the front of them
//
// The first four are integer work on tables of a few hundred thousand entries at most, bound by latency: one
// cluster of CTAs each (a single CTA for small tables), whose barrier stands between the passes that depend on each
// other (counts before ids, copies of counts before atomics on them), so that each is one launch and needs no
// workspace.  Fork and free of more than 256 pieces of rows go over the whole GPU instead, as their passes need no order once the
// counts are where they are wanted: behind a copy of them, where that is elsewhere.  Atomics are sums of integers: their
// order changes nothing.  Measured (replayed), 64 rows of 256 columns in 32768 pages: fork 5.5 us, grow 8.2, free 4.5, compact
// 10.9; 4 rows of 16: 1.8, 5.0, 2.1, 4.4.
#include "ptx.cuh"
#include "sdpa_internal.h"

namespace sdpa {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kChunk = 128;          // columns of a row that a warp takes at once
constexpr int kEach = 4;             // counts a thread takes at once
constexpr int kTile = kThreads * kEach;

// The CTAs of a launch are one cluster: of one CTA for small work, of 8 otherwise.
__device__ __forceinline__ int rank() { return static_cast<int>(blockIdx.x); }
__device__ __forceinline__ int ranks() { return static_cast<int>(gridDim.x); }

__device__ __forceinline__ void sync_all() {
  if (gridDim.x > 1) ptx::cluster_sync_all();
  else __syncthreads();
}

// Whatever ran before is done; what comes next may be put in place meanwhile (it waits here in its turn).  What the kernels read
// may have been written while they were already there, so it comes by plain loads, which stay behind the wait.
__device__ __forceinline__ void begin() {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
}

struct Range {
  int lo, hi;
};

// Pages that CTA `k` looks after.
__device__ __forceinline__ Range share(int n, int k) {
  const int per = (n + ranks() - 1) / ranks();
  return {static_cast<int>(min(static_cast<int64_t>(n), static_cast<int64_t>(k) * per)),
          static_cast<int>(min(static_cast<int64_t>(n), static_cast<int64_t>(k + 1) * per))};
}

// Exclusive prefix sum over the CTA's threads of x; the total in `total`.  `tmp`: kWarps words.
__device__ __forceinline__ int block_scan(int x, int* tmp, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = x;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) tmp[warp] = inc;
  __syncthreads();
  // (Every warp adds up the warps for itself: one barrier less than a warp that does it for all.)
  int w = tmp[lane];
  const int mine = w;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const int before = __shfl_sync(0xffffffffu, w - mine, warp) + inc - x;
  __syncthreads();
  return before;
}

__device__ __forceinline__ int block_sum(int x, int* tmp) {
  x = __reduce_add_sync(0xffffffffu, x);
  if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = x;
  __syncthreads();
  const int total = __reduce_add_sync(0xffffffffu, tmp[threadIdx.x & 31]);
  __syncthreads();
  return total;
}

// x of every CTA, in every CTA: all[k] is that of CTA k afterwards (the barrier is the cluster's).  Once in a kernel that begins
// with meet(): a CTA's shared memory is there for the others once it has begun.
__device__ __forceinline__ void meet() {
  if (gridDim.x > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}

__device__ __forceinline__ void exchange(int x, int* all) {
  if (gridDim.x == 1) {
    if (threadIdx.x == 0) all[0] = x;
    __syncthreads();
    return;
  }
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (threadIdx.x < gridDim.x) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(ptx::smem_u32(all + rank())), "r"(threadIdx.x));
    asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(a), "r"(x) : "memory");
  }
  ptx::cluster_sync_all();
}

__device__ __forceinline__ int clamp_tokens(const int32_t* lens, int i, int top) { return min(max(lens[i], 0), top); }

__device__ __forceinline__ int columns_of(const PagesParams& p, int len) {
  return static_cast<int>((static_cast<int64_t>(len) + p.page_size - 1) / p.page_size);
}

__device__ __forceinline__ bool is_page(int page, int n) { return page >= 0 && page < n; }

// f(row, first column) for every piece of kChunk columns of `rows` rows, a warp each.
template <typename F>
__device__ __forceinline__ void for_chunks(int rows, int columns, F f) {
  const uint32_t chunks = (columns + kChunk - 1) / kChunk, n = chunks * rows;
  for (uint32_t x = rank() * kWarps + (threadIdx.x >> 5); x < n; x += ranks() * kWarps) {
    const uint32_t i = x / chunks;
    f(static_cast<int>(i), static_cast<int>((x - i * chunks) * kChunk));
  }
}

// Counts as they are, where they are wanted elsewhere, before anyone adds to them.
__device__ __forceinline__ void copy_counts(const PagesParams& p) {
  if (p.ref_counts_out == p.ref_counts) return;
  const int step = ranks() * kThreads;
  for (int64_t i0 = rank() * kThreads + threadIdx.x; i0 < p.num_pages; i0 += kEach * step) {
    int count[kEach];
#pragma unroll
    for (int e = 0; e < kEach; ++e) count[e] = i0 + e * step < p.num_pages ? p.ref_counts[i0 + e * step] : 0;
#pragma unroll
    for (int e = 0; e < kEach; ++e)
      if (i0 + e * step < p.num_pages) p.ref_counts_out[i0 + e * step] = count[e];
  }
  sync_all();
}

// The number of pages in [lo, hi) that are in use, the CTA's own share on its way copied to where the counts are wanted.
__device__ __forceinline__ int used_in(const PagesParams& p, int lo, int hi, bool copy, int* tmp) {
  int used = 0;
  for (int i0 = lo + threadIdx.x; i0 < hi; i0 += kTile) {
    int count[kEach];
#pragma unroll
    for (int e = 0; e < kEach; ++e) count[e] = i0 + e * kThreads < hi ? p.ref_counts[i0 + e * kThreads] : 0;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      used += count[e] != 0;
      if (copy && i0 + e * kThreads < hi) p.ref_counts_out[i0 + e * kThreads] = count[e];
    }
  }
  return block_sum(used, tmp);
}

__global__ void __launch_bounds__(kThreads)
    fork_kernel(const __grid_constant__ PagesParams p, const int32_t* parents, int b_out, int32_t* seq_lens_out) {
  begin();
  copy_counts(p);
  const int lane = threadIdx.x & 31;
  // The new rows, and the old ones, whose ownership ends.
  for_chunks(b_out + p.b, p.max_pages, [&](int x, int c0) {
    const bool is_new = x < b_out;
    const int j = is_new ? parents[x] : x - b_out, len = j >= 0 && j < p.b ? clamp_tokens(p.seq_lens, j, p.max_len) : 0;
    const int reach = columns_of(p, len);
    if (is_new && c0 == 0 && lane == 0) seq_lens_out[x] = len;
    int page[kChunk / 32];
#pragma unroll
    for (int k = 0; k < kChunk / 32; ++k) {
      const int c = c0 + lane + 32 * k;
      page[k] = c < reach ? p.page_table[j * p.table_stride + c] : -1;
    }
#pragma unroll
    for (int k = 0; k < kChunk / 32; ++k) {
      const int c = c0 + lane + 32 * k;
      if (is_page(page[k], p.num_pages)) atomicAdd(p.ref_counts_out + page[k], is_new ? 1 : -1);
      if (is_new && c < p.max_pages) p.page_table_out[x * p.table_out_stride + c] = page[k];
    }
  });
}

__global__ void __launch_bounds__(kThreads) free_kernel(const __grid_constant__ PagesParams p, const int32_t* keep_lens) {
  begin();
  copy_counts(p);
  const int lane = threadIdx.x & 31;
  const bool in_place = p.page_table_out == p.page_table;
  for_chunks(p.b, p.max_pages, [&](int i, int c0) {
    const int len = clamp_tokens(p.seq_lens, i, p.max_len), keep = min(len, max(0, keep_lens[i]));
    const int first = columns_of(p, keep), end = columns_of(p, len);
    int page[kChunk / 32];
#pragma unroll
    for (int k = 0; k < kChunk / 32; ++k) {
      const int c = c0 + lane + 32 * k;
      page[k] = c < p.max_pages && (!in_place || (c >= first && c < end)) ? p.page_table[i * p.table_stride + c] : -1;
    }
#pragma unroll
    for (int k = 0; k < kChunk / 32; ++k) {
      const int c = c0 + lane + 32 * k;
      const bool ends = c >= first && c < end;
      if (ends && is_page(page[k], p.num_pages)) atomicSub(p.ref_counts_out + page[k], 1);
      if (ends || (!in_place && c < p.max_pages)) p.page_table_out[i * p.table_out_stride + c] = ends ? -1 : page[k];
    }
  });
}

struct GrowShared {
  int tail[kMaxPageRows];       // the partly filled page to replace, or -1; -2 - page: it has other owners, but is kept
  int base[kMaxPageRows + 1];   // pages wanted by the rows before this one
  int tmp[kWarps];
  int free[kMaxCluster];        // free pages of each CTA's share
};

struct GrowRow {
  int tail;            // column of the partly filled page that is written on, or -1
  int first, end;      // columns to fill
};

__device__ __forceinline__ GrowRow grow_row(const PagesParams& p, const int32_t* new_lens, int i) {
  const int old_len = clamp_tokens(p.seq_lens, i, p.max_len), new_len = clamp_tokens(new_lens, i, p.max_len);
  GrowRow r;
  r.first = columns_of(p, old_len);
  r.end = max(r.first, columns_of(p, new_len));
  r.tail = new_len > old_len && r.first * static_cast<int64_t>(p.page_size) != old_len ? r.first - 1 : -1;
  return r;
}

__global__ void __launch_bounds__(kThreads)
    grow_kernel(const __grid_constant__ PagesParams p, const int32_t* new_lens, int32_t* src, int32_t* dst, int32_t* missing) {
  __shared__ GrowShared sh;
  meet();
  begin();
  const int tid = threadIdx.x, lane = tid & 31;
  // What is wanted elsewhere goes there as it is, before the barrier behind which it changes.
  if (p.page_table_out != p.page_table)
    for_chunks(p.b, p.max_pages, [&](int i, int c0) {
#pragma unroll
      for (int k = 0; k < kChunk / 32; ++k) {
        const int c = c0 + lane + 32 * k;
        if (c < p.max_pages) p.page_table_out[i * p.table_out_stride + c] = p.page_table[i * p.table_stride + c];
      }
    });
  const Range mine = share(p.num_pages, rank());
  const int free_count = mine.hi - mine.lo - used_in(p, mine.lo, mine.hi, p.ref_counts_out != p.ref_counts, sh.tmp);

  // Every CTA looks at all rows: their partly filled pages that others own too ...
  for (int i = tid; i < p.b; i += kThreads) {
    const GrowRow r = grow_row(p, new_lens, i);
    int page = r.tail >= 0 ? p.page_table[i * p.table_stride + r.tail] : -1;
    if (!is_page(page, p.num_pages) || p.ref_counts[page] <= 1) page = -1;
    sh.tail[i] = page;
  }
  __syncthreads();
  // ... of which, row after row, all but the last owner take a copy (each counts the rows before it that grow in its page: nothing for
  // most; all rows in one page take 8.6 us for 64, 23.8 for 1024, 188 for 4096, in pages of their own 4.9, 7.1 and 16.6), ...
  int wanted = 0;
  for (int i0 = 0; i0 < p.b; i0 += kThreads) {
    const int i = i0 + tid;
    int want = 0, total = 0;
    bool keeps = false;
    if (i < p.b) {
      const GrowRow r = grow_row(p, new_lens, i);
      const int page = sh.tail[i];
      want = r.end - r.first;
      if (page >= 0) {
        int before = 0;
        for (int j = 0; j < i; ++j) before += sh.tail[j] == page || sh.tail[j] == -2 - page;
        keeps = p.ref_counts[page] - before <= 1;
        want += !keeps;
      }
    }
    const int before = block_scan(want, sh.tmp, total);
    if (i < p.b) {
      sh.base[i] = wanted + before;
      if (keeps) sh.tail[i] = -2 - sh.tail[i];
    }
    wanted += total;
    __syncthreads();
  }
  if (tid == 0) sh.base[p.b] = wanted;
  // ... and how many pages that makes.  Behind the barrier the counts and the table may change.
  exchange(free_count, sh.free);
  const int there = lane < ranks() ? sh.free[lane] : 0;
  const int all = __reduce_add_sync(0xffffffffu, there);
  int before = __reduce_add_sync(0xffffffffu, lane < rank() ? there : 0);
  const bool granted = wanted <= all;
  if (rank() == 0 && tid == 0) *missing = granted ? 0 : wanted - all;

  for (int i = rank() * kThreads + tid; i < p.b; i += ranks() * kThreads) {
    const bool copied = granted && sh.tail[i] >= 0;
    src[i] = copied ? sh.tail[i] : -1;
    if (!copied) dst[i] = -1;
  }
  // The k-th free page goes to the row whose run of wanted pages holds k.
  if (!granted) return;
  for (int i0 = mine.lo; i0 < mine.hi && before < wanted; i0 += kTile) {
    int count[kEach], here = 0, total = 0;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int page = i0 + tid * kEach + e;
      count[e] = page < mine.hi ? p.ref_counts[page] : 1;
      here += count[e] == 0;
    }
    int k = before + block_scan(here, sh.tmp, total);
    before += total;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int page = i0 + tid * kEach + e;
      if (count[e] == 0 && k < wanted) {
        p.ref_counts_out[page] = 1;
        int lo = 0, hi = p.b;                    // base[lo] <= k < base[hi]
        while (hi - lo > 1) {
          const int mid = (lo + hi) / 2;
          if (sh.base[mid] <= k) lo = mid;
          else hi = mid;
        }
        const GrowRow r = grow_row(p, new_lens, lo);
        const int nth = k - sh.base[lo], copies = sh.tail[lo] >= 0;
        if (nth < copies) dst[lo] = page;
        p.page_table_out[lo * p.table_out_stride + (nth < copies ? r.tail : r.first + nth - copies)] = page;
      }
      k += count[e] == 0;
    }
  }
  sync_all();
  for (int i = rank() * kThreads + tid; i < p.b; i += ranks() * kThreads)
    if (sh.tail[i] >= 0) atomicSub(p.ref_counts_out + sh.tail[i], 1);
}

__global__ void __launch_bounds__(kThreads)
    compact_kernel(const __grid_constant__ PagesParams p, int32_t* src, int32_t* dst, int pairs) {
  __shared__ int tmp[kWarps], s_used[kMaxCluster];
  meet();
  begin();
  const int tid = threadIdx.x, lane = tid & 31;
  const Range mine = share(p.num_pages, rank());
  exchange(used_in(p, mine.lo, mine.hi, p.ref_counts_out != p.ref_counts, tmp), s_used);
  int n = 0;
  for (int k = 0; k < ranks(); ++k) n += s_used[k];
  // Every share lies before n or at and behind it, but for one, of which every CTA counts the part behind.
  int cut = 0;
  while (cut < ranks() - 1 && share(p.num_pages, cut).hi <= n) ++cut;
  const Range at_cut = share(p.num_pages, cut);
  const int cut_movers = used_in(p, max(n, at_cut.lo), at_cut.hi, false, tmp);
  int mover = rank() > cut ? cut_movers : 0, hole = 0, moves = cut_movers;
  for (int k = 0; k < ranks(); ++k) {
    const Range r = share(p.num_pages, k);
    if (k > cut) moves += s_used[k];
    if (k > cut && k < rank()) mover += s_used[k];
    if (k < cut && k < rank()) hole += r.hi - r.lo - s_used[k];
  }
  moves = min(moves, pairs);        // (as many holes as movers)
  for (int i0 = mine.lo; i0 < mine.hi; i0 += kTile) {
    int count[kEach], here = 0, total = 0;      // holes in the upper 16 bits, movers in the lower
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int i = i0 + tid * kEach + e;
      count[e] = i < mine.hi ? p.ref_counts[i] : 0;
      if (i < mine.hi) here += i >= n ? count[e] != 0 : (count[e] == 0) << 16;
    }
    const int before = block_scan(here, tmp, total);
    int m = mover + (before & 0xffff), h = hole + (before >> 16);
    mover += total & 0xffff;
    hole += total >> 16;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int i = i0 + tid * kEach + e;
      if (i >= mine.hi) break;
      const bool moved = i >= n && count[e] != 0, filled = i < n && count[e] == 0;
      if (moved && m < moves) src[m] = i;
      if (filled && h < moves) dst[h] = i;
      m += moved;
      h += filled;
    }
  }
  for (int64_t k = moves + rank() * kThreads + tid; k < pairs; k += ranks() * kThreads) src[k] = dst[k] = -1;
  sync_all();
  // Once both lists are written the counts move along.  Where a page was, its new name stands until the table has it:
  // one load an entry of the table (bisection of the list: 17 in a row, 156 us against 73 for 256 rows of 1024).
  for (int k = rank() * kThreads + tid; k < moves; k += ranks() * kThreads) {
    const int a = src[k], b = dst[k], count = p.ref_counts[a];
    p.ref_counts_out[b] = count;
    p.ref_counts_out[a] = -1 - b;
  }
  sync_all();
  const int last = moves ? src[moves - 1] : -1;
  const bool in_place = p.page_table_out == p.page_table;
  for_chunks(p.b, p.max_pages, [&](int i, int c0) {
    const int reach = columns_of(p, clamp_tokens(p.seq_lens, i, p.max_len));
    int page[kChunk / 32], name[kChunk / 32];
#pragma unroll
    for (int k = 0; k < kChunk / 32; ++k) {
      const int c = c0 + lane + 32 * k;
      page[k] = c < (in_place ? reach : p.max_pages) ? p.page_table[i * p.table_stride + c] : -1;
    }
#pragma unroll
    for (int k = 0; k < kChunk / 32; ++k)
      name[k] = c0 + lane + 32 * k < reach && page[k] >= n && page[k] <= last ? p.ref_counts_out[page[k]] : 0;
#pragma unroll
    for (int k = 0; k < kChunk / 32; ++k) {
      const int c = c0 + lane + 32 * k;
      if (name[k] < 0 || (!in_place && c < p.max_pages)) p.page_table_out[i * p.table_out_stride + c] = name[k] < 0 ? -1 - name[k] : page[k];
    }
  });
  if (!moves) return;
  sync_all();
  for (int k = rank() * kThreads + tid; k < moves; k += ranks() * kThreads) p.ref_counts_out[src[k]] = 0;
}

int64_t pieces_of(const PagesParams& p, int rows) { return static_cast<int64_t>(rows) * ((p.max_pages + kChunk - 1) / kChunk); }

// One CTA for what its 32 warps do in one go, 8 for more.
unsigned cluster_for(const PagesParams& p, int rows) {
  return pieces_of(p, rows) <= kWarps && p.num_pages <= 2 * kTile ? 1u : static_cast<unsigned>(kMaxCluster);
}

// Launched while the kernel before still runs; begin() waits for it.
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), unsigned grid, unsigned threads, bool cluster, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = grid;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster && grid > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ---- pages copied, rows kept ---------------------------------------------------------------

constexpr int kCopyThreads = 256;
constexpr int kCopyWarps = kCopyThreads / 32;
constexpr int kCopyEach = 8;                    // units of 16 bytes that a lane has in flight
constexpr int kCopyUnits = 32 * kCopyEach;      // of an item

// An item, a warp's: 4 KB of K, of V or of the scales of one pair of pages.  A page's units come in the order of memory: units
// of a row, rows of the inner dimension (slot or head, whichever stride is smaller), the outer one.  A warp looks at
// 32 of its items at once, so that pairs that are none cost next to nothing.  Bound: HBM; 660 pages of 262 KB moved in 50.3 us,
// 6.9 TB/s.  (Through shared memory by bulk copies, 4 to 32 KB each: 66 to 82 us against 57 then.)
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ CopyParams p, const int32_t* src,
                                                            const int32_t* dst, int64_t items) {
  begin();
  const int lane = threadIdx.x & 31;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kCopyWarps;
  // Neighbouring items lie on neighbouring SMs.
  for (int64_t first = static_cast<int64_t>(threadIdx.x / 32) * gridDim.x + blockIdx.x; first < items; first += 32 * step) {
    const int64_t mine = first + lane * step;
    int pair = 0, from = -1, to = -1;
    if (mine < items) {
      pair = static_cast<int>(mine / p.items_per_pair);
      from = src[pair];
      to = dst[pair];
    }
    const int mine_part = static_cast<int>(mine - static_cast<int64_t>(pair) * p.items_per_pair);
    uint32_t live = __ballot_sync(0xffffffffu, is_page(from, p.num_pages) && is_page(to, p.num_pages) && from != to);
    for (; live; live &= live - 1) {
      const int who = __ffs(live) - 1;
      const int part = __shfl_sync(0xffffffffu, mine_part, who);
      const int64_t a_page = __shfl_sync(0xffffffffu, from, who), b_page = __shfl_sync(0xffffffffu, to, who);
      const int t = part >= p.first_item[3] ? 3 : part >= p.first_item[2] ? 2 : part >= p.first_item[1] ? 1 : 0;
      const CopyTensor& x = p.t[t];
      const uint8_t* a = x.base + a_page * x.page;
      uint8_t* b = x.base + b_page * x.page;
      const int u0 = (part - p.first_item[t]) * kCopyUnits + lane;
      uint4 v[kCopyEach];
      int64_t at[kCopyEach];
#pragma unroll
      for (int k = 0; k < kCopyEach; ++k) {
        const int u = u0 + k * 32;
        if (u >= x.units) continue;
        if (x.flat) {
          at[k] = static_cast<int64_t>(u) * 16;
        } else {
          const int row = u / x.row_units, outer = row / x.inner_n;
          at[k] = outer * x.outer + (row - outer * x.inner_n) * x.inner + static_cast<int64_t>(u - row * x.row_units) * 16;
        }
        v[k] = *reinterpret_cast<const uint4*>(a + at[k]);
      }
#pragma unroll
      for (int k = 0; k < kCopyEach; ++k)
        if (u0 + k * 32 < x.units) *reinterpret_cast<uint4*>(b + at[k]) = v[k];
    }
  }
}

constexpr int kKeepEach = 4;

// A thread: 16 bytes of one head's rows of K or V of one sequence (or its scales), all kept rows in ascending order.
// path[j] >= j, and the kept rows ascend, so row j is written when nothing behind it reads it any more: four
// rows are read, then written.
__global__ void __launch_bounds__(128) keep_kernel(const __grid_constant__ KeepParams p) {
  begin();
  const int units = p.row_units + (p.c.k_scale ? 1 : 0), per = p.c.h_kv * units;
  const int i = blockIdx.x / p.blocks, idx = (blockIdx.x - i * p.blocks) * 128 + threadIdx.x;
  if (idx >= 2 * per) return;
  const int which = idx / per, at = idx % per, h = at / units, u = at % units;
  const int len_q = p.seq_lens_q ? min(max(p.seq_lens_q[i], 0), p.s) : p.s;
  const int len_kv = clamp_tokens(p.c.seq_lens_kv, i, p.c.max_len);
  const int n = min(min(max(p.accepted[i], 0), p.s), len_q), start = len_kv - len_q;
  const int64_t(&st)[3] = which ? p.c.v_st : p.c.k_st;
  uint8_t* base = which ? p.c.v : p.c.k;
  float* scale = which ? p.c.v_scale : p.c.k_scale;
  const bool is_scale = u == p.row_units;
  auto slot_of = [&](int row, int64_t& to) {
    const int pos = start + row;
    if (row < 0 || row >= len_q || pos < 0 || pos >= len_kv) return false;
    const int col = pos / p.c.page_size, page = p.c.page_table[i * p.c.page_table_stride + col], slot = pos - col * p.c.page_size;
    if (!is_page(page, p.c.num_pages)) return false;
    to = is_scale ? (static_cast<int64_t>(page) * p.c.h_kv + h) * p.c.page_size + slot : page * st[0] + h * st[1] + slot * st[2] + u * 16;
    return true;
  };
  for (int j0 = 0; j0 < n; j0 += kKeepEach) {
    uint4 v[kKeepEach];
    int64_t to[kKeepEach];
    bool on[kKeepEach];
#pragma unroll
    for (int k = 0; k < kKeepEach; ++k) {
      const int j = j0 + k;
      int64_t from = 0;
      const int row = j < n ? p.path[static_cast<int64_t>(i) * p.s + j] : j;
      on[k] = j < n && row != j && slot_of(row, from) && slot_of(j, to[k]);
      if (on[k]) {
        if (is_scale) v[k].x = __float_as_uint(scale[from]);
        else v[k] = *reinterpret_cast<const uint4*>(base + from);
      }
    }
#pragma unroll
    for (int k = 0; k < kKeepEach; ++k) {
      if (!on[k]) continue;
      if (is_scale) scale[to[k]] = __uint_as_float(v[k].x);
      else *reinterpret_cast<uint4*>(base + to[k]) = v[k];
    }
  }
}

}  // namespace

// Large tables of a call that only adds to counts: the counts are copied ahead, and the pieces of rows need no order.
static bool spread(PagesParams& p, int rows, int num_sms, unsigned& grid, cudaStream_t st, cudaError_t& e) {
  const int64_t pieces = pieces_of(p, rows);
  if (pieces <= kMaxCluster * kWarps) return false;
  if (p.ref_counts_out != p.ref_counts)
    e = cudaMemcpyAsync(p.ref_counts_out, p.ref_counts, static_cast<size_t>(p.num_pages) * 4, cudaMemcpyDeviceToDevice, st);
  p.ref_counts = p.ref_counts_out;
  const int64_t blocks = (pieces + kWarps - 1) / kWarps;
  grid = static_cast<unsigned>(blocks < num_sms ? blocks : num_sms);
  return true;
}

cudaError_t launch_fork(PagesParams p, const int32_t* parents, int b_out, int32_t* seq_lens_out, int num_sms, cudaStream_t st) {
  unsigned grid = cluster_for(p, p.b + b_out);
  cudaError_t e = cudaSuccess;
  const bool wide = spread(p, p.b + b_out, num_sms, grid, st, e);
  return e != cudaSuccess ? e : launch(fork_kernel, grid, kThreads, !wide, st, p, parents, b_out, seq_lens_out);
}

cudaError_t launch_free(PagesParams p, const int32_t* keep_lens, int num_sms, cudaStream_t st) {
  unsigned grid = cluster_for(p, p.b);
  cudaError_t e = cudaSuccess;
  const bool wide = spread(p, p.b, num_sms, grid, st, e);
  return e != cudaSuccess ? e : launch(free_kernel, grid, kThreads, !wide, st, p, keep_lens);
}

cudaError_t launch_grow(const PagesParams& p, const int32_t* new_lens, int32_t* src, int32_t* dst, int32_t* missing, cudaStream_t st) {
  return launch(grow_kernel, cluster_for(p, p.b), kThreads, true, st, p, new_lens, src, dst, missing);
}

cudaError_t launch_compact(const PagesParams& p, int32_t* src, int32_t* dst, int pairs, cudaStream_t st) {
  return launch(compact_kernel, cluster_for(p, p.b), kThreads, true, st, p, src, dst, pairs);
}

cudaError_t launch_copy(CopyParams p, const int32_t* src, const int32_t* dst, int pairs, int num_sms, cudaStream_t st) {
  for (int t = 0; t < 4; ++t) {
    CopyTensor& x = p.t[t];
    x.flat = x.inner == x.row_units * 16 && x.outer == x.inner * x.inner_n;
    p.first_item[t] = p.items_per_pair;
    p.items_per_pair += (x.units + kCopyUnits - 1) / kCopyUnits;
  }
  const int64_t items = static_cast<int64_t>(pairs) * p.items_per_pair, most = static_cast<int64_t>(num_sms) * 8;
  return launch(copy_kernel, static_cast<unsigned>(items < most ? items : most), kCopyThreads, false, st, p, src, dst, items);
}

cudaError_t launch_keep(KeepParams p, cudaStream_t st) {
  p.blocks = (2 * p.c.h_kv * (p.row_units + (p.c.k_scale ? 1 : 0)) + 127) / 128;
  const int64_t blocks = static_cast<int64_t>(p.blocks) * p.c.b;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  return launch(keep_kernel, static_cast<unsigned>(blocks), 128, false, st, p);
}

}  // namespace sdpa
