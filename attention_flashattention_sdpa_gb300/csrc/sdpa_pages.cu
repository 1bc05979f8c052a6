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
// cluster of 8 CTAs each, whose barrier stands between the passes that depend on each other (counts before
// ids, copies of counts before atomics on them), so that each is one launch and needs no workspace.  Atomics are
// sums of integers: their order changes nothing.
#include <type_traits>

#include "ptx.cuh"
#include "sdpa_internal.h"

namespace sdpa {
namespace {

constexpr int kThreads = 1024;
constexpr int kCluster = 8;
constexpr int kWarps = kThreads / 32;

// The CTA's share of n items in runs of kThreads * kEach, and this thread's number in the cluster.
__device__ __forceinline__ int cluster_rank() { return static_cast<int>(blockIdx.x); }
__device__ __forceinline__ int64_t cluster_thread() { return static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; }

struct Range {
  int lo, hi;
};

__device__ __forceinline__ Range share(int n) {
  const int per = (n + kCluster - 1) / kCluster;
  return {min(n, cluster_rank() * per), min(n, (cluster_rank() + 1) * per)};
}

// Exclusive prefix sum over the CTA's threads of x; the total in `total`.  `tmp`: kWarps + 1 words.
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
  if (warp == 0) {
    const int mine = tmp[lane];
    int w = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    tmp[lane] = w - mine;
    if (lane == 31) tmp[kWarps] = w;
  }
  __syncthreads();
  const int before = tmp[warp] + inc - x;
  total = tmp[kWarps];
  __syncthreads();
  return before;
}

__device__ __forceinline__ int clamp_tokens(const int32_t* lens, int i, int top) { return min(max(__ldg(lens + i), 0), top); }

__device__ __forceinline__ bool is_page(int page, int n) { return page >= 0 && page < n; }

// Word `at` of CTA `rank`'s shared memory.
__device__ __forceinline__ int ld_cluster(const int* at, int rank) {
  uint32_t a;
  int x;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(ptx::smem_u32(at)), "r"(rank));
  asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(x) : "r"(a) : "memory");
  return x;
}

// Counts as they are, where they are wanted elsewhere; the barrier before anyone adds to them.
__device__ __forceinline__ void copy_counts(const PagesParams& p) {
  if (p.ref_counts_out == p.ref_counts) return;
  for (int64_t i = cluster_thread(); i < p.num_pages; i += kCluster * kThreads) p.ref_counts_out[i] = p.ref_counts[i];
  ptx::cluster_sync_all();
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
    fork_kernel(const __grid_constant__ PagesParams p, const int32_t* parents, int b_out, int32_t* seq_lens_out) {
  copy_counts(p);
  // The new rows first, entry by entry, then the old ones' ownership ends.
  const int64_t made = static_cast<int64_t>(b_out) * p.max_pages, gone = static_cast<int64_t>(p.b) * p.max_pages;
  for (int64_t x = cluster_thread(); x < made + gone; x += kCluster * kThreads) {
    const bool is_new = x < made;
    const int64_t y = is_new ? x : x - made;
    const int i = static_cast<int>(y / p.max_pages), c = static_cast<int>(y - static_cast<int64_t>(i) * p.max_pages);
    const int j = is_new ? __ldg(parents + i) : i;
    const bool there = j >= 0 && j < p.b;
    const int len = there ? clamp_tokens(p.seq_lens, j, p.max_len) : 0;
    const int page = c * static_cast<int64_t>(p.page_size) < len ? __ldg(p.page_table + j * p.table_stride + c) : -1;
    if (is_page(page, p.num_pages)) atomicAdd(p.ref_counts_out + page, is_new ? 1 : -1);
    if (is_new) {
      p.page_table_out[i * p.table_out_stride + c] = page;
      if (c == 0) seq_lens_out[i] = len;
    }
  }
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
    free_kernel(const __grid_constant__ PagesParams p, const int32_t* keep_lens) {
  copy_counts(p);
  const int64_t n = static_cast<int64_t>(p.b) * p.max_pages;
  const bool in_place = p.page_table_out == p.page_table;
  for (int64_t x = cluster_thread(); x < n; x += kCluster * kThreads) {
    const int i = static_cast<int>(x / p.max_pages), c = static_cast<int>(x - static_cast<int64_t>(i) * p.max_pages);
    const int len = clamp_tokens(p.seq_lens, i, p.max_len), keep = min(len, max(0, __ldg(keep_lens + i)));
    const int64_t first = c * static_cast<int64_t>(p.page_size);
    const bool ends = first >= keep && first < len;
    if (in_place && !ends) continue;
    const int page = p.page_table[i * p.table_stride + c];
    if (ends && is_page(page, p.num_pages)) atomicSub(p.ref_counts_out + page, 1);
    p.page_table_out[i * p.table_out_stride + c] = ends ? -1 : page;
  }
}

// Rows of a grow that are looked at: their pages' order, and which page each copies.
struct GrowShared {
  int base[kMaxPageRows + 1];   // pages wanted by the rows before this one
  int tail[kMaxPageRows];       // a partly filled page that has other owners, or -1; -2 - page where it is kept after all
  int tmp[kWarps + 1];
  int free_here;
};

struct GrowRow {
  int tail;            // column of the partly filled page
  int first, end;      // columns to fill
};

__device__ __forceinline__ GrowRow grow_row(const PagesParams& p, const int32_t* new_lens, int i) {
  const int old_len = clamp_tokens(p.seq_lens, i, p.max_len), new_len = clamp_tokens(new_lens, i, p.max_len);
  GrowRow r;
  r.first = (old_len + p.page_size - 1) / p.page_size;
  r.end = max(r.first, (new_len + p.page_size - 1) / p.page_size);
  r.tail = new_len > old_len && old_len % p.page_size ? old_len / p.page_size : -1;
  return r;
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
    grow_kernel(const __grid_constant__ PagesParams p, const int32_t* new_lens, int32_t* src, int32_t* dst, int32_t* missing) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  GrowShared& sh = *reinterpret_cast<GrowShared*>(smem_raw);
  const int rank = cluster_rank(), tid = threadIdx.x;

  // Free pages of this CTA's share.
  const Range mine = share(p.num_pages);
  int free_count = 0, total = 0;
  for (int i = mine.lo + tid; i < mine.hi; i += kThreads) free_count += p.ref_counts[i] == 0;
  block_scan(free_count, sh.tmp, total);
  if (tid == 0) sh.free_here = total;

  // Every CTA looks at all rows: their partly filled pages that others own too ...
  for (int i = tid; i < p.b; i += kThreads) {
    const GrowRow r = grow_row(p, new_lens, i);
    int page = r.tail >= 0 ? p.page_table[i * p.table_stride + r.tail] : -1;
    if (!is_page(page, p.num_pages) || p.ref_counts[page] <= 1) page = -1;
    sh.tail[i] = page;
  }
  __syncthreads();
  // ... of which, row after row, all but the last owner take a copy, ...
  int row_base = 0;
  for (int i0 = 0; i0 < p.b; i0 += kThreads) {
    const int i = i0 + tid;
    int want = 0;
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
      sh.base[i] = row_base + before;
      if (keeps) sh.tail[i] = -2 - sh.tail[i];    // (still told from another page by the rows behind it)
    }
    row_base += total;
    __syncthreads();
  }
  if (tid == 0) sh.base[p.b] = row_base;
  // ... and how many pages that makes.  Behind the barrier the counts and the table may change.
  ptx::cluster_sync_all();
  int before = 0, all = 0;
  for (int k = 0; k < kCluster; ++k) {
    const int n = ld_cluster(&sh.free_here, k);
    before += k < rank ? n : 0;
    all += n;
  }
  const bool granted = row_base <= all;
  if (rank == 0 && tid == 0) *missing = granted ? 0 : row_base - all;

  // Entries that stay as they are.
  if (p.page_table_out != p.page_table) {
    const int64_t n = static_cast<int64_t>(p.b) * p.max_pages;
    for (int64_t x = cluster_thread(); x < n; x += kCluster * kThreads) {
      const int i = static_cast<int>(x / p.max_pages), c = static_cast<int>(x - static_cast<int64_t>(i) * p.max_pages);
      const GrowRow r = grow_row(p, new_lens, i);
      const bool filled = (c >= r.first && c < r.end) || (c == r.tail && sh.tail[i] >= 0);
      if (!(granted && filled)) p.page_table_out[i * p.table_out_stride + c] = p.page_table[i * p.table_stride + c];
    }
  }
  for (int i = static_cast<int>(cluster_thread()); i < p.b; i += kCluster * kThreads) {
    const bool copied = granted && sh.tail[i] >= 0;
    src[i] = copied ? sh.tail[i] : -1;
    if (!copied) dst[i] = -1;
  }
  // The k-th free page goes to the row whose run of wanted pages holds k.
  const bool elsewhere = p.ref_counts_out != p.ref_counts;
  for (int i0 = mine.lo; i0 < mine.hi; i0 += kThreads) {
    if (!elsewhere && (!granted || before >= row_base)) break;
    const int page = i0 + tid;
    const int count = page < mine.hi ? p.ref_counts[page] : 1;
    const int k = before + block_scan(count == 0, sh.tmp, total);
    before += total;
    const bool given = granted && count == 0 && k < row_base;
    if (page < mine.hi && (elsewhere || given)) p.ref_counts_out[page] = given ? 1 : count;
    if (!given) continue;
    int lo = 0, hi = p.b;                        // base[lo] <= k < base[hi]
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
  // (Also what keeps every CTA here while its words are read.)
  ptx::cluster_sync_all();
  for (int i = static_cast<int>(cluster_thread()); i < p.b; i += kCluster * kThreads)
    if (granted && sh.tail[i] >= 0) atomicSub(p.ref_counts_out + sh.tail[i], 1);
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
    compact_plan_kernel(const __grid_constant__ PagesParams p, int32_t* src, int32_t* dst, int pairs) {
  __shared__ int tmp[kWarps + 1], s_used, s_movers, s_holes;
  const int rank = cluster_rank(), tid = threadIdx.x;
  const Range mine = share(p.num_pages);
  int used = 0, total = 0;
  for (int i = mine.lo + tid; i < mine.hi; i += kThreads) used += p.ref_counts[i] != 0;
  block_scan(used, tmp, total);
  if (tid == 0) s_used = total;
  ptx::cluster_sync_all();
  int n = 0;
  for (int k = 0; k < kCluster; ++k) n += ld_cluster(&s_used, k);
  int movers = 0, holes = 0;
  for (int i = mine.lo + tid; i < mine.hi; i += kThreads) {
    const bool in_use = p.ref_counts[i] != 0;
    movers += in_use && i >= n;
    holes += !in_use && i < n;
  }
  block_scan(movers, tmp, total);
  if (tid == 0) s_movers = total;
  block_scan(holes, tmp, total);
  if (tid == 0) s_holes = total;
  ptx::cluster_sync_all();
  int mover0 = 0, hole0 = 0, moves = 0;
  for (int k = 0; k < kCluster; ++k) {
    const int m = ld_cluster(&s_movers, k), h = ld_cluster(&s_holes, k);
    mover0 += k < rank ? m : 0;
    hole0 += k < rank ? h : 0;
    moves += m;
  }
  moves = min(moves, pairs);        // (as many holes as movers)
  const bool elsewhere = p.ref_counts_out != p.ref_counts;
  for (int i0 = mine.lo; i0 < mine.hi; i0 += kThreads) {
    const int i = i0 + tid;
    const int count = i < mine.hi ? p.ref_counts[i] : 0;
    const bool mover = i < mine.hi && count != 0 && i >= n, hole = i < mine.hi && count == 0 && i < n;
    // (A share lies on one side of n, but for the one that n cuts: one scan serves both but there.)
    const int m = mover0 + block_scan(mover, tmp, total);
    mover0 += total;
    const int h = hole0 + block_scan(hole, tmp, total);
    hole0 += total;
    if (mover && m < moves) src[m] = i;
    if (hole && h < moves) dst[h] = i;
    if (elsewhere && i < mine.hi && !(mover && m < moves) && !(hole && h < moves)) p.ref_counts_out[i] = count;
  }
  for (int64_t k = moves + cluster_thread(); k < pairs; k += kCluster * kThreads) src[k] = dst[k] = -1;
  ptx::cluster_sync_all();
  // The counts move along, once both lists are written.
  for (int64_t k = cluster_thread(); k < moves; k += kCluster * kThreads) {
    const int a = src[k], b = dst[k], count = p.ref_counts[a];
    p.ref_counts_out[b] = count;
    p.ref_counts_out[a] = 0;
  }
}

// Names in the table: src is in ascending order, so a page's new one is found by bisection.
__global__ void __launch_bounds__(256) compact_rename_kernel(const __grid_constant__ PagesParams p, const int32_t* src,
                                                             const int32_t* dst, int pairs) {
  const int64_t n = static_cast<int64_t>(p.b) * p.max_pages;
  const bool in_place = p.page_table_out == p.page_table;
  const int64_t x = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (x >= n) return;
  const int i = static_cast<int>(x / p.max_pages), c = static_cast<int>(x - static_cast<int64_t>(i) * p.max_pages);
  const bool reached = c * static_cast<int64_t>(p.page_size) < clamp_tokens(p.seq_lens, i, p.max_len);
  if (in_place && !reached) return;
  const int old_page = p.page_table[i * p.table_stride + c];
  int page = old_page;
  if (reached && is_page(page, p.num_pages)) {
    int lo = 0, hi = pairs;                    // the first entry that is -1 or at least the page
    while (lo < hi) {
      const int mid = (lo + hi) / 2, at = __ldg(src + mid);
      if (at >= 0 && at < page) lo = mid + 1;
      else hi = mid;
    }
    if (lo < pairs && __ldg(src + lo) == page) page = __ldg(dst + lo);
  }
  if (!in_place || page != old_page) p.page_table_out[i * p.table_out_stride + c] = page;
}

// ---- pages copied, rows kept ---------------------------------------------------------------

constexpr int kCopyThreads = 256;
constexpr int kCopyEach = 4;                                  // 16-byte units a thread has in flight
constexpr int kCopyUnits = kCopyThreads * kCopyEach;

// One item: kCopyUnits units of 16 bytes of K, of V or of the scales of one pair of pages.  A page's units in the
// order of memory: units of a row, rows of the inner dimension (slot or head, whichever stride is smaller), the
// outer one.
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ CopyParams p, const int32_t* src,
                                                            const int32_t* dst, int64_t items) {
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int pair = static_cast<int>(item / p.items_per_pair);
    const int from = __ldg(src + pair), to = __ldg(dst + pair);
    if (!is_page(from, p.num_pages) || !is_page(to, p.num_pages) || from == to) continue;
    const int part = static_cast<int>(item - static_cast<int64_t>(pair) * p.items_per_pair);
    const int t = part >= p.first_item[3] ? 3 : part >= p.first_item[2] ? 2 : part >= p.first_item[1] ? 1 : 0;
    const CopyTensor& x = p.t[t];
    const uint8_t* a = x.base + from * x.page;
    uint8_t* b = x.base + to * x.page;
    const int u0 = (part - p.first_item[t]) * kCopyUnits + threadIdx.x;
    uint4 v[kCopyEach];
    int64_t at[kCopyEach];
#pragma unroll
    for (int k = 0; k < kCopyEach; ++k) {
      const int u = u0 + k * kCopyThreads;
      if (u >= x.units) continue;
      const int row = u / x.row_units, outer = row / x.inner_n;
      at[k] = outer * x.outer + (row - outer * x.inner_n) * x.inner + static_cast<int64_t>(u - row * x.row_units) * 16;
      v[k] = *reinterpret_cast<const uint4*>(a + at[k]);
    }
#pragma unroll
    for (int k = 0; k < kCopyEach; ++k)
      if (u0 + k * kCopyThreads < x.units) *reinterpret_cast<uint4*>(b + at[k]) = v[k];
  }
}

constexpr int kKeepEach = 8;

// A thread: 16 bytes of one head's rows of K or V of one sequence (or its scales), all kept rows in ascending order.
// path[j] >= j, and the kept rows ascend, so row j is written when nothing behind it reads it any more: eight
// rows are read, then written.
__global__ void __launch_bounds__(128) keep_kernel(const __grid_constant__ KeepParams p) {
  const int units = p.row_units + (p.c.k_scale ? 1 : 0), per = p.c.h_kv * units;
  const int i = blockIdx.x / p.blocks, idx = (blockIdx.x - i * p.blocks) * 128 + threadIdx.x;
  if (idx >= 2 * per) return;
  const int which = idx / per, at = idx % per, h = at / units, u = at % units;
  const int len_q = p.seq_lens_q ? min(max(__ldg(p.seq_lens_q + i), 0), p.s) : p.s;
  const int len_kv = clamp_tokens(p.c.seq_lens_kv, i, p.c.max_len);
  const int n = min(min(max(__ldg(p.accepted + i), 0), p.s), len_q), start = len_kv - len_q;
  const int64_t(&st)[3] = which ? p.c.v_st : p.c.k_st;
  uint8_t* base = which ? p.c.v : p.c.k;
  float* scale = which ? p.c.v_scale : p.c.k_scale;
  const bool is_scale = u == p.row_units;
  auto slot_of = [&](int row, int64_t& to) {
    const int pos = start + row;
    if (row < 0 || row >= len_q || pos < 0 || pos >= len_kv) return false;
    const int col = pos / p.c.page_size, page = __ldg(p.c.page_table + i * p.c.page_table_stride + col), slot = pos - col * p.c.page_size;
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
      const int row = j < n ? __ldg(p.path + static_cast<int64_t>(i) * p.s + j) : j;
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

cudaError_t launch_fork(const PagesParams& p, const int32_t* parents, int b_out, int32_t* seq_lens_out, cudaStream_t st) {
  fork_kernel<<<kCluster, kThreads, 0, st>>>(p, parents, b_out, seq_lens_out);
  return cudaGetLastError();
}

cudaError_t launch_free(const PagesParams& p, const int32_t* keep_lens, cudaStream_t st) {
  free_kernel<<<kCluster, kThreads, 0, st>>>(p, keep_lens);
  return cudaGetLastError();
}

cudaError_t launch_grow(const PagesParams& p, const int32_t* new_lens, int32_t* src, int32_t* dst, int32_t* missing, cudaStream_t st) {
  grow_kernel<<<kCluster, kThreads, sizeof(GrowShared), st>>>(p, new_lens, src, dst, missing);
  return cudaGetLastError();
}

cudaError_t launch_compact(const PagesParams& p, int32_t* src, int32_t* dst, int pairs, cudaStream_t st) {
  compact_plan_kernel<<<kCluster, kThreads, 0, st>>>(p, src, dst, pairs);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t blocks = (static_cast<int64_t>(p.b) * p.max_pages + 255) / 256;
  compact_rename_kernel<<<static_cast<unsigned>(blocks), 256, 0, st>>>(p, src, dst, pairs);
  return cudaGetLastError();
}

cudaError_t launch_copy(CopyParams p, const int32_t* src, const int32_t* dst, int pairs, int num_sms, cudaStream_t st) {
  for (int t = 0; t < 4; ++t) {
    p.first_item[t] = p.items_per_pair;
    p.items_per_pair += (p.t[t].units + kCopyUnits - 1) / kCopyUnits;
  }
  const int64_t items = static_cast<int64_t>(pairs) * p.items_per_pair, most = static_cast<int64_t>(num_sms) * 8;
  copy_kernel<<<static_cast<unsigned>(items < most ? items : most), kCopyThreads, 0, st>>>(p, src, dst, items);
  return cudaGetLastError();
}

cudaError_t launch_keep(KeepParams p, cudaStream_t st) {
  p.blocks = (2 * p.c.h_kv * (p.row_units + (p.c.k_scale ? 1 : 0)) + 127) / 128;
  const int64_t blocks = static_cast<int64_t>(p.blocks) * p.c.b;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  keep_kernel<<<static_cast<unsigned>(blocks), 128, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace sdpa
