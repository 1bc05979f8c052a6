// sdpa_verify.cu — drafted tokens verified against the target's probabilities.
//
// Rows are nodes of a tree: row 0 the newest token that is decided, row i > 0 a drafted token behind row
// parents[i] < i (a chain: i - 1).  p_n is the target's distribution behind row n.  From row 0 on, the children
// of the accepted node n are tried in ascending order: child i with token x is accepted iff
//   u_i q_i(x) < p_n(x)                          with the draft's probabilities q (a chain), or
//   u_i max(0, 1 - sum of p_n(x') over the refused siblings' tokens x') < p_n(x)      without.
// Behind the last accepted node a token is drawn from max(p_n - q_i, 0) of the refused child i, or from p_n
// without its children's tokens, by its cumulative sum and u_0.  So the tokens are distributed as the
// target's own, whatever was drafted.
//
// Masses are whole numbers of 2^-42: sums do not depend on their order, and the drawn token on nothing
// but the inputs (fp32 sums of a vocabulary are off by 10^-6 and differ with the split).
//
// Bound: reading one row of p (and one of q) of each sequence.  The tests need a few single values, which a
// thread each fetches at once; a cluster of CTAs shares a row, sums meet in its shared memory, and the CTA
// that the drawn number falls into reads the piece of the row once more, from L2.  Measured (replayed): 64 rows of 131072 fp32
// values of p and q 16.0 us from HBM (3.7 TB/s), 10.5 from L2; one of 32000 5.4: the launch, and five latencies in a row
// (tokens, their probabilities, the row, the cluster's barrier, the piece), which the stream waits for; without q the random
// numbers of the tests are one more, behind the probabilities.  Rows of q lie at another offset from 16 bytes than p's where the vocabulary is
// no multiple of a vector, and come element by element then: 64 rows of 131073 16.5 us (BF16 15.3, of 131072 12.2).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "ptx.cuh"
#include "sdpa_internal.h"

namespace sdpa {
namespace {

constexpr int kMaxCluster = 8;
constexpr int kMaxWarps = 16;
// Vectors a thread has in flight: of one row (2: 64 rows of 131072 12.6 us, 4: 11.6), and of each of two (4: 16.6 us, 2: 16.0).
constexpr int kAheadOne = 4, kAheadTwo = 2;
constexpr float kUnit = 4398046511104.f;       // 2^42
constexpr int kMaxSteps = 520;                 // steps of 32 vectors in a warp's piece: at most 2^20 / 4 / (2 * 8) / 32, and what rounds up

template <typename T>
__device__ __forceinline__ float widen(T x) {
  return static_cast<float>(x);
}

// 16 bytes of a row as they lie there, and as values.
template <typename T>
struct Vec {
  static constexpr int N = 16 / sizeof(T);
  float x[N];
};

template <typename T>
__device__ __forceinline__ Vec<T> unpack(const uint4& u) {
  const T* e = reinterpret_cast<const T*>(&u);
  Vec<T> v;
#pragma unroll
  for (int i = 0; i < Vec<T>::N; ++i) v.x[i] = widen(e[i]);
  return v;
}

// Elements [first, first + N) of a row of n one by one; those outside are 0.
template <typename T>
__device__ __forceinline__ Vec<T> load_each(const T* row, int first, int n) {
  Vec<T> v;
#pragma unroll
  for (int i = 0; i < Vec<T>::N; ++i) v.x[i] = first + i >= 0 && first + i < n ? widen(row[first + i]) : 0.f;
  return v;
}

// A mass p 2^42 as h 2^22 + l: h = floor(p 2^20), and l = p 2^42 - h 2^22 rounded to the nearest (ties to even, as for the
// sum of both: h 2^22 is even).  Both are the last bits of fp32 sums with 2^23, at the rate of fp32 arithmetic, two
// elements an instruction (a conversion to 64 bits has the rate of fp64: 31 us against 19 for 64 rows of 131072 then).
// Sums of 2^9 to 2^10 of either fit 32 bits.
constexpr uint32_t kBits = 0x4B000000u;        // of 2^23

__device__ __forceinline__ float2 fma2_rz(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rz.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
  return d;
}

struct Masses {
  uint32_t h0, h1, l0, l1;      // of two elements, each kBits too large
};

// NaN and what is below zero counts nothing, what is above one counts one.
__device__ __forceinline__ Masses masses_of(float p0, float p1) {
  const float2 x = make_float2(__saturatef(p0), __saturatef(p1)), big = make_float2(8388608.f, 8388608.f);
  const float2 two20 = make_float2(1048576.f, 1048576.f), top = fma2_rz(x, two20, big);
  const float2 floors = ptx::fma2(top, make_float2(-1.f, -1.f), big);
  const float2 low = ptx::fma2(ptx::fma2(x, two20, floors), make_float2(4194304.f, 4194304.f), big);
  return {__float_as_uint(top.x), __float_as_uint(top.y), __float_as_uint(low.x), __float_as_uint(low.y)};
}

__device__ __forceinline__ long long mass_of(float p) {
  const Masses m = masses_of(p, 0.f);
  return (static_cast<long long>(m.h0 - kBits) << 22) + (m.l0 - kBits);
}

__device__ __forceinline__ long long warp_sum(long long x) {
#pragma unroll
  for (int o = 16; o > 0; o /= 2) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Inclusive sum over the lanes up to this one.
__device__ __forceinline__ long long warp_scan(long long x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

__device__ __forceinline__ void st_cluster(long long* at, int rank, long long x) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(ptx::smem_u32(at)), "r"(rank));
  asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(a), "l"(x) : "memory");
}

// Of n <= 32 masses (lane i has the i-th) the one that target falls into; target becomes its place in that one.
__device__ __forceinline__ int pick(long long mass, int n, long long& target, int lane) {
  const long long to = warp_scan(lane < n ? mass : 0, lane);
  const int k = min(n - 1, __popc(__ballot_sync(0xffffffffu, lane < n && to <= target)));
  const long long before = __shfl_sync(0xffffffffu, to - mass, k);
  target -= before;
  return k;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// What a CTA knows of its sequence's rows, s entries each.
struct Rows {
  long long* mass;          // of each drafted token behind its parent (0 where an earlier sibling has it too)
  long long* gone_mass;
  int32_t* gone;            // tokens that are not drawn any more
  int32_t* parent;          // -1: not a node
  int32_t* token;
  int32_t* path;
  uint8_t* good;
};

constexpr int kRowBytes = 2 * 8 + 4 * 4 + 1;

__device__ __forceinline__ Rows rows_at(uint8_t* smem, int s) {
  Rows r;
  r.mass = reinterpret_cast<long long*>(smem);
  r.gone_mass = r.mass + s;
  r.gone = reinterpret_cast<int32_t*>(r.gone_mass + s);
  r.parent = r.gone + s;
  r.token = r.parent + s;
  r.path = r.token + s;
  r.good = reinterpret_cast<uint8_t*>(r.path + s);
  return r;
}

struct Sums {
  int accepted, refused, n_gone;    // refused: the row of the refused draft of a chain, or -1
  long long warp[kMaxWarps];
  long long cta[2][kMaxCluster];    // of every CTA of the cluster, in each turn
  long long step[kMaxSteps];
};

// Which rows are accepted: r.path, sh.accepted; what may not be drawn: sh.refused (a chain with q), r.gone.
template <typename T, int THREADS>
__device__ void walk(const VerifyParams& p, const Rows& r, Sums& sh, int bi, int len) {
  const int tid = threadIdx.x;
  const T* probs = static_cast<const T*>(p.probs) + bi * p.probs_b;
  const T* draft = static_cast<const T*>(p.draft) + bi * p.draft_b;
  const int64_t at = static_cast<int64_t>(bi) * p.s;
  if (tid == 0) {
    sh.accepted = len;
    sh.n_gone = 0;
  }
  for (int j = tid; j < len; j += THREADS) {
    const int x = p.tokens[at + j];
    const int par = j == 0 ? -1 : p.parents ? p.parents[at + j] : j - 1;
    const bool node = j > 0 && par >= 0 && par < j, known = node && x >= 0 && x < p.vocab;
    const float pr = known ? widen(probs[par * p.probs_s + x]) : 0.f;
    r.token[j] = x;
    r.parent[j] = node ? par : -1;
    r.mass[j] = mass_of(pr);
    if (p.draft) {
      const float q = known ? widen(draft[j * p.draft_s + x]) : 0.f;
      // The product of two fp32 values is exact in fp64.
      r.good[j] = j == 0 || (known && static_cast<double>(p.uniform[at + j]) * q < static_cast<double>(pr));
    }
  }
  __syncthreads();
  if (!p.parents) {
    // A chain: up to the first that is not accepted.
    for (int j = tid; j < len; j += THREADS) {
      bool good = j == 0;
      if (j > 0) good = p.draft ? r.good[j] : p.uniform[at + j] * static_cast<double>(kUnit) < static_cast<double>(r.mass[j]);
      if (!good) atomicMin(&sh.accepted, j);
    }
    __syncthreads();
    const int n = sh.accepted;
    for (int j = tid; j < n; j += THREADS) r.path[j] = j;
    if (tid == 0) {
      sh.refused = p.draft && n < len ? n : -1;
      if (!p.draft && n < len) {
        r.gone[0] = r.token[n];
        r.gone_mass[0] = r.mass[n];
        sh.n_gone = 1;
      }
    }
    __syncthreads();
    return;
  }
  // A tree.  A token that an earlier sibling has counts nothing.
  bool twin[kVerifyRows / THREADS];
#pragma unroll
  for (int k = 0; k < kVerifyRows / THREADS; ++k) {
    const int j = tid + k * THREADS;
    twin[k] = false;
    if (j < len && r.parent[j] >= 0)
      for (int i = r.parent[j] + 1; i < j; ++i) twin[k] |= r.parent[i] == r.parent[j] && r.token[i] == r.token[j];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kVerifyRows / THREADS; ++k)
    if (twin[k]) r.mass[tid + k * THREADS] = 0;
  __syncthreads();
  for (int j = tid; j < len; j += THREADS) {
    long long left = static_cast<long long>(kUnit);
    if (r.parent[j] >= 0)
      for (int i = r.parent[j] + 1; i < j; ++i) left -= r.parent[i] == r.parent[j] ? r.mass[i] : 0;
    if (left < 0) left = 0;
    r.good[j] = r.parent[j] >= 0 && __dmul_rn(static_cast<double>(p.uniform[at + j]), static_cast<double>(left)) <
                                          static_cast<double>(r.mass[j]);
  }
  __syncthreads();
  if (tid < 32) {
    // From node to node: the first good child, all of them behind it.
    int n = 0, count = 1;
    if (tid == 0) r.path[0] = 0;
    for (int j0 = 1; j0 < len;) {
      const int j = j0 + tid;
      const uint32_t hit = __ballot_sync(0xffffffffu, j < len && r.parent[j] == n && r.good[j]);
      if (hit) {
        n = j0 + __ffs(hit) - 1;
        if (tid == 0) r.path[count] = n;
        ++count;
        j0 = n + 1;
      } else {
        j0 += 32;
      }
    }
    int gone = 0;
    for (int j0 = n + 1; j0 < len; j0 += 32) {
      const int j = j0 + tid;
      const bool child = j < len && r.parent[j] == n;
      const uint32_t hit = __ballot_sync(0xffffffffu, child);
      if (child) {
        const int k = gone + __popc(hit & ((1u << tid) - 1));
        r.gone[k] = r.token[j];
        r.gone_mass[k] = r.mass[j];
      }
      gone += __popc(hit);
    }
    if (tid == 0) {
      sh.accepted = count;
      sh.refused = -1;
      sh.n_gone = gone;
    }
  }
  __syncthreads();
}

template <typename T, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) verify_kernel(const __grid_constant__ VerifyParams p, int cluster) {
  constexpr int N = Vec<T>::N, WARPS = THREADS / 32;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ Sums sh;
  const Rows r = rows_at(smem_raw, p.s);
  const int bi = blockIdx.x / cluster, rank = blockIdx.x - bi * cluster;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  cluster_arrive();
  // The kernel before is done (and the next one may be put in place, to wait here in its turn).  It may have written anything that is
  // read below while this one was already there: plain loads, which stay behind the wait.
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int len = p.seq_lens_q ? min(max(p.seq_lens_q[bi], 0), p.s) : p.s;
  const int64_t at = static_cast<int64_t>(bi) * p.s;
  const float u0 = p.uniform[at];
  if (len > 0) walk<T, THREADS>(p, r, sh, bi, len);
  const int accepted = len > 0 ? sh.accepted : 0;
  // Behind the new token there is none; the token itself is written by the CTA that finds it.
  if (rank == 0) {
    if (tid == 0) p.accepted[bi] = accepted;
    for (int j = tid; j < p.s; j += THREADS) {
      p.path[at + j] = j < accepted ? r.path[j] : -1;
      if (j != accepted - 1) p.new_tokens[at + j] = j < accepted ? r.token[r.path[j + 1]] : -1;
    }
  }
  if (len == 0) {             // (the whole cluster)
    cluster_wait();
    return;
  }

  const int last = r.path[accepted - 1], refused = sh.refused;
  const T* row = static_cast<const T*>(p.probs) + bi * p.probs_b + last * p.probs_s;
  const T* less = refused >= 0 ? static_cast<const T*>(p.draft) + bi * p.draft_b + refused * p.draft_s : nullptr;
  // Vectors of 16 bytes from the multiple of 16 at or before the row's start; each warp has a piece of them.
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(row) % 16 / sizeof(T));
  const bool less_wide = less && reinterpret_cast<uintptr_t>(less) % 16 / sizeof(T) == static_cast<unsigned>(off);
  const int vectors = (off + p.vocab + N - 1) / N, pieces = cluster * WARPS, per = (vectors + pieces - 1) / pieces;
  // (Vectors 0 and `inner` may hold elements that are not the row's.)
  const int inner = (off + p.vocab) / N, inner0 = off ? 1 : 0;
  auto value = [&](int v, bool diff) {
    const int first = v * N - off;
    Vec<T> x = v >= inner0 && v < inner ? unpack<T>(*reinterpret_cast<const uint4*>(row + first)) : load_each(row, first, p.vocab);
    if (diff) {
      const Vec<T> y = load_each(less, first, p.vocab);
#pragma unroll
      for (int e = 0; e < N; ++e) x.x[e] -= y.x[e];
    }
    return x;
  };

  // What is left of the distribution first; where that is nothing, the distribution.
  bool diff = less != nullptr;
  int n_gone = sh.n_gone;
  const int piece = rank * WARPS + warp, v_lo = min(vectors, piece * per), v_hi = min(vectors, v_lo + per);
  long long total = 0, target = 0;
  for (int turn = 0; turn < 2; ++turn) {
    long long sum = 0;
    uint32_t h = 0, l = 0, n = 0;
    auto flush = [&] {
      sum += (static_cast<long long>(h - n * kBits) << 22) + (l - n * kBits);
      h = l = n = 0;
    };
    auto add = [&](const Vec<T>& x) {
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        const Masses m = masses_of(x.x[e], x.x[e + 1]);
        h += m.h0 + m.h1;
        l += m.l0 + m.l1;
      }
      n += N;
    };
    // Whole vectors, several of them loaded at once; MODE 0: the row, 1: less another row as aligned as it is, 2: less any other.
    auto stream = [&](auto mode) {
      constexpr int MODE = decltype(mode)::value;
      const int hi = min(v_hi, inner);
      int v = max(v_lo, inner0) + lane;
      auto some = [&](auto count) {
        constexpr int COUNT = decltype(count)::value;
        uint4 a[COUNT], b[COUNT];
        Vec<T> c[COUNT];
#pragma unroll
        for (int k = 0; k < COUNT; ++k) {
          const int first = (v + 32 * k) * N - off;
          a[k] = *reinterpret_cast<const uint4*>(row + first);
          if constexpr (MODE == 1) b[k] = *reinterpret_cast<const uint4*>(less + first);
          if constexpr (MODE == 2) {
#pragma unroll
            for (int e = 0; e < N; ++e) c[k].x[e] = widen(less[first + e]);      // (all of them are the row's)
          }
        }
#pragma unroll
        for (int k = 0; k < COUNT; ++k) {
          Vec<T> x = unpack<T>(a[k]);
          if constexpr (MODE == 1) c[k] = unpack<T>(b[k]);
#pragma unroll
          for (int e = 0; e < N; ++e)
            if constexpr (MODE != 0) x.x[e] -= c[k].x[e];
          add(x);
        }
        if (n > 512) flush();
      };
      constexpr int AHEAD = MODE == 0 ? kAheadOne : kAheadTwo;
      for (; v + 32 * (AHEAD - 1) < hi; v += 32 * AHEAD) some(std::integral_constant<int, AHEAD>());
      for (; v < hi; v += 32) some(std::integral_constant<int, 1>());
    };
    if (!diff) stream(std::integral_constant<int, 0>());
    else if (less_wide) stream(std::integral_constant<int, 1>());
    else stream(std::integral_constant<int, 2>());
    if (lane == 0 && inner0 > 0 && v_lo == 0 && v_hi > 0) add(value(0, diff));
    if (lane == 0 && inner >= max(v_lo, inner0) && inner < v_hi) add(value(inner, diff));
    flush();
    for (int g = lane; g < n_gone; g += 32)
      if (r.gone_mass[g] > 0) {
        const int v = (r.gone[g] + off) / N;
        if (v >= v_lo && v < v_hi) sum -= r.gone_mass[g];
      }
    sum = warp_sum(sum);
    if (lane == 0) sh.warp[warp] = sum;
    __syncthreads();
    if (warp == 0) {
      // The CTA's sum goes to every CTA of the cluster.
      const long long all = warp_sum(lane < WARPS ? sh.warp[lane] : 0);
      if (turn == 0) cluster_wait();           // they have all begun
      if (lane < cluster) st_cluster(&sh.cta[turn][rank], lane, all);
    } else if (turn == 0) {
      cluster_wait();
    }
    ptx::cluster_sync_all();
    const long long mine = lane < cluster ? sh.cta[turn][lane] : 0;
    total = warp_sum(mine);
    // floor(u 2^31) total / 2^31: below the total.
    const unsigned long long part = min(__float2uint_rd(u0 * 2147483648.f), 0x7fffffffu), all = total;
    target = static_cast<long long>((all >> 32) * part * 2 + (((all & 0xffffffffull) * part) >> 31));
    if (total > 0) {
      if (pick(mine, cluster, target, lane) != rank) return;
      break;
    }
    if (!diff && n_gone == 0) break;
    diff = false;
    n_gone = 0;
  }
  int32_t* out = p.new_tokens + at + accepted - 1;
  if (total == 0) {
    if (rank == 0 && tid == 0) *out = -1;
    return;
  }
  const int w = pick(lane < WARPS ? sh.warp[lane] : 0, WARPS, target, lane);
  // The piece of warp w once more, a step of 32 vectors a warp.
  const int lo = min(vectors, (rank * WARPS + w) * per), hi = min(vectors, lo + per), steps = (hi - lo + 31) / 32;
  auto left_of = [&](int v, long long (&mass)[N]) {
    long long sum = 0;
    if (v < hi) {
      const Vec<T> x = value(v, diff);
#pragma unroll
      for (int e = 0; e < N; ++e) mass[e] = mass_of(x.x[e]);
      for (int g = 0; g < n_gone; ++g) {
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (r.gone[g] == v * N - off + e) mass[e] = 0;
      }
#pragma unroll
      for (int e = 0; e < N; ++e) sum += mass[e];
    }
    return sum;
  };
  long long mass[N], sum = 0;
  int k = warp;
  for (; k < steps; k += WARPS) {
    sum = left_of(lo + 32 * k + lane, mass);
    const long long all = warp_sum(sum);
    if (lane == 0) sh.step[k] = all;
  }
  __syncthreads();
  int step = 0;
  for (int k0 = 0; k0 < steps; k0 += 32) {
    const int n = min(32, steps - k0);
    const long long mine = lane < n ? sh.step[k0 + lane] : 0, all = warp_sum(mine);
    if (target < all || k0 + 32 >= steps) {
      step = k0 + pick(mine, n, target, lane);
      break;
    }
    target -= all;
  }
  // The warp that had this step goes on: its values are at hand where it had no other behind it.
  if (step % WARPS != warp) return;
  if (step + WARPS < steps) sum = left_of(lo + 32 * step + lane, mass);
  long long to = warp_scan(sum, lane) - sum;       // before this lane
  if (target < to || target >= to + sum) return;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    if (target >= to && target < to + mass[e]) *out = (lo + 32 * step + lane) * N - off + e;
    to += mass[e];
  }
}

template <typename T>
cudaError_t launch_t(const VerifyParams& p, int num_sms, cudaStream_t st) {
  // CTAs of a row: 8, or as many as leave all rows on the GPU at once (1024 threads an SM), 2 at least.  Measured, 131072 fp32 values from L2:
  // 64 rows 9.6 us with 8, 12.4 with 4; 96 rows 16.2 and 14.8; 200 rows of 32000 18.5 with 8, 13.2 with 4, 10.7 with 2.
  int cluster = kMaxCluster;
  while (cluster > 2 && static_cast<int64_t>(p.b) * cluster > 4 * static_cast<int64_t>(num_sms)) cluster /= 2;
  // Twice the threads a CTA for fp32 rows while there are two vectors for each thread and all CTAs stay on the GPU: 16 rows of 131072 9.9 ->
  // 8.2 us, one 7.1 -> 6.1; 64 rows 16 -> 20, one of 1000 4.1 -> 4.4.  (16-bit rows: 7.5 and 7.6; trees of 48 in a step 12.1 and 13.8.)
  constexpr int kMore = sizeof(T) == 4 ? 512 : 256;
  const bool more = static_cast<int64_t>(p.b) * kMaxCluster <= 2 * static_cast<int64_t>(num_sms) && p.vocab >= 2 * Vec<T>::N * kMore * kMaxCluster;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.b) * cluster);
  cfg.blockDim = dim3(more ? kMore : 256);
  cfg.dynamicSmemBytes = static_cast<size_t>(p.s) * kRowBytes;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, more ? verify_kernel<T, kMore> : verify_kernel<T, 256>, p, cluster);
}

}  // namespace

cudaError_t launch_verify(const VerifyParams& p, int dtype, int num_sms, cudaStream_t st) {
  if (dtype == kF32) return launch_t<float>(p, num_sms, st);
  if (dtype == kBF16) return launch_t<__nv_bfloat16>(p, num_sms, st);
  return launch_t<__half>(p, num_sms, st);
}

}  // namespace sdpa
