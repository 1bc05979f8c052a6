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
// that the drawn number falls into reads the piece of the row once more, from L2.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx.cuh"
#include "sdpa_internal.h"

namespace sdpa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kAhead = 2;                      // vectors a thread has in flight
constexpr float kUnit = 4398046511104.f;       // 2^42
constexpr int kMaxSteps = 130;                 // steps of 32 vectors in a warp's piece: at most 2^20 / 4 / (8 * 8) / 32, and what rounds up

template <typename T>
__device__ __forceinline__ float widen(T x) {
  return static_cast<float>(x);
}

// 16 bytes of a row as values.
template <typename T>
struct Vec {
  static constexpr int N = 16 / sizeof(T);
  float x[N];
};

// Elements [first, first + N) of a row of n; those outside are 0.  `wide`: first is at a multiple of 16 bytes.
template <typename T>
__device__ __forceinline__ Vec<T> load_vec(const T* row, int first, int n, bool wide) {
  Vec<T> v;
  if (wide && first >= 0 && first + Vec<T>::N <= n) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(row + first));
    const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int i = 0; i < Vec<T>::N; ++i) v.x[i] = widen(e[i]);
  } else {
#pragma unroll
    for (int i = 0; i < Vec<T>::N; ++i) v.x[i] = first + i >= 0 && first + i < n ? widen(row[first + i]) : 0.f;
  }
  return v;
}

// A mass p 2^42 as h 2^22 + l: h = floor(p 2^20), and l = p 2^42 - h 2^22 rounded to the nearest (ties to even, as for the
// sum of both: h 2^22 is even).  Both come out of the last bits of fp32 sums with 2^23, at the rate of fp32
// arithmetic (a conversion to 64 bits has the rate of fp64: 36 us against 16 for 64 rows of 131072).  Sums of up to 2^9 of either fit 32 bits.
struct Mass {
  uint32_t h, l;
  __device__ __forceinline__ long long whole() const { return (static_cast<long long>(h) << 22) + l; }
};

// NaN and what is below zero counts nothing, what is above one counts one.
__device__ __forceinline__ Mass mass_of(float p) {
  const float x = __saturatef(p), top = __fmaf_rz(x, 1048576.f, 8388608.f), rest = fmaf(x, 1048576.f, 8388608.f - top);
  const float low = __fmaf_rn(rest, 4194304.f, 8388608.f);
  return {__float_as_uint(top) - 0x4B000000u, __float_as_uint(low) - 0x4B000000u};
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

struct Shared {
  long long mass[kVerifyRows];      // of each drafted token behind its parent (0 where an earlier sibling has it too)
  int32_t parent[kVerifyRows];      // -1: not a node
  int32_t token[kVerifyRows];
  uint8_t good[kVerifyRows];
  int32_t path[kVerifyRows];
  int32_t gone[kVerifyRows];        // tokens that are not drawn any more
  long long gone_mass[kVerifyRows];
  int accepted, refused, n_gone;    // refused: the row of the refused draft of a chain, or -1
  long long warp[kWarps];
  long long cta[2][kMaxCluster];    // of every CTA of the cluster, in each turn
  long long step[kMaxSteps];
};

// Which rows are accepted: sh.path, sh.accepted; what may not be drawn: sh.refused (a chain with q), sh.gone.
template <typename T>
__device__ void walk(const VerifyParams& p, Shared& sh, int bi, int len) {
  const int tid = threadIdx.x;
  const T* probs = static_cast<const T*>(p.probs) + bi * p.probs_b;
  const T* draft = static_cast<const T*>(p.draft) + bi * p.draft_b;
  const int64_t at = static_cast<int64_t>(bi) * p.s;
  if (tid == 0) {
    sh.accepted = len;
    sh.n_gone = 0;
  }
  for (int j = tid; j < len; j += kThreads) {
    const int x = __ldg(p.tokens + at + j);
    const int par = j == 0 ? -1 : p.parents ? __ldg(p.parents + at + j) : j - 1;
    const bool node = j > 0 && par >= 0 && par < j, known = node && x >= 0 && x < p.vocab;
    const float pr = known ? widen(probs[par * p.probs_s + x]) : 0.f;
    sh.token[j] = x;
    sh.parent[j] = node ? par : -1;
    sh.mass[j] = mass_of(pr).whole();
    if (p.draft) {
      const float q = known ? widen(draft[j * p.draft_s + x]) : 0.f;
      // The product of two fp32 values is exact in fp64.
      sh.good[j] = j == 0 || (known && static_cast<double>(__ldg(p.uniform + at + j)) * q < static_cast<double>(pr));
    }
  }
  __syncthreads();
  if (!p.parents) {
    // A chain: up to the first that is not accepted.
    for (int j = tid; j < len; j += kThreads) {
      bool good = j == 0;
      if (j > 0) good = p.draft ? sh.good[j] : __ldg(p.uniform + at + j) * static_cast<double>(kUnit) < static_cast<double>(sh.mass[j]);
      if (!good) atomicMin(&sh.accepted, j);
    }
    __syncthreads();
    const int n = sh.accepted;
    for (int j = tid; j < n; j += kThreads) sh.path[j] = j;
    if (tid == 0) {
      sh.refused = p.draft && n < len ? n : -1;
      if (!p.draft && n < len) {
        sh.gone[0] = sh.token[n];
        sh.gone_mass[0] = sh.mass[n];
        sh.n_gone = 1;
      }
    }
    __syncthreads();
    return;
  }
  // A tree.  A token that an earlier sibling has counts nothing.
  bool twin[kVerifyRows / kThreads];
#pragma unroll
  for (int k = 0; k < kVerifyRows / kThreads; ++k) {
    const int j = tid + k * kThreads;
    twin[k] = false;
    if (j < len && sh.parent[j] >= 0)
      for (int i = sh.parent[j] + 1; i < j; ++i) twin[k] |= sh.parent[i] == sh.parent[j] && sh.token[i] == sh.token[j];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kVerifyRows / kThreads; ++k)
    if (twin[k]) sh.mass[tid + k * kThreads] = 0;
  __syncthreads();
  for (int j = tid; j < len; j += kThreads) {
    long long left = static_cast<long long>(kUnit);
    if (sh.parent[j] >= 0)
      for (int i = sh.parent[j] + 1; i < j; ++i) left -= sh.parent[i] == sh.parent[j] ? sh.mass[i] : 0;
    if (left < 0) left = 0;
    sh.good[j] = sh.parent[j] >= 0 && __dmul_rn(static_cast<double>(__ldg(p.uniform + at + j)), static_cast<double>(left)) <
                                          static_cast<double>(sh.mass[j]);
  }
  __syncthreads();
  if (tid < 32) {
    // From node to node: the first good child, all of them behind it.
    int n = 0, count = 1;
    if (tid == 0) sh.path[0] = 0;
    for (int j0 = 1; j0 < len;) {
      const int j = j0 + tid;
      const uint32_t hit = __ballot_sync(0xffffffffu, j < len && sh.parent[j] == n && sh.good[j]);
      if (hit) {
        n = j0 + __ffs(hit) - 1;
        if (tid == 0) sh.path[count] = n;
        ++count;
        j0 = n + 1;
      } else {
        j0 += 32;
      }
    }
    int gone = 0;
    for (int j0 = n + 1; j0 < len; j0 += 32) {
      const int j = j0 + tid;
      const bool child = j < len && sh.parent[j] == n;
      const uint32_t hit = __ballot_sync(0xffffffffu, child);
      if (child) {
        const int k = gone + __popc(hit & ((1u << tid) - 1));
        sh.gone[k] = sh.token[j];
        sh.gone_mass[k] = sh.mass[j];
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

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) verify_kernel(const __grid_constant__ VerifyParams p, int cluster) {
  constexpr int N = Vec<T>::N;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Shared& sh = *reinterpret_cast<Shared*>(smem_raw);
  const int bi = blockIdx.x / cluster, rank = blockIdx.x - bi * cluster;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  cluster_arrive();
  // The kernel before is done (and the next one may be put in place, to wait here in its turn).
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int len = p.seq_lens_q ? min(max(__ldg(p.seq_lens_q + bi), 0), p.s) : p.s;
  const int64_t at = static_cast<int64_t>(bi) * p.s;
  const float u0 = __ldg(p.uniform + at);
  if (len > 0) walk<T>(p, sh, bi, len);
  const int accepted = len > 0 ? sh.accepted : 0;
  // Behind the new token there is none; the token itself is written by the CTA that finds it.
  if (rank == 0) {
    if (tid == 0) p.accepted[bi] = accepted;
    for (int j = tid; j < p.s; j += kThreads) {
      p.path[at + j] = j < accepted ? sh.path[j] : -1;
      if (j != accepted - 1) p.new_tokens[at + j] = j < accepted ? sh.token[sh.path[j + 1]] : -1;
    }
  }
  if (len == 0) {             // (the whole cluster)
    cluster_wait();
    return;
  }

  const int last = sh.path[accepted - 1], refused = sh.refused;
  const T* row = static_cast<const T*>(p.probs) + bi * p.probs_b + last * p.probs_s;
  const T* less = refused >= 0 ? static_cast<const T*>(p.draft) + bi * p.draft_b + refused * p.draft_s : nullptr;
  // Vectors of 16 bytes from the multiple of 16 at or before the row's start; each warp has a piece of them.
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(row) % 16 / sizeof(T));
  const bool less_wide = less && reinterpret_cast<uintptr_t>(less) % 16 / sizeof(T) == static_cast<unsigned>(off);
  const int vectors = (off + p.vocab + N - 1) / N, pieces = cluster * kWarps, per = (vectors + pieces - 1) / pieces;
  auto value = [&](int v, bool diff) {
    const int first = v * N - off;
    Vec<T> x = load_vec(row, first, p.vocab, true);
    if (diff) {
      const Vec<T> y = load_vec(less, first, p.vocab, less_wide);
#pragma unroll
      for (int e = 0; e < N; ++e) x.x[e] -= y.x[e];
    }
    return x;
  };

  // What is left of the distribution first; where that is nothing, the distribution.
  bool diff = less != nullptr;
  int n_gone = sh.n_gone;
  const int piece = rank * kWarps + warp, v_lo = min(vectors, piece * per), v_hi = min(vectors, v_lo + per);
  long long total = 0, target = 0;
  for (int turn = 0; turn < 2; ++turn) {
    long long sum = 0;
    for (int v0 = v_lo + lane; v0 < v_hi; v0 += 32 * kAhead) {
      Vec<T> x[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (v0 + 32 * k < v_hi) x[k] = value(v0 + 32 * k, diff);
      Mass part = {0, 0};
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (v0 + 32 * k >= v_hi) continue;
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const Mass m = mass_of(x[k].x[e]);
          part.h += m.h;
          part.l += m.l;
        }
      }
      sum += part.whole();
    }
    for (int g = lane; g < n_gone; g += 32)
      if (sh.gone_mass[g] > 0) {
        const int v = (sh.gone[g] + off) / N;
        if (v >= v_lo && v < v_hi) sum -= sh.gone_mass[g];
      }
    sum = warp_sum(sum);
    if (lane == 0) sh.warp[warp] = sum;
    __syncthreads();
    if (warp == 0) {
      // The CTA's sum goes to every CTA of the cluster.
      const long long all = warp_sum(lane < kWarps ? sh.warp[lane] : 0);
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
  const int w = pick(lane < kWarps ? sh.warp[lane] : 0, kWarps, target, lane);
  // The piece of warp w once more, a step of 32 vectors a warp.
  const int lo = min(vectors, (rank * kWarps + w) * per), hi = min(vectors, lo + per), steps = (hi - lo + 31) / 32;
  auto left_of = [&](int v, long long (&mass)[N]) {
    long long sum = 0;
    if (v < hi) {
      const Vec<T> x = value(v, diff);
#pragma unroll
      for (int e = 0; e < N; ++e) mass[e] = mass_of(x.x[e]).whole();
      for (int g = 0; g < n_gone; ++g) {
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (sh.gone[g] == v * N - off + e) mass[e] = 0;
      }
#pragma unroll
      for (int e = 0; e < N; ++e) sum += mass[e];
    }
    return sum;
  };
  long long mass[N], sum = 0;
  int k = warp;
  for (; k < steps; k += kWarps) {
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
  if (step % kWarps != warp) return;
  if (step + kWarps < steps) sum = left_of(lo + 32 * step + lane, mass);
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
  const int cluster = 8;
  cudaError_t e = set_smem_once(reinterpret_cast<const void*>(&verify_kernel<T>), sizeof(Shared));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.b) * cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Shared);
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, verify_kernel<T>, p, cluster);
}

}  // namespace

cudaError_t launch_verify(const VerifyParams& p, int dtype, int num_sms, cudaStream_t st) {
  if (dtype == kF32) return launch_t<float>(p, num_sms, st);
  if (dtype == kBF16) return launch_t<__nv_bfloat16>(p, num_sms, st);
  return launch_t<__half>(p, num_sms, st);
}

}  // namespace sdpa
