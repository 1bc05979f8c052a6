// sdpa_decode.cu — attention of one or a few new tokens over a paged cache.
//
// The s_q tokens of a sequence times the query heads of a KV head's group are `rows` query rows
// that share the cache of that KV head.  Work is counted in tiles of 64 keys of one (sequence, KV
// head, block of 16 rows); every CTA takes an equal run of consecutive tiles over the whole batch,
// so that ragged lengths balance by themselves, and a run may end one sequence and begin the
// next.  A block that lies in one CTA's run is finished there; the others leave unnormalised
// partial results (O, running max, sum) that decode_combine_kernel joins, in a fixed order.
//
// Bound: reading the cache once.  With 16 rows a key costs 2 x 16 x d multiply-adds for 2 d
// elements read, far below what the tensor cores do in the time of the read; so the products are
// warp-level m16n8k16 MMAs on registers (a 128-row tcgen05 tile would be 7/8 empty and put its P
// through shared memory), and what counts is bytes in flight: each warp streams its own 16-key
// slices through a ring of cp.async stages and needs no other warp until the end of a run.
//
// Both products read the ring with 16-byte loads and no transposition:
//   S = Q K^T sums over d in any order, so a lane takes 16 contiguous bytes of its key and Q's
//   fragments are permuted to match;
//   O = P V wants pairs of keys in one register: a lane loads the same 16 bytes of two
//   neighbouring keys and interleaves them with byte permutes.
//
// E4M3 caches: codes widen exactly to F16; a key's scale multiplies its score, and the scale of
// its value joins the exponent, w = 2^(s + log2 vs - max), so that O = sum w v_code and
// l = sum w / vs.  The row max then bounds w whatever the scales, and no product with vs is rounded.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "ptx.cuh"
#include "sdpa_internal.h"

namespace sdpa {
namespace {

using namespace ptx;

constexpr int kWarps = 4;
constexpr int kSlice = 16;                 // keys of a warp's slice
constexpr int kTile = kWarps * kSlice;     // keys of a tile
constexpr int kRows = 16;                  // query rows of a block
constexpr int kThreads = kWarps * 32;

template <int D, int CT>
struct DecCfg {
  static constexpr int ES = CT == kE4M3 ? 1 : 2;
  static constexpr int RB = D * ES;                     // bytes of a row
  static constexpr int CH = RB / 16;                    // 16-byte chunks of a row
  static constexpr int EPC = 16 / ES;                   // elements of a chunk
  static constexpr int KCH = D / (4 * EPC);             // chunks of a key that one lane of four reads
  static constexpr int VB = RB >= 128 ? 16 : 8;         // bytes of a value row a lane reads at once
  static constexpr int EPV = VB / ES;                   // and elements
  static constexpr int VJ = D / (8 * EPV);              // such reads of a value row
  static constexpr int SC_BYTES = CT == kE4M3 ? 2 * kSlice * 4 : 0;
  static constexpr int STAGE = 2 * kSlice * RB + SC_BYTES;
  static constexpr int MERGE = kWarps * kRows * D * 4;  // the warps' partial O at the end of a run
  static constexpr int NS = D == 256 ? (CT == kE4M3 ? 3 : 3) : (STAGE > 4608 ? 3 : 6);
  static constexpr int RING = kWarps * NS * STAGE;
  static constexpr int SMEM = RING > MERGE ? RING : MERGE;
  static constexpr float P_OFF = (CT == kBF16) ? 0.f : 6.f;   // F16 weights: kept away from F16's lowest
  static constexpr float THRESH = 8.f;                  // the running max moves when exceeded by this much
};

// Position of 16-byte chunk `ch` of row `r` in a stage: neighbouring rows differ in bit 2 (the
// key reads of a quarter-warp are two rows of four chunks), rows 2c in bits 1-2 (the value
// reads are four even or odd rows of two chunks), so both are free of bank conflicts.
template <int CH>
__device__ __forceinline__ int swz(int r, int ch) {
  if constexpr (CH >= 8) return ch ^ ((((r >> 1) ^ (r << 1)) & 3) << 1);
  return ch ^ ((r >> 1) & (CH - 1));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// D += A B, 16x8x16, F16 or BF16 with fp32 accumulators.
template <bool BF>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
}

__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two_codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two_codes), __NV_E4M3);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <bool BF>
__device__ __forceinline__ uint32_t pack_pair(float a, float b) {
  if constexpr (BF) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

template <bool BF>
__device__ __forceinline__ float2 unpack_pair(uint32_t w) {
  if constexpr (BF) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// Clears the halves of a 16-bit pair that are infinite or NaN; `found` gathers whether any was.
template <bool BF>
__device__ __forceinline__ uint32_t finite_pair(uint32_t w, bool& found) {
  constexpr uint32_t kExp = BF ? 0x7F80u : 0x7C00u;
  if ((w & kExp) == kExp) {
    w &= 0xFFFF0000u;
    found = true;
  }
  if ((w & (kExp << 16)) == (kExp << 16)) {
    w &= 0x0000FFFFu;
    found = true;
  }
  return w;
}

// ---- the batch as one row of tiles -----------------------------------------------------------

struct SeqLens {
  int len_q, len_kv;
};

__device__ __forceinline__ SeqLens seq_lens(const DecodeParams& p, int bi) {
  SeqLens L;
  L.len_q = p.seq_lens_q ? min(max(__ldg(p.seq_lens_q + bi), 0), p.s_q) : p.s_q;
  L.len_kv = min(max(__ldg(p.c.seq_lens_kv + bi), 0), p.c.max_len);
  return L;
}

// Tiles of one block of rows of sequence bi (none where no row takes part).
__device__ __forceinline__ int seq_tiles(const DecodeParams& p, int bi) {
  const SeqLens L = seq_lens(p, bi);
  return L.len_q == 0 ? 0 : (L.len_kv + kTile - 1) / kTile;
}

// Sum of seq_tiles over sequences [0, n), by a whole warp.
__device__ long long tiles_before(const DecodeParams& p, int n, int lane) {
  long long t = 0;
  for (int i = lane; i < n; i += 32) t += seq_tiles(p, i);
#pragma unroll
  for (int o = 16; o > 0; o /= 2) t += __shfl_xor_sync(0xffffffffu, t, o);
  return t;
}

// CTAs that have a run: no more than tiles, so that none of them is empty.
__device__ __forceinline__ int working_ctas(const DecodeParams& p, long long total) {
  return total < p.ctas ? static_cast<int>(total) : p.ctas;
}

// First tile of CTA c's run, and the CTA whose run holds tile t, of `total` tiles over g CTAs.
__device__ __forceinline__ long long run_start(long long total, int c, int g) { return total * c / g; }
__device__ __forceinline__ int cta_of(long long total, long long t, int g) {
  return static_cast<int>(((t + 1) * g - 1) / total);
}

// Element offset of query row r (token r / group, head hk * group + r % group).
__device__ __forceinline__ int64_t row_offset(const DecodeParams& p, const int64_t (&st)[3], int bi, int hk, int r) {
  return bi * st[0] + (hk * p.group + r % p.group) * st[1] + (r / p.group) * st[2];
}

__device__ __forceinline__ bool tree_sees(const DecodeParams& p, int bi, int token, int j) {
  const uint32_t* w = p.tree_mask + bi * p.tree_mask_stride + static_cast<int64_t>(token) * p.tree_words;
  return (__ldg(w + j / 32) >> (j % 32)) & 1u;
}

// Whether query row r sees position `key` (< len_kv) of its sequence.
__device__ __forceinline__ bool row_sees(const DecodeParams& p, int bi, const SeqLens& L, int token, int key) {
  const int j = key - (L.len_kv - L.len_q);
  if (p.causal) return j <= token;
  if (p.tree_mask && j >= 0) return tree_sees(p, bi, token, j);
  return true;
}

template <int DT>
__device__ __forceinline__ void store_o(void* o, int64_t at, float x) {
  static_cast<uint16_t*>(o)[at] = static_cast<uint16_t>(pack_pair<DT == kBF16>(x, 0.f) & 0xFFFFu);
}

// Infinities and NaNs of the drafted tokens' values: the products ran without them (a hidden
// one times a weight of zero would be NaN); the rows that see them get them here.
template <int D, int CT>
__device__ float add_nonfinite(const DecodeParams& p, int bi, int hk, const SeqLens& L, int r, int d, int key0, int key1,
                               float x) {
  const int token = r / p.group;
  // From the first slice that holds a new token (all of it was cleared).
  for (int key = max(key0, (L.len_kv - L.len_q) & ~(kSlice - 1)); key < key1; ++key) {
    if (!row_sees(p, bi, L, token, key)) continue;
    const int page = __ldg(p.c.page_table + bi * p.c.page_table_stride + key / p.c.page_size);
    if (page < 0 || page >= p.c.num_pages) continue;
    const uint8_t* row = p.c.v + page * p.c.v_st[0] + hk * p.c.v_st[1] + (key % p.c.page_size) * p.c.v_st[2];
    float v;
    if (CT == kE4M3) v = (row[d] & 0x7F) == 0x7F ? __uint_as_float(0x7FC00000u) : 0.f;
    else v = unpack_pair<CT == kBF16>(reinterpret_cast<const uint16_t*>(row)[d]).x;
    if (!isfinite(v)) x += v;
  }
  return x;
}

// ---- main kernel -----------------------------------------------------------------------------

template <int D, int CT, int QT>
__global__ void __launch_bounds__(kThreads) decode_kernel(const __grid_constant__ DecodeParams p) {
  using C = DecCfg<D, CT>;
  constexpr bool E4 = CT == kE4M3;
  constexpr bool BF = CT == kBF16;           // type of the products' operands
  constexpr int NT = D / 8;                  // 8-column tiles of O
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
  __shared__ int s_found;

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, c = lane % 4;
  uint8_t* ring = smem + warp * C::NS * C::STAGE;
  const uint32_t ring_a = smem_u32(ring);

  const int per_seq = p.c.h_kv * p.row_tiles;              // blocks of rows of a sequence
  const long long total = tiles_before(p, p.c.b, lane) * per_seq;
  griddep_launch_dependents();
  const int n_cta = working_ctas(p, total);
  if (static_cast<int>(blockIdx.x) >= n_cta) return;
  long long t = run_start(total, blockIdx.x, n_cta);
  const long long t_end = run_start(total, blockIdx.x + 1, n_cta);

  // The sequence that holds tile t.
  int bi = 0;
  long long base = 0;    // first tile of sequence bi
  for (;; ) {
    const int i = bi + lane;
    const long long n = i < p.c.b ? static_cast<long long>(seq_tiles(p, i)) * per_seq : 0;
    long long incl = n;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const long long x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, base + incl > t);
    if (hit != 0) {
      const int k = __ffs(hit) - 1;
      base += __shfl_sync(0xffffffffu, incl - n, k);
      bi += k;
      break;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
    bi += 32;
    if (bi >= p.c.b) return;   // not reached: t < total
  }

  while (t < t_end) {
    const SeqLens L = seq_lens(p, bi);
    const int n_tiles = seq_tiles(p, bi);
    if (t >= base + static_cast<long long>(n_tiles) * per_seq) {
      base += static_cast<long long>(n_tiles) * per_seq;
      ++bi;
      continue;
    }
    const int blk = static_cast<int>((t - base) / n_tiles);
    const int hk = blk / p.row_tiles, r0 = (blk % p.row_tiles) * kRows;
    const long long blk_t0 = base + static_cast<long long>(blk) * n_tiles;
    const int tile0 = static_cast<int>(t - blk_t0);
    const int tile1 = static_cast<int>(min(static_cast<long long>(n_tiles), t_end - blk_t0));
    const int off = L.len_kv - L.len_q;           // position of the first new token
    const bool masked = p.causal != 0 || p.tree_mask != nullptr;

    // ---- the ring: slice i of this warp is keys (tile0 + i) * 64 + warp * 16 ------------------
    const int n_slices = tile1 - tile0;
    int page_cache = 0;    // lane i: page of slice (i of the last 32 asked for), or -1
    auto page_of = [&](int i) {
      if (i % 32 == 0) {
        const int key = (tile0 + i + lane) * kTile + warp * kSlice;
        page_cache = -1;
        if (i + lane < n_slices && key < L.len_kv) {
          const int page = __ldg(p.c.page_table + bi * p.c.page_table_stride + key / p.c.page_size);
          if (page >= 0 && page < p.c.num_pages) page_cache = page;
        }
      }
      return __shfl_sync(0xffffffffu, page_cache, i % 32);
    };
    unsigned valid_hist = 0;   // 5 bits a stage in flight: keys of the slice that exist
    auto load = [&](int i) {
      if (i < n_slices) {
        const int key = (tile0 + i) * kTile + warp * kSlice;
        const int page = page_of(i);
        const int valid = page < 0 ? 0 : min(max(L.len_kv - key, 0), kSlice);
        const int slot = key % p.c.page_size;
        const int64_t pg = page < 0 ? 0 : page;
        const uint8_t* kp = p.c.k + pg * p.c.k_st[0] + hk * p.c.k_st[1] + slot * p.c.k_st[2];
        const uint8_t* vp = p.c.v + pg * p.c.v_st[0] + hk * p.c.v_st[1] + slot * p.c.v_st[2];
        const uint32_t dst = ring_a + (i % C::NS) * C::STAGE;
#pragma unroll
        for (int x = 0; x < kSlice * C::CH / 32; ++x) {
          const int id = x * 32 + lane, r = id / C::CH, ch = id % C::CH;
          const bool on = r < valid;
          const uint32_t at = dst + r * C::RB + swz<C::CH>(r, ch) * 16;
          cp_async16(at, on ? kp + r * p.c.k_st[2] + ch * 16 : p.c.k, on);
          cp_async16(at + kSlice * C::RB, on ? vp + r * p.c.v_st[2] + ch * 16 : p.c.v, on);
        }
        if constexpr (E4) {
          if (lane < 8) {
            const bool on = valid > 0;
            const float* src = (lane < 4 ? p.c.k_scale : p.c.v_scale) + (pg * p.c.h_kv + hk) * p.c.page_size + slot + (lane % 4) * 4;
            cp_async16(dst + 2 * kSlice * C::RB + lane * 16, on ? src : p.c.k_scale, on);
          }
        }
        valid_hist = (valid_hist & ~(31u << (5 * (i % C::NS)))) | (static_cast<unsigned>(valid) << (5 * (i % C::NS)));
      }
      cp_commit();
    };
    static_assert(C::NS * 5 <= 32, "valid_hist");
    for (int i = 0; i < C::NS - 1; ++i) load(i);

    // ---- Q fragments (rows g and g + 8), permuted to the order in which lanes read keys -------
    uint32_t qf[D / 16][4];
    float cs[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int r = r0 + g + 8 * u;
      const bool on = r < p.rows && r / p.group < L.len_q;
      const uint16_t* row = static_cast<const uint16_t*>(p.q) + (on ? row_offset(p, p.q_st, bi, hk, r) : 0);
      uint32_t w[D / 8];
#pragma unroll
      for (int j = 0; j < C::KCH; ++j) {
#pragma unroll
        for (int e = 0; e < C::EPC / 8; ++e) {
          uint4 x = make_uint4(0, 0, 0, 0);
          if (on) x = *reinterpret_cast<const uint4*>(row + (j * 4 + c) * C::EPC + e * 8);
          const int at = j * (C::EPC / 2) + e * 4;
          w[at] = x.x; w[at + 1] = x.y; w[at + 2] = x.z; w[at + 3] = x.w;
        }
      }
      cs[u] = p.scale_log2;
      if constexpr (E4 && QT == kBF16) {
        // The products of an E4M3 cache run in F16: a power of two brings the row's largest
        // element to [256, 512), where F16 holds every BF16 value down to 2^-22 of it exactly.
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) m = max(m, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const int ex = static_cast<int>(m >> 7);           // biased exponent of the largest
        const int sh = (ex == 0 || ex == 255) ? 0 : min(127 + 8 - ex, 126);
        const float up = __uint_as_float(static_cast<uint32_t>(127 + sh) << 23);
        cs[u] *= __uint_as_float(static_cast<uint32_t>(127 - sh) << 23);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const float2 f = unpack_pair<true>(w[i]);
          w[i] = pack_pair<false>(f.x * up, f.y * up);
        }
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        qf[i][u] = w[2 * i];
        qf[i][u + 2] = w[2 * i + 1];
      }
    }

    float o[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m_ref[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    bool found = false;
    if (threadIdx.x == 0) s_found = 0;

    for (int i = 0; i < n_slices; ++i) {
      cp_wait<C::NS - 2>();
      __syncwarp();             // slice i has landed, and every lane is done with slice i - 1
      load(i + C::NS - 1);
      const uint8_t* st = ring + (i % C::NS) * C::STAGE;
      const int valid = (valid_hist >> (5 * (i % C::NS))) & 31;
      const int key0 = (tile0 + i) * kTile + warp * kSlice;
      if (valid > 0) {
        // ---- S = Q K^T -------------------------------------------------------------------
        float s[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
          const int r = n * 8 + g;
#pragma unroll
          for (int j = 0; j < C::KCH; ++j) {
            const uint4 k4 = *reinterpret_cast<const uint4*>(st + r * C::RB + swz<C::CH>(r, j * 4 + c) * 16);
            const uint32_t w[4] = {k4.x, k4.y, k4.z, k4.w};
            if constexpr (E4) {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                mma16816<BF>(s[n], qf[4 * j + e], e4m3x2_to_f16x2(w[e] & 0xFFFFu), e4m3x2_to_f16x2(w[e] >> 16));
            } else {
              mma16816<BF>(s[n], qf[2 * j], w[0], w[1]);
              mma16816<BF>(s[n], qf[2 * j + 1], w[2], w[3]);
            }
          }
        }
        // ---- scale, mask; thread: rows g, g + 8, keys 2c, 2c + 1 of each n ----------------------
        float rvs[2][2];   // 1 / scale of a key's value (E4M3)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float ks = 1.f, lv = 0.f;
            if constexpr (E4) {
              const float* sc = reinterpret_cast<const float*>(st + 2 * kSlice * C::RB);
              ks = sc[n * 8 + 2 * c + e];
              float vs = sc[kSlice + n * 8 + 2 * c + e];
              if (n * 8 + 2 * c + e >= valid) vs = 1.f;
              lv = __log2f(vs);
              rvs[n][e] = __fdividef(1.f, vs);
            }
            s[n][e] = fmaf(s[n][e], cs[0] * ks, lv);
            s[n][e + 2] = fmaf(s[n][e + 2], cs[1] * ks, lv);
          }
        const bool tail = masked && key0 + kSlice > off;
        if (valid < kSlice || tail) {
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int kk = n * 8 + 2 * c + (e & 1);
              const int r = r0 + g + 8 * (e >> 1), token = r / p.group;
              bool see = kk < valid;
              if (see && tail && r < p.rows && token < L.len_q) see = row_sees(p, bi, L, token, key0 + kk);
              if (!see) s[n][e] = -INFINITY;
            }
        }
        // ---- running max, weights, sums ----------------------------------------------------
        uint32_t pa[4];
        float alpha[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float mx = fmaxf(fmaxf(s[0][2 * u], s[0][2 * u + 1]), fmaxf(s[1][2 * u], s[1][2 * u + 1]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          alpha[u] = 1.f;
          if (mx > m_ref[u] + C::THRESH) {
            alpha[u] = ex2(m_ref[u] - mx);
            m_ref[u] = mx;
          }
          const float nm = m_ref[u] == -INFINITY ? 0.f : C::P_OFF - m_ref[u];
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = ex2(s[e / 2][2 * u + e % 2] + nm);
          float add;
          if constexpr (E4) add = (w[0] * rvs[0][0] + w[1] * rvs[0][1]) + (w[2] * rvs[1][0] + w[3] * rvs[1][1]);
          else add = (w[0] + w[1]) + (w[2] + w[3]);
          l[u] = l[u] * alpha[u] + add;
          pa[u] = pack_pair<BF>(w[0], w[1]);
          pa[u + 2] = pack_pair<BF>(w[2], w[3]);
        }
        if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
          for (int x = 0; x < NT; ++x) {
            o[x][0] *= alpha[0];
            o[x][1] *= alpha[0];
            o[x][2] *= alpha[1];
            o[x][3] *= alpha[1];
          }
        }
        // ---- O += P V ------------------------------------------------------------------------
#pragma unroll
        for (int j = 0; j < C::VJ; ++j) {
          uint32_t v[4][C::VB / 4];   // keys 2c, 2c + 1, 2c + 8, 2c + 9
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const int r = 2 * c + (kk & 1) + 8 * (kk >> 1);
            const uint8_t* row = st + (kSlice + r) * C::RB;
            if constexpr (C::VB == 16) {
              const uint4 x = *reinterpret_cast<const uint4*>(row + swz<C::CH>(r, j * 8 + g) * 16);
              v[kk][0] = x.x; v[kk][1] = x.y; v[kk][2] = x.z; v[kk][3] = x.w;
            } else {
              const uint2 x = *reinterpret_cast<const uint2*>(row + swz<C::CH>(r, (j * 8 + g) / 2) * 16 + (g % 2) * 8);
              v[kk][0] = x.x; v[kk][1] = x.y;
            }
          }
#pragma unroll
          for (int x = 0; x < C::EPV; ++x) {
            uint32_t b0, b1;
            if constexpr (E4) {
              const uint32_t sel = (x % 4) | ((x % 4 + 4) << 4);
              b0 = e4m3x2_to_f16x2(prmt(v[0][x / 4], v[1][x / 4], sel));
              b1 = e4m3x2_to_f16x2(prmt(v[2][x / 4], v[3][x / 4], sel));
            } else {
              const uint32_t sel = x % 2 ? 0x7632u : 0x5410u;
              b0 = prmt(v[0][x / 2], v[1][x / 2], sel);
              b1 = prmt(v[2][x / 2], v[3][x / 2], sel);
            }
            if (tail) {
              b0 = finite_pair<BF>(b0, found);
              b1 = finite_pair<BF>(b1, found);
            }
            mma16816<BF>(o[j * C::EPV + x], pa, b0, b1);
          }
        }
      }
    }
    cp_wait<0>();

    // ---- the four warps' results meet -----------------------------------------------------------
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      l[u] += __shfl_xor_sync(0xffffffffu, l[u], 1);
      l[u] += __shfl_xor_sync(0xffffffffu, l[u], 2);
      if (c == 0) {
        s_m[warp][g + 8 * u] = m_ref[u];
        s_l[warp][g + 8 * u] = l[u];
      }
    }
    __syncthreads();
    if (found) s_found = 1;
    float big[2];
    float* merge = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int r = g + 8 * u;
      big[u] = s_m[0][r];
      for (int w = 1; w < kWarps; ++w) big[u] = fmaxf(big[u], s_m[w][r]);
      const float f = m_ref[u] == -INFINITY ? 0.f : ex2(m_ref[u] - big[u]);
      // Columns of 8-wide tile j * EPV + x: d = (j * 8 + n) * EPV + x for n = 2c, 2c + 1.
      float* row = merge + (warp * kRows + r) * D;
#pragma unroll
      for (int j = 0; j < C::VJ; ++j)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int x = 0; x < C::EPV; x += 4) {
            float4 q4;
            q4.x = o[j * C::EPV + x][2 * u + n] * f;
            q4.y = o[j * C::EPV + x + 1][2 * u + n] * f;
            q4.z = o[j * C::EPV + x + 2][2 * u + n] * f;
            q4.w = o[j * C::EPV + x + 3][2 * u + n] * f;
            if (m_ref[u] == -INFINITY && f == 0.f && l[u] == 0.f) q4 = make_float4(0.f, 0.f, 0.f, 0.f);
            *reinterpret_cast<float4*>(row + (j * 8 + 2 * c + n) * C::EPV + x) = q4;
          }
    }
    __syncthreads();
    const bool whole = tile0 == 0 && tile1 == n_tiles;
    const int part = 2 * blockIdx.x + (tile0 == 0 ? 1 : 0);
    const bool fix = s_found != 0;
    for (int idx = threadIdx.x; idx < kRows * D; idx += kThreads) {
      const int r = idx / D, d = idx % D;
      float mb = s_m[0][r], lb = 0.f, x = 0.f;
      for (int w = 1; w < kWarps; ++w) mb = fmaxf(mb, s_m[w][r]);
      for (int w = 0; w < kWarps; ++w) {
        x += merge[(w * kRows + r) * D + d];
        if (s_l[w][r] != 0.f) lb += s_l[w][r] * (s_m[w][r] == -INFINITY ? 1.f : ex2(s_m[w][r] - mb));
      }
      const int row = r0 + r, token = row / p.group;
      const bool on = row < p.rows && token < L.len_q;
      if (fix && on) x = add_nonfinite<D, CT>(p, bi, hk, L, row, d, tile0 * kTile, min(tile1 * kTile, L.len_kv), x);
      if (!whole) {
        p.part_o[(static_cast<int64_t>(part) * kRows + r) * D + d] = x;
        if (d == 0) {
          p.part_ml[(part * kRows + r) * 2] = mb;
          p.part_ml[(part * kRows + r) * 2 + 1] = lb;
        }
      } else if (row < p.rows) {
        const bool none = !on || lb == 0.f;
        store_o<QT>(p.o, row_offset(p, p.o_st, bi, hk, row) + d, none ? 0.f : x / lb);
        if (p.lse && d == 0)
          p.lse[(static_cast<int64_t>(bi) * p.h_q + hk * p.group + row % p.group) * p.s_q + token] =
              none ? -INFINITY : (mb - C::P_OFF + __log2f(lb)) * 0.6931471805599453f;
      }
    }
    __syncthreads();   // the ring and the exchange arrays are free again
    t = blk_t0 + tile1;
  }
}

// Joins the partial results of every block of rows that more than one CTA worked on, and writes
// the rows that no key reaches.  One CTA a row: its lanes weigh the parts side by side (a part is
// a maximum, a sum and d values), then each warp adds up every fourth part, 8 loads in flight,
// and the four sums meet.  The order is that of the parts, so results do not change between calls.
template <int D, int QT>
__global__ void __launch_bounds__(kThreads) decode_combine_kernel(const __grid_constant__ DecodeParams p, float p_off) {
  constexpr int EL = D / 32;          // elements a lane owns
  __shared__ float s_sum[kWarps][D];
  __shared__ float s_l[kWarps];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rows_blk = min(p.rows, kRows);
  const int per_seq = p.c.h_kv * p.row_tiles;
  const int unit = blockIdx.x / rows_blk, r = blockIdx.x % rows_blk;
  const int bi = unit / per_seq, blk = unit % per_seq;
  const int hk = blk / p.row_tiles, row = blk % p.row_tiles * kRows + r, token = row / p.group;
  const int n_tiles = seq_tiles(p, bi);
  const SeqLens L = seq_lens(p, bi);
  int c0 = 0, n = 0;                  // parts: CTAs c0 .. c0 + n - 1 (none where there are no tiles)
  if (n_tiles > 0) {
    const long long total = tiles_before(p, p.c.b, lane) * per_seq;
    const long long t0 = tiles_before(p, bi, lane) * per_seq + static_cast<long long>(blk) * n_tiles;
    c0 = cta_of(total, t0, working_ctas(p, total));
    n = cta_of(total, t0 + n_tiles - 1, working_ctas(p, total)) - c0 + 1;
  }
  griddep_wait();   // (by every CTA, so that this grid never ends before the one it follows)
  if (n == 1 || row >= p.rows) return;       // finished by that CTA
  // Part k: the first holds its block's first tile and is that CTA's second part.
  auto part = [&](int k) { return static_cast<int64_t>(2 * (c0 + k) + (k == 0 ? 1 : 0)) * kRows + r; };
  float m = -INFINITY;
  for (int k = lane; k < n; k += 32) {
    const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + 2 * part(k));
    if (ml.y != 0.f) m = fmaxf(m, ml.x);
  }
#pragma unroll
  for (int o = 16; o > 0; o /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float x[EL], l = 0.f;
#pragma unroll
  for (int e = 0; e < EL; ++e) x[e] = 0.f;
  for (int k0 = warp; k0 < n; k0 += 8 * kWarps) {
    float f[8], v[8][EL];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int k = k0 + u * kWarps;
      f[u] = 0.f;
#pragma unroll
      for (int e = 0; e < EL; ++e) v[u][e] = 0.f;
      if (k < n) {
        const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + 2 * part(k));
        const float* src = p.part_o + part(k) * D + lane * EL;
#pragma unroll
        for (int e = 0; e < EL; e += 2) {
          const float2 w = *reinterpret_cast<const float2*>(src + e);
          v[u][e] = w.x;
          v[u][e + 1] = w.y;
        }
        // A part without a visible key has sum 0 and weighs nothing.  (All sums NaN: m stays -inf.)
        if (ml.y != 0.f) {
          f[u] = ml.x == -INFINITY ? 1.f : ex2(ml.x - m);
          l += ml.y * f[u];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
#pragma unroll
      for (int e = 0; e < EL; ++e) x[e] += f[u] == 0.f ? 0.f : v[u][e] * f[u];
  }
#pragma unroll
  for (int e = 0; e < EL; ++e) s_sum[warp][lane * EL + e] = x[e];
  if (lane == 0) s_l[warp] = l;
  __syncthreads();
  l = (s_l[0] + s_l[1]) + (s_l[2] + s_l[3]);
  const bool none = token >= L.len_q || l == 0.f;
  const int64_t at = row_offset(p, p.o_st, bi, hk, row);
  for (int d = threadIdx.x; d < D; d += kThreads)
    store_o<QT>(p.o, at + d, none ? 0.f : ((s_sum[0][d] + s_sum[1][d]) + (s_sum[2][d] + s_sum[3][d])) / l);
  if (p.lse && threadIdx.x == 0)
    p.lse[(static_cast<int64_t>(bi) * p.h_q + hk * p.group + row % p.group) * p.s_q + token] =
        none ? -INFINITY : (m - p_off + __log2f(l)) * 0.6931471805599453f;
}

template <int D, int CT, int QT>
cudaError_t launch_t(const DecodeParams& p, cudaStream_t st) {
  using C = DecCfg<D, CT>;
  auto kern = decode_kernel<D, CT, QT>;
  cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kern), C::SMEM);
  if (e != cudaSuccess) return e;
  kern<<<p.ctas, kThreads, C::SMEM, st>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.c.b) * p.c.h_kv * p.row_tiles * (p.rows < kRows ? p.rows : kRows));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_combine_kernel<D, QT>, p, C::P_OFF);
}

template <int D>
cudaError_t launch_d(const DecodeParams& p, int qt, int ct, cudaStream_t st) {
  if (qt == kBF16) return ct == kE4M3 ? launch_t<D, kE4M3, kBF16>(p, st) : launch_t<D, kBF16, kBF16>(p, st);
  return ct == kE4M3 ? launch_t<D, kE4M3, kF16>(p, st) : launch_t<D, kF16, kF16>(p, st);
}

}  // namespace

int decode_ctas(const DecodeParams& p, int num_sms) {
  const long long tiles = static_cast<long long>(p.c.b) * p.c.h_kv * p.row_tiles * ((p.c.max_len + kTile - 1ll) / kTile);
  return static_cast<int>(tiles < 2ll * num_sms ? (tiles < 1 ? 1 : tiles) : 2ll * num_sms);
}

size_t decode_workspace_bytes(const DecodeParams& p, int d, int num_sms, size_t* ml_offset) {
  const size_t parts = 2 * static_cast<size_t>(decode_ctas(p, num_sms)) * kRows;
  if (ml_offset) *ml_offset = parts * d * 4;
  return (parts * d * 4 + parts * 8 + 255) & ~size_t(255);
}

cudaError_t launch_decode(const DecodeParams& p, int d, int qt, int ct, cudaStream_t st) {
  if (d == 64) return launch_d<64>(p, qt, ct, st);
  if (d == 128) return launch_d<128>(p, qt, ct, st);
  if (d == 256) return launch_d<256>(p, qt, ct, st);
  return cudaErrorInvalidValue;
}

}  // namespace sdpa
