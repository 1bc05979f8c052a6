// sdpa_decode.cuh — what the kernels of attention over a cache share: the split of a batch into runs of
// tiles, what a row sees, 16-bit packing.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "ptx.cuh"
#include "sdpa_internal.h"

namespace sdpa {

using namespace ptx;

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

// 2^e, e in -126 .. 127.
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// E4M3 caches: the exponent v of a row, 2^v being above the scales of the values that it sees.
// Bounds: 2^-v and 2^v are fp32 values, and weights over 2^v stay below 2^15 (scales reach 2^128).  Up to
// +-kNearV, far wider than ordinary values need, v joins the exponents of a row's weights and of its sum, so that
// a weight costs one multiplication by the scale; what v is beyond that takes another one (`wild`).
constexpr int kMinV = -125, kMaxV = 127, kNearV = 60;
__device__ __forceinline__ int near_v(int v) { return min(max(v, -kNearV), kNearV); }
// For a scale given as the bits of its magnitude.
__device__ __forceinline__ int needed_v(uint32_t bits) { return static_cast<int>(bits >> 23) - 126; }

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
  return L.len_q == 0 ? 0 : (L.len_kv + (1 << p.tile_shift) - 1) >> p.tile_shift;
}

// Sum of seq_tiles over sequences [0, n), by a whole warp.
__device__ __forceinline__ long long tiles_before(const DecodeParams& p, int n, int lane) {
  long long t = 0;
  for (int i = lane; i < n; i += 32) t += seq_tiles(p, i);
#pragma unroll
  for (int o = 16; o > 0; o /= 2) t += __shfl_xor_sync(0xffffffffu, t, o);
  return t;
}

// Teams that have a run: no more than tiles, so that none of them is empty.
__device__ __forceinline__ int working_teams(const DecodeParams& p, long long total) {
  return total < p.teams ? static_cast<int>(total) : p.teams;
}

// First tile of team c's run, and the team whose run holds tile t, of `total` tiles over g teams.
__device__ __forceinline__ long long run_start(long long total, int c, int g) { return total * c / g; }
__device__ __forceinline__ int team_of(long long total, long long t, int g) {
  const long long x = (t + 1) * g - 1;
  if (x < (1ll << 31) && total < (1ll << 31)) return static_cast<int>(x) / static_cast<int>(total);
  return static_cast<int>(x / total);
}

// The run of this CTA's team, and the sequence that holds its first tile; by a whole warp.
struct Run {
  long long t, t_end, base;     // tiles [t, t_end) of the batch; base: the first of sequence bi
  int bi;
};

__device__ __forceinline__ Run find_run(const DecodeParams& p, int team, int lane) {
  Run r{0, 0, 0, 0};
  const long long total = tiles_before(p, p.c.b, lane);
  const int g = working_teams(p, total);
  if (team >= g) return r;
  r.t = run_start(total, team, g);
  r.t_end = run_start(total, team + 1, g);
  for (;;) {
    const int i = r.bi + lane;
    const long long n = i < p.c.b ? seq_tiles(p, i) : 0;
    long long incl = n;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const long long x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, r.base + incl > r.t);
    if (hit != 0) {
      const int k = __ffs(hit) - 1;
      r.base += __shfl_sync(0xffffffffu, incl - n, k);
      r.bi += k;
      return r;
    }
    r.base += __shfl_sync(0xffffffffu, incl, 31);
    r.bi += 32;
    if (r.bi >= p.c.b) return Run{0, 0, 0, 0};   // not reached: t < total
  }
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

// Element of lse [b][h_q][s_q], and its value for a maximum m (log2 units) and a sum of 2^(x - m).
__device__ __forceinline__ int64_t lse_offset(const DecodeParams& p, int bi, int hk, int r) {
  return (static_cast<int64_t>(bi) * p.h_q + hk * p.group + r % p.group) * p.s_q + r / p.group;
}
__device__ __forceinline__ float natural_lse(float m, float l) { return (m + __log2f(l)) * 0.6931471805599453f; }

template <int DT>
__device__ __forceinline__ void store_o(void* o, int64_t at, float x) {
  static_cast<uint16_t*>(o)[at] = static_cast<uint16_t>(pack_pair<DT == kBF16>(x, 0.f) & 0xFFFFu);
}

// Infinities and NaNs of the drafted tokens' values: the products ran without them (a hidden
// one times a weight of zero would be NaN); the rows that see them get them here.
template <int D, int CT>
__device__ __noinline__ float add_nonfinite(const DecodeParams& p, int bi, int hk, const SeqLens& L, int r, int d, int key0, int key1,
                               float x) {
  const int token = r / p.group;
  // From the first tile that may hold a new token (all of it may have been cleared; a value added
  // twice is still the same infinity or NaN).
  for (int key = max(key0, (L.len_kv - L.len_q) & ~127); key < key1; ++key) {
    if (!row_sees(p, bi, L, token, key)) continue;
    const int page = __ldg(p.c.page_table + bi * p.c.page_table_stride + key / p.c.page_size);
    if (page < 0 || page >= p.c.num_pages) continue;
    const uint8_t* row = p.c.v + page * p.c.v_st[0] + hk * p.c.v_st[1] + (key % p.c.page_size) * p.c.v_st[2];
    float v;
    if (CT == kE4M3)
      v = __half2float(__ushort_as_half(static_cast<unsigned short>(e4m3x2_to_f16x2(row[d]) & 0xFFFFu))) *
          __ldg(p.c.v_scale + (static_cast<int64_t>(page) * p.c.h_kv + hk) * p.c.page_size + key % p.c.page_size);
    else
      v = unpack_pair<CT == kBF16>(reinterpret_cast<const uint16_t*>(row)[d]).x;
    if (!isfinite(v)) x += v;
  }
  return x;
}

// ---- joining partial results ---------------------------------------------------------------------

// The parts of one block of rows: teams c0 .. c0 + n - 1 (n = 0: no key reaches it).
struct Parts {
  int bi, hk, r0, c0, n;
  int blk, blocks;       // block of rows among those of a sequence
  SeqLens L;
  // Part k among [2 * ctas]: the first holds the sequence's first tile and is its CTA's second part.
  __device__ __forceinline__ int64_t part(int k) const {
    return 2 * (static_cast<int64_t>(c0 + k) * blocks + blk) + (k == 0 ? 1 : 0);
  }
};

// By a whole warp.
__device__ __forceinline__ Parts find_parts(const DecodeParams& p, int unit, int lane) {
  Parts u;
  u.blocks = p.c.h_kv * p.row_tiles;
  u.blk = unit % u.blocks;
  u.bi = unit / u.blocks;
  u.hk = u.blk / p.row_tiles;
  u.r0 = u.blk % p.row_tiles * p.tile_rows;
  u.L = seq_lens(p, u.bi);
  u.c0 = u.n = 0;
  const int n_tiles = seq_tiles(p, u.bi);
  if (n_tiles > 0) {
    long long total = 0, t0 = 0;      // tiles of all sequences, and of those before this one
    for (int i = lane; i < p.c.b; i += 32) {
      const int x = seq_tiles(p, i);
      total += x;
      if (i < u.bi) t0 += x;
    }
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
      total += __shfl_xor_sync(0xffffffffu, total, o);
      t0 += __shfl_xor_sync(0xffffffffu, t0, o);
    }
    const int g = working_teams(p, total);
    u.c0 = team_of(total, t0, g);
    u.n = team_of(total, t0 + n_tiles - 1, g) - u.c0 + 1;
  }
  return u;
}

// Weight of a part (its maximum, its sum) under the common maximum m.  A part without a visible
// key has sum 0 and weighs nothing; where all sums are NaN, m stays -inf and they stay NaN.
__device__ __forceinline__ float part_weight(float2 ml, float m) {
  return ml.y == 0.f ? 0.f : ml.x == -INFINITY ? 1.f : ex2(ml.x - m);
}

// Launches a kernel that may start while the one ahead of it on the stream finishes.
template <typename... A, typename... B>
cudaError_t launch_after(void (*kern)(A...), dim3 grid, dim3 block, cudaStream_t st, B... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace sdpa
