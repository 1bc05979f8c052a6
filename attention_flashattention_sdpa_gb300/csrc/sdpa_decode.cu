// sdpa_decode.cu — attention of one or a few new tokens over a paged cache.
//
// The s_q tokens of a sequence times the query heads of a KV head's group are `rows` query rows
// that share the cache of that KV head.  Work is counted in tiles of 64 keys; the tiles of the whole
// batch are cut into equal runs, so that ragged lengths balance by themselves, and a run may end one
// sequence and begin the next.  A team of CTAs, one for each KV head and block of rows, walks a run
// together: in a slot-major cache the heads of a token lie side by side, and CTAs that read them at
// the same time share DRAM pages (runs over (head, tile) pairs, a head at a time, read 128-byte rows
// at 4.6 instead of 5.2 TB/s and 64-byte rows at 3.7 instead of 5.0).  A sequence that lies in one
// run is finished there; the others leave unnormalised partial results (O, running max, sum) that
// decode_combine_kernel joins, in a fixed order.  Short sequences go to a cluster of CTAs each (and
// block of rows) instead, whose parts meet in its shared memory: one launch.
//
// Bound: reading the cache once.  With 8 rows a key costs 2 x 8 x d multiply-adds for 2 d elements
// read, far below what the tensor cores do in the time of the read; so the products are warp-level
// m16n8k16 MMAs on registers (a 128-row tcgen05 tile would be 15/16 empty and put its P through
// shared memory), and what counts is bytes in flight and few instructions a key: each warp streams
// its own 16-key slices through a ring of cp.async stages and needs no other warp until the end of
// a run.
//
// Keys, and then elements of d, are the 16 rows of the MMAs, and query rows their 8 columns:
//   S^T = K Q^T sums over d in any order, so a lane takes 16 contiguous bytes of its key and Q's
//   fragments are permuted to match;
//   O^T = V^T P^T wants pairs of keys in one register: a lane loads the same 16 bytes of two
//   neighbouring keys and interleaves them with byte permutes.  P^T turns from one product's
//   result layout to the other's operand layout by an 8x8 transposition (movmatrix).
// (Query rows as the 16 rows instead cost twice the MMAs, exponentials and registers for groups
// of up to 8 heads: 209 us against 92 us of reading at 32 sequences of 1K..16K tokens.)
//
// In blocks of 8 rows a weight enters the second product as two 16-bit terms where results keep as many bits as
// one holds, so that O is off by little more than its own rounding (131000 keys, BF16: 0.0017 of it, with one
// term 0.0023): beside the reading the second MMA costs under 0.5%.  One term it is for an E4M3 cache and BF16
// results, whose rounding covers F16's, and for blocks of 16 rows, which it would slow by 2% (BF16, d = 128) to 13%.
//
// E4M3 caches: codes widen exactly to F16; a key's scale multiplies its score, and the scale of
// its value, over 2^v, its weight: w = 2^(s - m) vs / 2^v, O = 2^v sum w v_code / l, l = sum 2^(s - m).  2^v is a running
// maximum as m is one, above the scales that a row sees, so that F16 holds w whatever the scales; l, and LSE,
// depend on Q and K alone.  (log2 vs in the exponent and l = sum w / vs saves a multiplication a score, but is infinite
// for a subnormal vs, and loses ordinary keys beside a vs 2^110 times as large.)  F16's least step is 2^-30 of the
// largest w that these bounds allow, so beside its half step of its own a key's part of O is off by at most
// 2^-31 448 2^v times the row's largest weight: far below E4M3's own rounding of the row with that scale.
//
// Measured, groups of 8 heads, d = 128: 32 sequences of 1000 to 16384 tokens, E4M3, 110 us (5.65 TB/s, 83%
// of a copy; BF16 131000 tokens of one sequence 86 us, 6.25 TB/s, 92%); 1000 tokens of one sequence 7.0 us, of
// which reading is 0.6: the launch, a load's latency for the lengths, the page and the keys, the cluster.
#include <type_traits>

#include "sdpa_decode.cuh"

namespace sdpa {
namespace {

constexpr int kWarps = 4;
constexpr int kSlice = 16;                 // keys of a warp's slice
constexpr int kTile = kWarps * kSlice;     // keys of a tile (decode_plan's tile_shift)
static_assert(kTile == 64);
constexpr int kThreads = kWarps * 32;
constexpr int kMaxCluster = 8;

// NR: blocks of 8 query rows that a CTA works on at once.
template <int D, int CT, int NR>
struct DecCfg {
  static constexpr int ROWS = 8 * NR;
  static constexpr int ES = CT == kE4M3 ? 1 : 2;
  static constexpr int RB = D * ES;                     // bytes of a row
  static constexpr int CH = RB / 16;                    // 16-byte chunks of a row
  static constexpr int EPC = 16 / ES;                   // elements of a chunk
  static constexpr int KCH = D / (4 * EPC);             // chunks of a key that one lane of four reads
  static constexpr int VB = RB >= 128 ? 16 : 8;         // bytes of a value row a lane reads at once
  static constexpr int EPV = VB / ES;                   // and elements
  static constexpr int VJ = D / (8 * EPV);              // such reads of a value row
  static constexpr int NT = D / 16;                     // 16-element tiles of O^T
  static constexpr int SC_BYTES = CT == kE4M3 ? 2 * kSlice * 4 : 0;
  static constexpr int STAGE = 2 * kSlice * RB + SC_BYTES;
  static constexpr int MERGE = kWarps * ROWS * D * 4;   // the warps' partial O at the end of a run
  static constexpr int CTAS = RB > 256 ? 1 : (D * NR > 256 || RB > 128 ? 2 : 3);   // of an SM
  static constexpr int NS_FIT = (232448 / CTAS - 3 * 1024) / (kWarps * STAGE);
  static constexpr int NS = NS_FIT > 6 ? 6 : NS_FIT;
  static constexpr int RING = kWarps * NS * STAGE;
  static constexpr int SMEM = RING > MERGE ? RING : MERGE;
  static constexpr float P_OFF = (CT == kBF16) ? 0.f : 6.f;   // F16 weights: kept away from F16's lowest
  static constexpr float THRESH = 8.f;                  // the running max moves when exceeded by this much
  static_assert(NS >= 2 && NS * 5 <= 32, "ring");
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
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if constexpr (BF) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
}

// Transposes an 8x8 matrix of 16-bit elements held as rows of pairs by the warp.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// ---- main kernel -----------------------------------------------------------------------------

template <int D, int CT, int QT, int NR>
__global__ void __launch_bounds__(kThreads, DecCfg<D, CT, NR>::CTAS) decode_kernel(const __grid_constant__ DecodeParams p) {
  using C = DecCfg<D, CT, NR>;
  constexpr bool E4 = CT == kE4M3;
  constexpr bool BF = CT == kBF16;           // type of the products' operands
  constexpr bool TWO = NR == 1 && (!E4 || QT == kF16);   // weights as two terms
  constexpr int ROWS = C::ROWS, NT = C::NT;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_m[kWarps][ROWS], s_l[kWarps][ROWS];
  __shared__ int s_v[E4 ? kWarps : 1][ROWS];     // E4M3: v of each row
  __shared__ int s_found;
  __shared__ float2 s_part[ROWS];   // clusters: this CTA's maximum and sum of each row

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, c = lane % 4;
  uint8_t* ring = smem + warp * C::NS * C::STAGE;

  // This CTA's block of rows, the same of every sequence, and its team's run; or, in a cluster, its
  // share of one sequence.
  const int cl = p.cluster, unit = cl ? static_cast<int>(blockIdx.x) / cl : static_cast<int>(blockIdx.x);
  const int blocks = p.c.h_kv * p.row_tiles, blk = unit % blocks;
  const int hk = blk / p.row_tiles, r0 = (blk % p.row_tiles) * ROWS;
  griddep_launch_dependents();
  Run run;
  if (cl) {
    const int k = blockIdx.x % cl, n = seq_tiles(p, unit / blocks);
    run = Run{static_cast<long long>(n) * k / cl, static_cast<long long>(n) * (k + 1) / cl, 0, unit / blocks};
    if (threadIdx.x < ROWS) s_part[threadIdx.x] = make_float2(-INFINITY, 0.f);
  } else {
    run = find_run(p, unit / blocks, lane);
  }

  // cp.async: lane's chunk of rows (lane / CH) + x * RPX of a slice.
  constexpr int RPX = 32 / C::CH;
  const int ld_row = lane / C::CH, ld_ch = lane % C::CH;

  while (run.t < run.t_end) {
    const int bi = run.bi;
    const SeqLens L = seq_lens(p, bi);
    const int n_tiles = seq_tiles(p, bi);
    if (run.t >= run.base + n_tiles) {
      run.base += n_tiles;
      ++run.bi;
      continue;
    }
    const int tile0 = static_cast<int>(run.t - run.base);
    const int tile1 = static_cast<int>(min(static_cast<long long>(n_tiles), run.t_end - run.base));
    const int off = L.len_kv - L.len_q;           // position of the first new token
    const bool masked = p.causal != 0 || p.tree_mask != nullptr;

    // ---- the ring: slice i of this warp is keys (tile0 + i) * 64 + warp * 16 ------------------
    const int n_slices = tile1 - tile0;
    const int32_t* pages = p.c.page_table + bi * p.c.page_table_stride;
    const uint8_t* k_lane = p.c.k + hk * p.c.k_st[1] + ld_row * p.c.k_st[2] + ld_ch * 16;
    const uint8_t* v_lane = p.c.v + hk * p.c.v_st[1] + ld_row * p.c.v_st[2] + ld_ch * 16;
    int my_page = -1, my_slot = 0;   // lane i: page and slot of slice i of the last 32 asked for
    unsigned valid_hist = 0;         // 5 bits a stage: keys of its slice that exist
    auto load = [&](int i) {
      if (i < n_slices) {
        if (i % 32 == 0) {
          const int key = (tile0 + i + lane) * kTile + warp * kSlice;
          my_page = -1;
          if (i + lane < n_slices && key < L.len_kv) {
            const int col = key / p.c.page_size;
            my_slot = key - col * p.c.page_size;
            my_page = __ldg(pages + col);
            if (my_page >= p.c.num_pages) my_page = -1;
          }
        }
        const int page = __shfl_sync(0xffffffffu, my_page, i % 32);
        const int slot = __shfl_sync(0xffffffffu, my_slot, i % 32);
        const int left = L.len_kv - ((tile0 + i) * kTile + warp * kSlice);
        const int valid = page < 0 ? 0 : min(max(left, 0), kSlice);
        const uint8_t* kp = k_lane + page * p.c.k_st[0] + slot * p.c.k_st[2];
        const uint8_t* vp = v_lane + page * p.c.v_st[0] + slot * p.c.v_st[2];
        const int stage = i % C::NS;
        const uint32_t dst = smem_u32(ring) + stage * C::STAGE;
        if (valid == kSlice) {
#pragma unroll
          for (int x = 0; x < kSlice / RPX; ++x) {
            const uint32_t at = dst + (x * RPX + ld_row) * C::RB + swz<C::CH>(x * RPX + ld_row, ld_ch) * 16;
            cp_async16(at, kp + x * RPX * p.c.k_st[2], true);
            cp_async16(at + kSlice * C::RB, vp + x * RPX * p.c.v_st[2], true);
          }
        } else {
#pragma unroll
          for (int x = 0; x < kSlice / RPX; ++x) {
            const bool on = x * RPX + ld_row < valid;
            const uint32_t at = dst + (x * RPX + ld_row) * C::RB + swz<C::CH>(x * RPX + ld_row, ld_ch) * 16;
            cp_async16(at, on ? kp + x * RPX * p.c.k_st[2] : p.c.k, on);
            cp_async16(at + kSlice * C::RB, on ? vp + x * RPX * p.c.v_st[2] : p.c.v, on);
          }
        }
        if constexpr (E4) {
          if (lane < 8) {
            const bool on = valid > 0;
            const float* src = (lane < 4 ? p.c.k_scale : p.c.v_scale) +
                               (static_cast<int64_t>(page) * p.c.h_kv + hk) * p.c.page_size + slot + (lane % 4) * 4;
            cp_async16(dst + 2 * kSlice * C::RB + lane * 16, on ? src : p.c.k_scale, on);
          }
        }
        valid_hist = (valid_hist & ~(31u << (5 * stage))) | (static_cast<unsigned>(valid) << (5 * stage));
      }
      cp_commit();
    };
    for (int i = 0; i < C::NS - 1; ++i) load(i);

    // ---- Q^T fragments (columns: rows g of each block of 8), permuted to the order in which
    // lanes read keys ----------------------------------------------------------------------------
    uint32_t qf[NR][D / 8];
    float cs[NR][2];           // factor on the scores of this lane's result columns, rows 2c, 2c + 1
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      const int r = r0 + n * 8 + g;
      const bool on = r < p.rows && r / p.group < L.len_q;
      const uint16_t* row = static_cast<const uint16_t*>(p.q) + (on ? row_offset(p, p.q_st, bi, hk, r) : 0);
      uint32_t (&w)[D / 8] = qf[n];
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
      cs[n][0] = cs[n][1] = p.scale_log2;
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
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const float2 f = unpack_pair<true>(w[i]);
          w[i] = pack_pair<false>(f.x * up, f.y * up);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)   // row 2c + u is held by lanes 4 (2c + u) ..
          cs[n][u] *= __uint_as_float(static_cast<uint32_t>(127 - __shfl_sync(0xffffffffu, sh, 4 * (2 * c + u))) << 23);
      }
    }

    float o[NR][NT][4];
    float m_ref[NR][2], l[NR][2];
    float v_min = 0.f;         // E4M3: 2^v of the warp's row with the least
    bool wild = E4;            // E4M3: v of some row is beyond +-kNearV
    float nm[NR][2];           // what a row's scores take to the exponent of their weights
#pragma unroll
    for (int n = 0; n < NR; ++n) {
#pragma unroll
      for (int i = 0; i < NT; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
      m_ref[n][0] = m_ref[n][1] = -INFINITY;
      nm[n][0] = nm[n][1] = E4 ? kNearV : 0.f;
      l[n][0] = l[n][1] = 0.f;
    }
    // E4M3: v of row 2c + u of block n (written by every lane that holds the row; seldom read or written).
    int* const v_row = s_v[E4 ? warp : 0] + 2 * c;
    if constexpr (E4) {
      for (int r = lane; r < ROWS; r += 32) s_v[warp][r] = kMinV;
      __syncwarp();
    }
    bool found = false;
    if (threadIdx.x == 0) s_found = 0;

    for (int i = 0; i < n_slices; ++i) {
      cp_wait<C::NS - 2>();
      __syncwarp();             // slice i has landed, and every lane is done with slice i - 1
      load(i + C::NS - 1);
      const int stage = i % C::NS;
      const uint8_t* st = ring + stage * C::STAGE;
      const int valid = (valid_hist >> (5 * stage)) & 31;
      if (valid == 0) continue;
      const int key0 = (tile0 + i) * kTile + warp * kSlice;
      const bool tail = masked && key0 + kSlice > off;

      // ---- S^T = K Q^T; lane: keys g, g + 8 by rows 2c, 2c + 1 ------------------------------------
      float s[NR][4];
      {
        float s2[NR][4];     // two sums, so that the MMAs of one need not wait for each other
#pragma unroll
        for (int n = 0; n < NR; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = s2[n][0] = s2[n][1] = s2[n][2] = s2[n][3] = 0.f;
#pragma unroll
        for (int j = 0; j < C::KCH; ++j) {
          const uint4 ka = *reinterpret_cast<const uint4*>(st + g * C::RB + swz<C::CH>(g, j * 4 + c) * 16);
          const uint4 kb = *reinterpret_cast<const uint4*>(st + (g + 8) * C::RB + swz<C::CH>(g + 8, j * 4 + c) * 16);
          const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
          if constexpr (E4) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t a0 = e4m3x2_to_f16x2(wa[e] & 0xFFFFu), a1 = e4m3x2_to_f16x2(wb[e] & 0xFFFFu);
              const uint32_t a2 = e4m3x2_to_f16x2(wa[e] >> 16), a3 = e4m3x2_to_f16x2(wb[e] >> 16);
#pragma unroll
              for (int n = 0; n < NR; ++n)
                mma16816<BF>(e % 2 ? s2[n] : s[n], a0, a1, a2, a3, qf[n][8 * j + 2 * e], qf[n][8 * j + 2 * e + 1]);
            }
          } else {
#pragma unroll
            for (int n = 0; n < NR; ++n) {
              mma16816<BF>(s[n], wa[0], wb[0], wa[1], wb[1], qf[n][4 * j], qf[n][4 * j + 1]);
              mma16816<BF>(s2[n], wa[2], wb[2], wa[3], wb[3], qf[n][4 * j + 2], qf[n][4 * j + 3]);
            }
          }
        }
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][e] += s2[n][e];
      }

      // ---- scale (log2 units), mask ----------------------------------------------------------------
      float vs[2];               // E4M3: scales of this lane's keys' values
      if constexpr (E4) {
        const float* sc = reinterpret_cast<const float*>(st + 2 * kSlice * C::RB);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float ks = sc[g + 8 * u];
          vs[u] = sc[kSlice + g + 8 * u];
#pragma unroll
          for (int n = 0; n < NR; ++n) {
            s[n][2 * u] *= cs[n][0] * ks;
            s[n][2 * u + 1] *= cs[n][1] * ks;
          }
        }
      } else {
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][e] *= cs[n][e % 2];
      }
      uint32_t hidden = 0;        // bit 4 n + e
      if (valid < kSlice || tail) {
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int kk = g + 8 * (e / 2), r = r0 + n * 8 + 2 * c + e % 2, token = r / p.group;
            bool see = kk < valid;
            if (see && tail && r < p.rows && token < L.len_q) see = row_sees(p, bi, L, token, key0 + kk);
            if (!see) {
              s[n][e] = -INFINITY;
              hidden |= 1u << (4 * n + e);
            }
          }
      }

      // ---- running max: moved, for the lanes of a row together, when a score exceeds it by 2^8 -------
      bool over = false;
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) over |= s[n][e] > m_ref[n][e % 2] + C::THRESH;
      if constexpr (E4) over |= vs[0] > v_min || vs[1] > v_min;
      const bool move = __any_sync(0xffffffffu, over);
      if (move) {
#pragma unroll
        for (int n = 0; n < NR; ++n) {
          float alpha[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            float mx = fmaxf(s[n][u], s[n][u + 2]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            alpha[u] = 1.f;
            if (mx > m_ref[n][u] + C::THRESH) {
              alpha[u] = ex2(m_ref[n][u] - mx);
              m_ref[n][u] = mx;
              nm[n][u] = C::P_OFF - mx - (E4 ? near_v(v_row[n * 8 + u]) : 0);
            }
            l[n][u] *= alpha[u];
          }
#pragma unroll
          for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][x][e] *= alpha[e % 2];
        }
      }
      // ---- 2^v: moved to two to four times the largest finite scale that a row sees when that exceeds it (an
      // infinite scale or a NaN spoils O as it is) ---------------------------------------------------------
      if constexpr (E4) {
        if (move && __any_sync(0xffffffffu, vs[0] > v_min || vs[1] > v_min)) {
          uint32_t top[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) top[k] = vs[k] < INFINITY ? __float_as_uint(fabsf(vs[k])) : 0u;
          const uint32_t of_all = __reduce_max_sync(0xffffffffu, max(top[0], top[1]));
          const bool same = __all_sync(0xffffffffu, hidden == 0);       // every row sees every key
          int least = kMaxV, most = kMinV;
#pragma unroll
          for (int n = 0; n < NR; ++n) {
            float alpha[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              uint32_t t = of_all;
              if (!same) {
                t = max((hidden >> (4 * n + u)) & 1u ? 0u : top[0], (hidden >> (4 * n + u + 2)) & 1u ? 0u : top[1]);
                t = max(t, __shfl_xor_sync(0xffffffffu, t, 4));
                t = max(t, __shfl_xor_sync(0xffffffffu, t, 8));
                t = max(t, __shfl_xor_sync(0xffffffffu, t, 16));
              }
              const int before = v_row[n * 8 + u], need = needed_v(t);
              const int now = before >= need ? before : min(need + 1, kMaxV), step = near_v(before) - near_v(now);
              alpha[u] = pow2(max(before - now, -126));
              l[n][u] *= pow2(step);
              nm[n][u] += static_cast<float>(step);
              __syncwarp();
              v_row[n * 8 + u] = now;
              least = min(least, now);
              most = max(most, now);
            }
            if (i > 0) {
#pragma unroll
              for (int x = 0; x < NT; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][x][e] *= alpha[e % 2];
            }
          }
#pragma unroll
          for (int x = 1; x < 4; x *= 2) {
            least = min(least, __shfl_xor_sync(0xffffffffu, least, x));
            most = max(most, __shfl_xor_sync(0xffffffffu, most, x));
          }
          __syncwarp();
          v_min = pow2(least);
          wild = least < -kNearV || most > kNearV;
        }
      }
      // ---- weights, sums, P^T ------------------------------------------------------------------------
      uint32_t pb[NR][2], pl[TWO ? NR : 1][2];
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[n][e] = ex2(s[n][e] + nm[n][e % 2]);
          l[n][e % 2] += s[n][e];
          if constexpr (E4) s[n][e] *= vs[e / 2];
        }
      if constexpr (E4) {
        if (wild || hidden) {
#pragma unroll
          for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int v = v_row[n * 8 + e % 2];
              s[n][e] *= pow2(near_v(v) - v);
              if ((hidden >> (4 * n + e)) & 1u) s[n][e] = 0.f;     // whatever the scale of a hidden key
            }
        }
      }
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t w = pack_pair<BF>(s[n][2 * u], s[n][2 * u + 1]);
          pb[n][u] = transpose8x8(w);
          if constexpr (TWO) {
            const float2 f = unpack_pair<BF>(w);
            pl[n][u] = transpose8x8(pack_pair<BF>(s[n][2 * u] - f.x, s[n][2 * u + 1] - f.y));
          }
        }

      // ---- O^T += V^T P^T; lane's part of a value: d = (8 j + g) * EPV + 0 .. EPV - 1 --------------------
      auto product = [&](auto clear) {
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
          for (int x = 0; x < C::EPV; x += 2) {   // elements x, x + 1: rows g, g + 8 of one tile of O^T
            uint32_t a[4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if constexpr (E4) {
                // bytes x, x + 1 of both keys: (key, key + 1) of x in the low half, of x + 1 in the high
                const uint32_t two = prmt(v[2 * h][x / 4], v[2 * h + 1][x / 4], x % 4 ? 0x7362u : 0x5140u);
                a[2 * h] = e4m3x2_to_f16x2(two & 0xFFFFu);
                a[2 * h + 1] = e4m3x2_to_f16x2(two >> 16);
              } else {
                a[2 * h] = prmt(v[2 * h][x / 2], v[2 * h + 1][x / 2], 0x5410u);
                a[2 * h + 1] = prmt(v[2 * h][x / 2], v[2 * h + 1][x / 2], 0x7632u);
              }
            }
            if constexpr (decltype(clear)::value) {
#pragma unroll
              for (int h = 0; h < 4; ++h) a[h] = finite_pair<BF>(a[h], found);
            }
#pragma unroll
            for (int n = 0; n < NR; ++n) {
              mma16816<BF>(o[n][(j * C::EPV + x) / 2], a[0], a[1], a[2], a[3], pb[n][0], pb[n][1]);
              if constexpr (TWO) mma16816<BF>(o[n][(j * C::EPV + x) / 2], a[0], a[1], a[2], a[3], pl[n][0], pl[n][1]);
            }
          }
        }
      };
      if (tail) product(std::true_type{});
      else product(std::false_type{});
    }
    cp_wait<0>();

    // ---- the four warps' results meet -----------------------------------------------------------
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if constexpr (E4) l[n][u] *= pow2(near_v(v_row[n * 8 + u]));
#pragma unroll
        for (int x = 4; x < 32; x *= 2) l[n][u] += __shfl_xor_sync(0xffffffffu, l[n][u], x);
        if (g == 0) {
          s_m[warp][n * 8 + 2 * c + u] = m_ref[n][u];
          s_l[warp][n * 8 + 2 * c + u] = l[n][u];
        }
      }
    __syncthreads();
    if (found) s_found = 1;
    float* merge = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int r = n * 8 + 2 * c + u;
        float big = s_m[0][r];
        for (int w = 1; w < kWarps; ++w) big = fmaxf(big, s_m[w][r]);
        // A warp that saw no key (sum 0) adds nothing; a sum of NaN with no maximum stays NaN.
        const bool none = m_ref[n][u] == -INFINITY;
        float f = none ? 1.f : ex2(m_ref[n][u] - big);
        if constexpr (E4) {
          int v = s_v[0][r];
          for (int w = 1; w < kWarps; ++w) v = max(v, s_v[w][r]);
          f *= pow2(max(s_v[warp][r] - v, -126));
        }
        float* row = merge + (warp * ROWS + r) * D + g * C::EPV;
#pragma unroll
        for (int j = 0; j < C::VJ; ++j)
#pragma unroll
          for (int x = 0; x < C::EPV; x += 4) {
            const int i = (j * C::EPV + x) / 2;
            float4 q4 = make_float4(o[n][i][u] * f, o[n][i][u + 2] * f, o[n][i + 1][u] * f, o[n][i + 1][u + 2] * f);
            if (l[n][u] == 0.f) q4 = make_float4(0.f, 0.f, 0.f, 0.f);
            *reinterpret_cast<float4*>(row + j * 8 * C::EPV + x) = q4;
          }
      }
    __syncthreads();
    const bool whole = tile0 == 0 && tile1 == n_tiles;
    const int part = 2 * blockIdx.x + (tile0 == 0 ? 1 : 0);
    const bool fix = s_found != 0;
    const int live = min(ROWS, p.rows - r0);
    for (int idx = threadIdx.x; idx < live * (D / 4); idx += kThreads) {
      const int r = idx / (D / 4), d = idx % (D / 4) * 4;
      float mb = s_m[0][r], lb = 0.f;
      for (int w = 1; w < kWarps; ++w) mb = fmaxf(mb, s_m[w][r]);
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 y = *reinterpret_cast<const float4*>(merge + (w * ROWS + r) * D + d);
        x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
        if (s_l[w][r] != 0.f) lb += s_l[w][r] * (s_m[w][r] == -INFINITY ? 1.f : ex2(s_m[w][r] - mb));
      }
      const int row = r0 + r, token = row / p.group;
      const bool on = token < L.len_q;
      if (fix && on) {
        const int k0 = tile0 * kTile, k1 = min(tile1 * kTile, L.len_kv);
        x.x = add_nonfinite<D, CT>(p, bi, hk, L, row, d, k0, k1, x.x);
        x.y = add_nonfinite<D, CT>(p, bi, hk, L, row, d + 1, k0, k1, x.y);
        x.z = add_nonfinite<D, CT>(p, bi, hk, L, row, d + 2, k0, k1, x.z);
        x.w = add_nonfinite<D, CT>(p, bi, hk, L, row, d + 3, k0, k1, x.w);
      }
      if constexpr (E4) {
        // 2^v joins.  Where O would pass fp32's range with it, O and the sum are brought down and the
        // reference up, to a sum of 2^-12: sums over the parts then stay in range where the values do.
        int v = s_v[0][r];
        for (int w = 1; w < kWarps; ++w) v = max(v, s_v[w][r]);
        float up = pow2(v);
        if (v > kNearV && lb > 0.f && lb < INFINITY) {
          const int e = static_cast<int>(__float_as_uint(lb) >> 23) - 127 + 12;
          up *= pow2(-e);
          lb *= pow2(-e);
          mb += static_cast<float>(e);
        }
        x = make_float4(x.x * up, x.y * up, x.z * up, x.w * up);
      }
      if (cl) {      // over the first warp's part, which no other thread reads here
        *reinterpret_cast<float4*>(merge + r * D + d) = x;
        if (d == 0) s_part[r] = make_float2(mb, lb);
      } else if (!whole) {
        const int64_t at = static_cast<int64_t>(part) * ROWS + r;
        *reinterpret_cast<float4*>(p.part_o + at * D + d) = x;
        if (d == 0) *reinterpret_cast<float2*>(p.part_ml + 2 * at) = make_float2(mb, lb);
      } else {
        const bool none = !on || lb == 0.f;
        const float inv = none ? 0.f : 1.f / lb;
        if (none) x = make_float4(0.f, 0.f, 0.f, 0.f);
        uint2 w;
        w.x = pack_pair<QT == kBF16>(x.x * inv, x.y * inv);
        w.y = pack_pair<QT == kBF16>(x.z * inv, x.w * inv);
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + row_offset(p, p.o_st, bi, hk, row) + d) = w;
        if (p.lse && d == 0)
          p.lse[lse_offset(p, bi, hk, row)] = none ? -INFINITY : natural_lse(mb - C::P_OFF, lb);
      }
    }
    __syncthreads();   // the ring and the exchange arrays are free again
    run.t = run.base + tile1;
  }

  // ---- a cluster's results meet in shared memory, its CTAs joining a share of the elements each -----
  if (cl) {
    __syncwarp();
    cluster_sync_all();
    const int bi = unit / blocks, live = min(ROWS, p.rows - r0);
    const SeqLens L = seq_lens(p, bi);
    for (int idx = (blockIdx.x % cl) * kThreads + threadIdx.x; idx < live * (D / 4); idx += cl * kThreads) {
      const int r = idx / (D / 4), d = idx % (D / 4) * 4;
      float2 ml[kMaxCluster];
      float4 v[kMaxCluster];
#pragma unroll
      for (int k = 0; k < kMaxCluster; ++k) {
        ml[k] = make_float2(-INFINITY, 0.f);
        v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k < cl) {
          ml[k] = ld_cluster_f2(&s_part[r], k);
          v[k] = ld_cluster_f4(smem + (r * D + d) * 4, k);
        }
      }
      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int k = 0; k < kMaxCluster; ++k)
        if (ml[k].y != 0.f) m = fmaxf(m, ml[k].x);
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kMaxCluster; ++k) {
        const float f = part_weight(ml[k], m);     // 0 where a CTA had no key: its part was not written
        l += ml[k].y * f;
        x.x += f == 0.f ? 0.f : v[k].x * f;
        x.y += f == 0.f ? 0.f : v[k].y * f;
        x.z += f == 0.f ? 0.f : v[k].z * f;
        x.w += f == 0.f ? 0.f : v[k].w * f;
      }
      const int row = r0 + r;
      const bool none = row / p.group >= L.len_q || l == 0.f;
      const float inv = none ? 0.f : 1.f / l;
      const uint2 w = none ? make_uint2(0, 0)
                           : make_uint2(pack_pair<QT == kBF16>(x.x * inv, x.y * inv), pack_pair<QT == kBF16>(x.z * inv, x.w * inv));
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + row_offset(p, p.o_st, bi, hk, row) + d) = w;
      if (p.lse && d == 0) p.lse[lse_offset(p, bi, hk, row)] = none ? -INFINITY : natural_lse(m - C::P_OFF, l);
    }
    __syncwarp();
    cluster_sync_all();    // nobody leaves while its shared memory is read
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
  const int per_unit = min(p.rows, p.tile_rows);
  const Parts u = find_parts(p, blockIdx.x / per_unit, lane);
  const int r = blockIdx.x % per_unit, row = u.r0 + r, token = row / p.group;
  griddep_wait();   // (by every CTA, so that this grid never ends before the one it follows)
  if (u.n == 1 || row >= p.rows) return;     // finished by that CTA
  float m = -INFINITY;
  for (int k = lane; k < u.n; k += 32) {
    const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + 2 * (u.part(k) * p.tile_rows + r));
    if (ml.y != 0.f) m = fmaxf(m, ml.x);
  }
#pragma unroll
  for (int o = 16; o > 0; o /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float x[EL], l = 0.f;
#pragma unroll
  for (int e = 0; e < EL; ++e) x[e] = 0.f;
  for (int k0 = warp; k0 < u.n; k0 += 8 * kWarps) {
    float f[8], v[8][EL];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int k = k0 + i * kWarps;
      f[i] = 0.f;
#pragma unroll
      for (int e = 0; e < EL; ++e) v[i][e] = 0.f;
      if (k < u.n) {
        const int64_t at = u.part(k) * p.tile_rows + r;
        const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + 2 * at);
        const float* src = p.part_o + at * D + lane * EL;
#pragma unroll
        for (int e = 0; e < EL; e += 2) {
          const float2 w = *reinterpret_cast<const float2*>(src + e);
          v[i][e] = w.x;
          v[i][e + 1] = w.y;
        }
        f[i] = part_weight(ml, m);
        l += ml.y * f[i];
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < EL; ++e) x[e] += f[i] == 0.f ? 0.f : v[i][e] * f[i];
  }
#pragma unroll
  for (int e = 0; e < EL; ++e) s_sum[warp][lane * EL + e] = x[e];
  if (lane == 0) s_l[warp] = l;
  __syncthreads();
  l = (s_l[0] + s_l[1]) + (s_l[2] + s_l[3]);
  const bool none = token >= u.L.len_q || l == 0.f;
  const int64_t at = row_offset(p, p.o_st, u.bi, u.hk, row);
  for (int d = threadIdx.x; d < D; d += kThreads)
    store_o<QT>(p.o, at + d, none ? 0.f : ((s_sum[0][d] + s_sum[1][d]) + (s_sum[2][d] + s_sum[3][d])) / l);
  if (p.lse && threadIdx.x == 0) p.lse[lse_offset(p, u.bi, u.hk, row)] = none ? -INFINITY : natural_lse(m - p_off, l);
}

template <int D, int CT, int QT, int NR>
cudaError_t launch_t(const DecodeParams& p, cudaStream_t st) {
  using C = DecCfg<D, CT, NR>;
  auto kern = decode_kernel<D, CT, QT, NR>;
  cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kern), C::SMEM);
  if (e != cudaSuccess) return e;
  if (p.cluster) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = p.cluster;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
  }
  kern<<<p.ctas, kThreads, C::SMEM, st>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_after(decode_combine_kernel<D, QT>,
                      dim3(static_cast<unsigned>(p.c.b) * p.c.h_kv * p.row_tiles * (p.rows < p.tile_rows ? p.rows : p.tile_rows)),
                      dim3(kThreads), st, p, C::P_OFF);
}

template <int D, int CT, int QT>
cudaError_t launch_r(const DecodeParams& p, cudaStream_t st) {
  return p.tile_rows == 8 ? launch_t<D, CT, QT, 1>(p, st) : launch_t<D, CT, QT, 2>(p, st);
}

template <int D>
cudaError_t launch_d(const DecodeParams& p, int qt, int ct, cudaStream_t st) {
  if (qt == kBF16) return ct == kE4M3 ? launch_r<D, kE4M3, kBF16>(p, st) : launch_r<D, kBF16, kBF16>(p, st);
  return ct == kE4M3 ? launch_r<D, kE4M3, kF16>(p, st) : launch_r<D, kF16, kF16>(p, st);
}

template <int D>
int ctas_of_sm(int tile_rows, bool e4m3) {
  if (e4m3) return tile_rows == 8 ? DecCfg<D, kE4M3, 1>::CTAS : DecCfg<D, kE4M3, 2>::CTAS;
  return tile_rows == 8 ? DecCfg<D, kF16, 1>::CTAS : DecCfg<D, kF16, 2>::CTAS;
}

}  // namespace

void decode_plan(DecodeParams* p, int d, int ct, int num_sms) {
  // Many rows: measured at 8 x 8192 tokens, 8 KV heads of 128, blocks of 8 or 16 rows against the wide
  // ones: E4M3 66 us against 79 for 32 rows, 89 against 80 for 40; BF16 62 against 58 for 24 (d = 64:
  // E4M3 48 against 55, 63 against 55; BF16 42 against 37).
  p->wide = d <= 128 && p->rows > (ct == kE4M3 ? 32 : 16);
  p->tile_rows = p->wide ? 256 : p->rows <= 8 ? 8 : 16;
  p->row_tiles = (p->rows + p->tile_rows - 1) / p->tile_rows;
  p->tile_shift = p->wide ? 7 : 6;
  const bool e4 = ct == kE4M3;
  const int per_sm = p->wide ? 1 : d == 64 ? ctas_of_sm<64>(p->tile_rows, e4) : d == 128 ? ctas_of_sm<128>(p->tile_rows, e4)
                                                                                         : ctas_of_sm<256>(p->tile_rows, e4);
  // Teams: as many as fill the GPU once with the blocks of rows of a sequence, or, where whole teams
  // leave over a tenth of it idle, the count among up to four rounds (two of wide blocks, whose
  // parts are large) that leaves least.
  const int blocks = p->c.h_kv * p->row_tiles, top = per_sm * num_sms;
  auto used = [&](long long teams) {
    const long long n = teams * blocks;
    return static_cast<double>(n) / static_cast<double>((n + top - 1) / top * top);
  };
  long long teams = top / blocks > 0 ? top / blocks : 1;
  if (used(teams) < 0.9) {
    for (long long k = teams + 1; k * blocks <= (p->wide ? 2ll : 4ll) * top; ++k)
      if (used(k) > used(teams) + 0.02) teams = k;
  }
  const long long keys = 1ll << p->tile_shift;
  const long long tiles = static_cast<long long>(p->c.b) * ((p->c.max_len + keys - 1) / keys);
  p->teams = static_cast<int>(teams < tiles ? teams : tiles);
  p->ctas = p->teams * blocks;
  // Short sequences (by the page table's columns: lengths are on the device): a cluster of CTAs for
  // each sequence and block of rows, which join in shared memory and spare the second launch (about
  // the time of 10 tiles), where all of them fit on the GPU at once (clusters of CTAs that fill an SM
  // leave some SMs out) and no CTA gets more than 20 tiles, or 10 more than a team would.  Measured, clusters
  // against teams, 32 heads over 8 of 128, BF16: 1 x 1000 tokens 7.0 against 7.2 us, 4 x 1000 8.2 against
  // 9.7, 4 x 4000 16.6 against 19.5, 32 x 10..1000 19.5 against 22.1; 1 x 8000 14.8 against 13.6.  A call from
  // Python, which pays for two launches, takes 11 us against 13.
  p->cluster = 0;
  if (!p->wide) {
    const long long cap = (p->c.max_len + keys - 1) / keys, units = static_cast<long long>(p->c.b) * blocks;
    const long long room = per_sm == 1 ? top * 3 / 4 : top, of_team = p->c.b * cap / (top / blocks > 0 ? top / blocks : 1);
    int cl = 1;
    while (cl < kMaxCluster && cl < cap && units * cl * 2 <= room) cl *= 2;
    const long long mine = (cap + cl - 1) / cl;
    if (units * cl <= room && mine <= 20 && mine <= of_team + 10) {
      p->cluster = cl;
      p->ctas = static_cast<int>(units) * cl;
    }
  }
}

size_t decode_workspace_bytes(const DecodeParams& p, int d, size_t* ml_offset) {
  // A single team finishes every sequence itself and leaves no parts.
  const size_t parts = p.teams > 1 && !p.cluster ? 2 * static_cast<size_t>(p.ctas) * p.tile_rows : 0;
  if (ml_offset) *ml_offset = parts * d * 4;
  return (parts * d * 4 + parts * 8 + 256) & ~size_t(255);
}

cudaError_t launch_decode(const DecodeParams& p, int d, int qt, int ct, cudaStream_t st) {
  if (d == 64) return launch_d<64>(p, qt, ct, st);
  if (d == 128) return launch_d<128>(p, qt, ct, st);
  if (d == 256) return launch_d<256>(p, qt, ct, st);
  return cudaErrorInvalidValue;
}

}  // namespace sdpa
