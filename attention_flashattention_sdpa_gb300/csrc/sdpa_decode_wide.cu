// sdpa_decode_wide.cu — attention over a paged cache for many query rows a KV head: drafted trees
// and short chunks whose s_q tokens times the heads of a group fill tcgen05 tiles.
//
// The split of the batch is that of sdpa_decode.cu with tiles of 128 keys and blocks of 256 rows:
// one persistent CTA an SM walks an equal run of tiles, segment by segment (a segment: the part
// of its run in one (sequence, KV head, block of rows)).  Roles:
//   warp 0       pages and TMA: K and V tiles, box by box (a box lies in one page) into a ring;
//                boxes of missing pages and behind the sequence are filled with zeros.
//   warp 1       MMA issuer: S = Q K^T into TMEM, O += P V with P read from TMEM.
//   warps 4-11   two softmax warpgroups, one for each 128-row tile; thread r owns row r: loads it
//                into shared memory, the running max and sum, P, and the segment's results.
//   warps 12-15  E4M3 caches: widen K to F16 on its way from the TMA's stage to the ring (and warps
//                16-19 V); 16-bit caches: clear, in V tiles that end behind the sequence or hold
//                drafted tokens, rows that do not exist and values that are not finite (a weight of
//                zero does not hide a NaN in a product).
//
// E4M3: a tile's codes are multiplied by scale / 2^E (E: the exponent of the tile's largest scale)
// as a sum of two F16 factors, so one rounding to F16's 11 bits is left, whatever the scales; 2^E
// of K joins the factor on the scores and 2^E of V the exponent, both once a tile.
//
// Bound: the tensor cores (4 x 128 x 128 x d MMAs a block of two tiles) and the exponentials, as
// the prompt's forward pass; reading the cache once bounds it for 64 rows and fewer.
#include "sdpa_decode.cuh"

namespace sdpa {
namespace {

constexpr int kKeys = 128;
constexpr int kLog2Keys = 7;

template <int D, int CT>
struct WideCfg {
  static constexpr bool E4 = CT == kE4M3;
  static constexpr int THREADS = E4 ? 640 : 512;
  // Registers of the producer's, the softmax and the widening or clearing warpgroups, out of 96
  // (E4M3) or 128 a thread at launch: 64 + 2 x 152 + 2 x 56 = 5 x 96, 64 + 2 x 184 + 80 = 4 x 128.
  static constexpr int REGS0 = 64, REGS_SOFTMAX = E4 ? 152 : 184, REGS_WIDEN = E4 ? 56 : 80;
  static constexpr int TILE = 128 * D * 2;                // a 16-bit tile of 128 rows
  static constexpr int RAW = E4 ? 128 * D : 0;            // an E4M3 tile as loaded
  static constexpr int NCHUNK = D / 64;                   // 128-byte columns of a 16-bit tile
  static constexpr int Q_BYTES = 2 * TILE;
  static constexpr int NS = D == 128 ? (E4 ? 3 : 4) : 6;  // ring of 16-bit tiles
  static constexpr int NRAW = E4 ? 4 : 0;
  static constexpr int SMEM = Q_BYTES + NS * TILE + NRAW * RAW + 1024;
  static constexpr int KSTEPS = D / 16;
  static constexpr int O_COL0 = 256;
  static constexpr float P_OFF = CT == kBF16 ? 0.f : 6.f;
  static constexpr float THRESH = 8.f;
  static_assert(SMEM + 1536 <= 232448, "shared memory");
  static_assert(O_COL0 + 2 * D <= 512, "TMEM");
};

struct alignas(8) WideBarriers {
  uint64_t q_full[2];
  uint64_t raw_full[4], raw_empty[4];
  uint64_t kv_full[6], kv_empty[6], kv_clean[6];
  uint64_t s_full[2], p_full[2], o_full[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

// A part of this CTA's run: tiles [tile0, tile1) of one (sequence, KV head, block of rows).
struct Segment {
  int bi, hk, r0, n_tiles, tile0, tile1, off;
  SeqLens L;
};

// The run's position; every role walks it by itself.
struct Walk {
  long long t, t_end, base;
  int bi;
  __device__ __forceinline__ bool next(const DecodeParams& p, Segment& g) {
    const int per_seq = p.c.h_kv * p.row_tiles;
    while (t < t_end) {
      const int n = seq_tiles(p, bi);
      if (t >= base + static_cast<long long>(n) * per_seq) {
        base += static_cast<long long>(n) * per_seq;
        ++bi;
        continue;
      }
      const int blk = static_cast<int>((t - base) / n);
      const long long t0 = base + static_cast<long long>(blk) * n;
      g.bi = bi;
      g.hk = blk / p.row_tiles;
      g.r0 = blk % p.row_tiles * 256;
      g.n_tiles = n;
      g.tile0 = static_cast<int>(t - t0);
      g.tile1 = static_cast<int>(min(static_cast<long long>(n), t_end - t0));
      g.L = seq_lens(p, bi);
      g.off = g.L.len_kv - g.L.len_q;
      t = t0 + g.tile1;
      return true;
    }
    return false;
  }
};

// Whether V's tile of a 16-bit cache has to be cleared of what no row may meet.
__device__ __forceinline__ bool needs_cleaning(const DecodeParams& p, const Segment& g, int tile) {
  const int end = (tile + 1) * kKeys;
  return end > g.L.len_kv || ((p.causal || p.tree_mask) && end > g.off);
}

// Exponent e of a positive fp32 given as bits (2^e <= x < 2^(e+1)), kept where 2^e and 2^-e are normal.
__device__ __forceinline__ int exponent_of(uint32_t bits) { return min(max(static_cast<int>(bits >> 23) - 127, -100), 100); }
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// Bits of scale s where the key exists and the scale is a finite positive number, else 0.
__device__ __forceinline__ uint32_t scale_bits(float s, bool on) {
  const uint32_t b = __float_as_uint(s);
  return on && b < 0x7F800000u ? b : 0u;
}

struct WideParams {
  DecodeParams d;
  CUtensorMap tm_k, tm_v;
  int box;                 // rows of a TMA box: a common divisor of page_size and 128
  int negate;              // attn_scale < 0: Q enters negated
  float abs_scale_log2;    // |attn_scale| * log2(e), not 0
  long long wait_limit;
};

template <int D, int CT, int QT>
__global__ void __launch_bounds__(WideCfg<D, CT>::THREADS, 1) decode_wide_kernel(const __grid_constant__ WideParams wp) {
  using C = WideCfg<D, CT>;
  constexpr bool E4 = C::E4;
  constexpr bool BF = CT == kBF16;     // type of the products' operands
  constexpr int NS = C::NS;
  const DecodeParams& p = wp.d;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sRing = smem + C::Q_BYTES;
  uint8_t* sRaw = sRing + NS * C::TILE;
  __shared__ WideBarriers bars;
  __shared__ Walk s_walk;
  __shared__ volatile int s_ek[8], s_ev[8];    // exponents of a tile's scales, by tile count
  __shared__ volatile int s_found[8];          // segment count + 1 of a segment with cleared values

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  // ---- set-up: this CTA's run ----------------------------------------------------------------
  const int per_seq = p.c.h_kv * p.row_tiles;
  if (warp == 0) {
    const long long total = tiles_before(p, p.c.b, lane) * per_seq;
    const int n_cta = working_ctas(p, total);
    Walk w;
    w.t = w.t_end = 0;
    w.base = 0;
    w.bi = 0;
    if (static_cast<int>(blockIdx.x) < n_cta) {
      w.t = run_start(total, blockIdx.x, n_cta);
      w.t_end = run_start(total, blockIdx.x + 1, n_cta);
      for (;;) {
        const int i = w.bi + lane;
        const long long n = i < p.c.b ? static_cast<long long>(seq_tiles(p, i)) * per_seq : 0;
        long long incl = n;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
          const long long x = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += x;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, w.base + incl > w.t);
        if (hit != 0) {
          const int k = __ffs(hit) - 1;
          w.base += __shfl_sync(0xffffffffu, incl - n, k);
          w.bi += k;
          break;
        }
        w.base += __shfl_sync(0xffffffffu, incl, 31);
        w.bi += 32;
        if (w.bi >= p.c.b) {   // not reached: t < total
          w.t = w.t_end;
          break;
        }
      }
    }
    if (lane == 0) s_walk = w;
  }
  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars.q_full[t], 128);
      mbar_init(&bars.s_full[t], 1);
      mbar_init(&bars.p_full[t], 128);
      mbar_init(&bars.o_full[t], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bars.raw_full[i], 1);
      mbar_init(&bars.raw_empty[i], 128);
    }
    for (int i = 0; i < 6; ++i) {
      mbar_init(&bars.kv_full[i], E4 ? 128 : 1);
      mbar_init(&bars.kv_empty[i], E4 ? 1 : 1 + 4);   // the MMAs that read the slot, and the clearing warps
      mbar_init(&bars.kv_clean[i], 128);
    }
    mbar_init(&bars.drain, 1);
    bars.abort = 0;
    fence_mbar_init();
    for (int i = 0; i < 8; ++i) s_found[i] = 0;
  }
  if (warp == 1) {
    tmem_alloc(&bars.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_launch_dependents();
  const uint32_t tmem = bars.tmem_base;
  volatile int* abort_flag = &bars.abort;
  const Waiter wt{abort_flag, wp.wait_limit};
  Walk walk = s_walk;
  Segment sg;

  bool producer = false;
  int kv_issued = 0;     // tiles whose copies the producer issued

  if (warp < 4) {
    regs_dec<C::REGS0>();
    if (warp == 0) {
      // ================================ pages and TMA =====================================
      producer = lane == 0;
      if (lane == 0) {
        tma_prefetch_desc(&wp.tm_k);
        tma_prefetch_desc(&wp.tm_v);
      }
      bool ok = true;
      int it = 0;
      const int boxes = kKeys / wp.box;     // boxes of a tile: 1, 2, 4 or 8
      while (ok && walk.next(p, sg)) {
        const int32_t* pages = p.c.page_table + sg.bi * p.c.page_table_stride;
        // Lane l: page and slot of box l of 32 consecutive boxes; missing ones get the page behind
        // the last, which the TMA unit fills with zeros.
        const int n_box = (sg.tile1 - sg.tile0) * boxes;
        auto look_up = [&](int b0, int& page, int& slot) {
          const int b = b0 + lane, key = sg.tile0 * kKeys + b * wp.box;
          page = p.c.num_pages;
          slot = 0;
          if (b < n_box && key < sg.L.len_kv) {
            const int col = key / p.c.page_size;
            slot = key - col * p.c.page_size;
            const int pg = __ldg(pages + col);
            if (pg >= 0 && pg < p.c.num_pages) page = pg;
          }
        };
        int page, slot, next_page, next_slot;
        look_up(0, next_page, next_slot);
        for (int j = sg.tile0; ok && j < sg.tile1; ++j) {
          const int b0 = (j - sg.tile0) * boxes;
          if (b0 % 32 == 0) {
            page = next_page;
            slot = next_slot;
            look_up(b0 + 32, next_page, next_slot);
          }
          for (int kv = 0; ok && kv < 2; ++kv) {
            uint8_t* dst;
            uint64_t* bar;
            if (lane == 0) {
              if constexpr (E4) {
                const int s = it % C::NRAW;
                ok = mbar_wait(&bars.raw_empty[s], ((it / C::NRAW) & 1) ^ 1, wt);
                dst = sRaw + s * C::RAW;
                bar = &bars.raw_full[s];
                if (ok) mbar_arrive_expect_tx(bar, C::RAW);
              } else {
                const int s = it % NS;
                ok = mbar_wait(&bars.kv_empty[s], ((it / NS) & 1) ^ 1, wt);
                dst = sRing + s * C::TILE;
                bar = &bars.kv_full[s];
                if (ok) mbar_arrive_expect_tx(bar, C::TILE);
              }
              if (ok) kv_issued = it + 1;
            }
            ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
            if (!ok) break;
            for (int x = 0; x < boxes; ++x) {
              const int pg = __shfl_sync(0xffffffffu, page, (b0 + x) % 32);
              const int sl = __shfl_sync(0xffffffffu, slot, (b0 + x) % 32);
              if (lane == 0) {
                const CUtensorMap* map = kv ? &wp.tm_v : &wp.tm_k;
                if constexpr (E4) {
                  tma_load_4d(dst + x * wp.box * D, map, bar, 0, sl, sg.hk, pg);
                } else {
                  for (int c = 0; c < C::NCHUNK; ++c)
                    tma_load_4d(dst + c * 16384 + x * wp.box * 128, map, bar, c * 64, sl, sg.hk, pg);
                }
              }
            }
            ++it;
          }
        }
      }
    } else if (warp == 1) {
      // ================================ MMA issuer ========================================
      if (elect_one_sync()) {
        const uint32_t fmt = BF ? 1u : 0u;
        const uint32_t idesc_s = make_idesc(fmt, 128, 128, false, false);
        const uint32_t idesc_pv = make_idesc(fmt, 128, D, false, true);
        bool ok = true;
        int it = 0;
        uint32_t clean_par = 0;           // by slot: parity of its next cleaning
        uint32_t q_par = 0, p_par = 0;    // by tile
        auto wait_full = [&](bool cleaned) -> int {
          const int s = it % NS;
          if (!mbar_wait(&bars.kv_full[s], (it / NS) & 1, wt)) return -1;
          if (!E4 && cleaned) {
            if (!mbar_wait(&bars.kv_clean[s], (clean_par >> s) & 1, wt)) return -1;
            clean_par ^= 1u << s;
          }
          ++it;
          tc_fence_after();
          return s;
        };
        auto issue_s = [&](int t, int s) {
          const uint32_t qa = smem_u32(sQ + t * C::TILE), kb = smem_u32(sRing + s * C::TILE);
#pragma unroll
          for (int k = 0; k < C::KSTEPS; ++k) {
            const uint32_t o = (k / 4) * 16384 + (k % 4) * 32;
            mma_ss(tmem + t * 128, make_sdesc_sw128(qa + o, 16, 1024), make_sdesc_sw128(kb + o, 16, 1024), idesc_s, k > 0, false);
          }
          tc_commit(&bars.s_full[t]);
        };
        auto issue_pv = [&](int t, int s, bool first) {
          const uint32_t vb = smem_u32(sRing + s * C::TILE);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mma_ts(tmem + C::O_COL0 + t * D, tmem + t * 128 + k * 8, make_sdesc_sw128(vb + k * 16 * 128, 16384, 1024),
                   idesc_pv, (!first || k > 0) ? 1u : 0u, false);
        };
        while (ok && walk.next(p, sg)) {
          const int n_t = p.rows - sg.r0 > 128 ? 2 : 1;
          for (int t = 0; t < n_t && ok; ++t) {
            ok = mbar_wait(&bars.q_full[t], (q_par >> t) & 1, wt);
            q_par ^= 1u << t;
          }
          if (!ok) break;
          tc_fence_after();
          const int k0 = wait_full(false);
          if (k0 < 0) { ok = false; break; }
          for (int t = 0; t < n_t; ++t) issue_s(t, k0);
          tc_commit(&bars.kv_empty[k0]);
          for (int j = sg.tile0; j < sg.tile1; ++j) {
            const int vs = wait_full(needs_cleaning(p, sg, j));
            if (vs < 0) { ok = false; break; }
            int nk = -1;
            for (int t = 0; t < n_t; ++t) {
              if (!mbar_wait(&bars.p_full[t], (p_par >> t) & 1, wt)) { ok = false; break; }
              p_par ^= 1u << t;
              tc_fence_after();
              issue_pv(t, vs, j == sg.tile0);
              if (j + 1 == sg.tile1) tc_commit(&bars.o_full[t]);
              if (t == n_t - 1) tc_commit(&bars.kv_empty[vs]);
              if (j + 1 < sg.tile1) {
                if (nk < 0) {
                  nk = wait_full(false);
                  if (nk < 0) { ok = false; break; }
                }
                issue_s(t, nk);
                if (t == n_t - 1) tc_commit(&bars.kv_empty[nk]);
              }
            }
            if (!ok) break;
          }
        }
        tc_commit(&bars.drain);
        mbar_wait_drain(&bars.drain, 0);
      }
    }
  } else if (warp >= 12) {
    regs_dec<C::REGS_WIDEN>();
    // ============================ widening / clearing =========================================
    const int w4 = warp % 4;
    const bool masked = p.causal != 0 || p.tree_mask != nullptr;
    bool ok = true;
    int it = 0, n_seg = 0, n_tile = 0;
    while (ok && walk.next(p, sg)) {
      bool found = false;
      if constexpr (E4) {
        // Tiles of K (warps 12-15) or of V (16-19).  Scales of a tile: the lane's own row
        // (32 w4 + lane), and four of the 128 for the largest; K's warps find both exponents.
        const bool is_v = warp >= 16;
        const int32_t* pages = p.c.page_table + sg.bi * p.c.page_table_stride;
        const int ps = p.c.page_size, col_step = kKeys / ps, slot_step = kKeys % ps;
        struct Spot {      // a key of this lane, moving tile by tile
          int key, col, slot;
        };
        auto spot_at = [&](int key) { return Spot{key, key / ps, key % ps}; };
        auto step = [&](Spot& x) {
          x.key += kKeys;
          x.col += col_step;
          x.slot += slot_step;
          if (x.slot >= ps) {
            x.slot -= ps;
            ++x.col;
          }
        };
        auto page_at = [&](const Spot& x) -> int {
          if (x.key >= min(sg.tile1 * kKeys, sg.L.len_kv)) return -1;
          const int pg = __ldg(pages + x.col);
          return pg < p.c.num_pages ? pg : -1;
        };
        auto scale_at = [&](const Spot& x, int pg) {
          return (static_cast<int64_t>(pg) * p.c.h_kv + sg.hk) * ps + x.slot;
        };
        const float4 kZero4 = make_float4(0.f, 0.f, 0.f, 0.f);
        float nxt_own = 0.f;
        float4 nxt_k = kZero4, nxt_v = kZero4;
        bool nxt_on = false;
        int nxt_left = 0;
        auto fetch = [&](const Spot& own, int pg_own, const Spot& four, int pg_four) {
          nxt_on = pg_own >= 0;
          nxt_left = pg_four >= 0 ? sg.L.len_kv - four.key : 0;
          nxt_own = 0.f;
          nxt_k = nxt_v = kZero4;
          if (pg_own >= 0) nxt_own = __ldg((is_v ? p.c.v_scale : p.c.k_scale) + scale_at(own, pg_own));
          if (pg_four >= 0) {
            if (!is_v) nxt_k = __ldg(reinterpret_cast<const float4*>(p.c.k_scale + scale_at(four, pg_four)));
            nxt_v = __ldg(reinterpret_cast<const float4*>(p.c.v_scale + scale_at(four, pg_four)));
          }
        };
        Spot own = spot_at(sg.tile0 * kKeys + w4 * 32 + lane), four = spot_at(sg.tile0 * kKeys + lane * 4);
        fetch(own, page_at(own), four, page_at(four));
        step(own);
        step(four);
        int pg_own = page_at(own), pg_four = page_at(four);     // of tile j + 1
        for (int j = sg.tile0; ok && j < sg.tile1; ++j) {
          const float cur = nxt_own;
          const float4 cur_k = nxt_k, cur_v = nxt_v;
          const bool on = nxt_on;
          const int left = nxt_left;
          fetch(own, pg_own, four, pg_four);
          step(own);
          step(four);
          pg_own = page_at(own);
          pg_four = page_at(four);
          auto largest = [&](const float4& f) {
            return exponent_of(__reduce_max_sync(0xffffffffu, max(max(scale_bits(f.x, left > 0), scale_bits(f.y, left > 1)),
                                                                  max(scale_bits(f.z, left > 2), scale_bits(f.w, left > 3)))));
          };
          const int ev = largest(cur_v), ex = is_v ? ev : largest(cur_k);
          if (threadIdx.x == 12 * 32) {
            s_ek[n_tile % 8] = ex;
            s_ev[n_tile % 8] = ev;
          }
          ++n_tile;
          // scale / 2^E of the lane's row as two F16, each twice in a word
          const float f = on ? cur * pow2(-ex) : 0.f;
          const __half fh = __float2half_rn(f), fl = __float2half_rn(f - __half2float(fh));
          const __half2 h2 = __half2half2(fh), l2 = __half2half2(fl);
          const bool tail = is_v && masked && (j + 1) * kKeys > sg.off;
          const int mine = it + (is_v ? 1 : 0);
          it += 2;
          const int rs = mine % C::NRAW, s = mine % NS;
          ok = mbar_wait_warp(&bars.raw_full[rs], (mine / C::NRAW) & 1, wt) &&
               mbar_wait_warp(&bars.kv_empty[s], ((mine / NS) & 1) ^ 1, wt);
          if (!ok) break;
          // A lane takes its row, 16 codes at a time; the swizzles of both tiles put the 8 rows
          // of a quarter-warp into 8 different 16-byte columns.
          const int r = w4 * 32 + lane, sw = D == 128 ? r & 7 : (r >> 1) & 3;
          const uint8_t* src = sRaw + rs * C::RAW + r * D;
          uint8_t* dst = sRing + s * C::TILE + r * 128;
#pragma unroll
          for (int c0 = 0; c0 < D / 16; c0 += 4) {
            uint4 in[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              in[x] = *reinterpret_cast<const uint4*>(src + ((c0 + x) ^ sw) * 16);
              if (!on) in[x] = make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const uint32_t w[4] = {in[x].x, in[x].y, in[x].z, in[x].w};
              uint32_t out[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                out[e] = e4m3x2_to_f16x2(e % 2 ? w[e / 2] >> 16 : w[e / 2] & 0xFFFFu);
                const __half2 v = *reinterpret_cast<const __half2*>(&out[e]);
                const __half2 y = __hfma2(v, h2, __hmul2(v, l2));
                out[e] = *reinterpret_cast<const uint32_t*>(&y);
              }
              if (tail) {
#pragma unroll
                for (int e = 0; e < 8; ++e) out[e] = finite_pair<false>(out[e], found);
              }
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int u = 2 * (c0 + x) + h;    // 16-byte unit of the 16-bit row
                *reinterpret_cast<uint4*>(dst + (u / 8) * 16384 + ((u % 8) ^ (r & 7)) * 16) =
                    make_uint4(out[4 * h], out[4 * h + 1], out[4 * h + 2], out[4 * h + 3]);
              }
            }
          }
          if (found) s_found[n_seg % 8] = n_seg + 1;
          fence_proxy_async_smem();
          mbar_arrive(&bars.kv_full[s]);
          mbar_arrive(&bars.raw_empty[rs]);
        }
      } else {
        // Every tile's phase is followed, and its slot returned, by these warps too: a parity says
        // nothing about a phase that lies further back or ahead.
        for (int j = sg.tile0; ok && j < sg.tile1; ++j) {
#pragma unroll 1
          for (int kv = 0; ok && kv < 2; ++kv, ++it) {
            const int s = it % NS;
            ok = mbar_wait_warp(&bars.kv_full[s], (it / NS) & 1, wt);
            if (!ok) break;
            if (kv && needs_cleaning(p, sg, j)) {
              const bool tail = masked && (j + 1) * kKeys > sg.off;
              const int r = w4 * 32 + lane;
              const bool on = j * kKeys + r < sg.L.len_kv;
              if (!on || tail) {
#pragma unroll 1
                for (int u = 0; u < D / 8; ++u) {
                  uint4* at = reinterpret_cast<uint4*>(sRing + s * C::TILE + (u / 8) * 16384 + r * 128 + ((u % 8) ^ (r & 7)) * 16);
                  if (!on) {
                    *at = make_uint4(0, 0, 0, 0);
                  } else {
                    uint4 x = *at;
                    x.x = finite_pair<BF>(x.x, found);
                    x.y = finite_pair<BF>(x.y, found);
                    x.z = finite_pair<BF>(x.z, found);
                    x.w = finite_pair<BF>(x.w, found);
                    *at = x;
                  }
                }
              }
              if (found) s_found[n_seg % 8] = n_seg + 1;
              fence_proxy_async_smem();
              mbar_arrive(&bars.kv_clean[s]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.kv_empty[s]);
          }
        }
      }
      ++n_seg;
    }
  } else {
    regs_inc<C::REGS_SOFTMAX>();
    // ============================ softmax, results ==============================================
    const int t = (warp - 4) / 4, quad = warp % 4;
    const int r = quad * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t s_addr = tmem + lane_off + t * 128, o_addr = tmem + lane_off + C::O_COL0 + t * D;
    const bool masked = p.causal != 0 || p.tree_mask != nullptr;
    bool ok = true;
    int n_seg = 0, n_tile = 0;
    uint32_t blk = 0, on = 0;      // blocks and segments of this tile so far
    // Segments that have rows for this tile; the blocks and segments passed over are counted.
    auto advance = [&](Segment& to, int& tiles, int& segs) {
      tiles = segs = 0;
      while (walk.next(p, to)) {
        if (t == 0 || p.rows - to.r0 > 128) return true;
        tiles += to.tile1 - to.tile0;
        ++segs;
      }
      return false;
    };
    // This thread's row of Q of a segment to shared memory; returns the factor on its scores.  To
    // be called when the last S of the segment before has been read.
    auto load_q = [&](const Segment& g) -> float {
      const int row = g.r0 + t * 128 + r;
      const bool live = row < p.rows && row / p.group < g.L.len_q;
      float cs = wp.abs_scale_log2;
      {
        const uint16_t* src = static_cast<const uint16_t*>(p.q) + (live ? row_offset(p, p.q_st, g.bi, g.hk, row) : 0);
        uint4 x[D / 8];
#pragma unroll
        for (int u = 0; u < D / 8; ++u) x[u] = live ? *reinterpret_cast<const uint4*>(src + u * 8) : make_uint4(0, 0, 0, 0);
        uint32_t* w = reinterpret_cast<uint32_t*>(x);
        if (wp.negate) {
#pragma unroll
          for (int i = 0; i < D / 2; ++i) w[i] ^= 0x80008000u;
        }
        if constexpr (E4 && QT == kBF16) {
          // To F16 by a power of two that brings the largest element to [256, 512).
          uint32_t m = 0;
#pragma unroll
          for (int i = 0; i < D / 2; ++i) m = max(m, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
          const int ex = static_cast<int>(m >> 7);
          const int sh = (ex == 0 || ex == 255) ? 0 : min(127 + 8 - ex, 126);
          const float up = pow2(sh);
          cs *= pow2(-sh);
#pragma unroll
          for (int i = 0; i < D / 2; ++i) {
            const float2 f = unpack_pair<true>(w[i]);
            w[i] = pack_pair<false>(f.x * up, f.y * up);
          }
        }
        uint8_t* q_row = sQ + t * C::TILE + r * 128;
#pragma unroll
        for (int u = 0; u < D / 8; ++u)
          *reinterpret_cast<uint4*>(q_row + (u / 8) * 16384 + ((u % 8) ^ (r & 7)) * 16) = x[u];
        fence_proxy_async_smem();
        mbar_arrive(&bars.q_full[t]);
      }
      return cs;
    };
    int skip_tiles, skip_segs;
    bool more = advance(sg, skip_tiles, skip_segs);
    float cs = more ? load_q(sg) : 0.f;
    while (ok && more) {
      n_tile += skip_tiles;
      n_seg += skip_segs;
      const int row = sg.r0 + t * 128 + r, token = row / p.group;
      const bool live = row < p.rows && token < sg.L.len_q;
      // ---- pages that do not exist (none, as a rule) -------------------------------------------------
      const int32_t* pages = p.c.page_table + sg.bi * p.c.page_table_stride;
      bool bad = false;
      {
        const int last = min(sg.tile1 * kKeys, sg.L.len_kv) - 1;
        for (int col = sg.tile0 * kKeys / p.c.page_size + lane; col <= last / p.c.page_size; col += 32) {
          const int pg = __ldg(pages + col);
          bad |= pg < 0 || pg >= p.c.num_pages;
        }
        bad = __any_sync(0xffffffffu, bad) != 0;
      }
      float m_ref = -INFINITY, l = 0.f;
      for (int j = sg.tile0; j < sg.tile1; ++j, ++blk) {
        if (!mbar_wait_warp(&bars.s_full[t], blk & 1, wt)) { ok = false; break; }
        tc_fence_after();
        float cst = cs, ev = 0.f, back = 1.f;
        if constexpr (E4) {
          cst = cs * pow2(s_ek[n_tile % 8]);
          const int e = s_ev[n_tile % 8];
          ev = static_cast<float>(e);
          back = pow2(-e);
        }
        ++n_tile;
        const int key0 = j * kKeys;
        const bool need = key0 + kKeys > sg.L.len_kv || (masked && key0 + kKeys > sg.off) || bad;
        uint32_t vis[4];       // visible columns
        if (need) {
          int lim = sg.L.len_kv - 1;
          if (p.causal) lim = min(lim, sg.off + token);
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int k0 = key0 + 32 * w, n = lim - k0 + 1;
            uint32_t v = n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u;
            const int j0 = k0 - sg.off;
            if (p.tree_mask && j0 > -32 && live) {
              const uint32_t* words = p.tree_mask + sg.bi * p.tree_mask_stride + static_cast<int64_t>(token) * p.tree_words;
              if (j0 >= 0) {
                const uint32_t lo = j0 / 32 < p.tree_words ? __ldg(words + j0 / 32) : 0u;
                const uint32_t hi = j0 / 32 + 1 < p.tree_words ? __ldg(words + j0 / 32 + 1) : 0u;
                v &= __funnelshift_r(lo, hi, j0 % 32);
              } else {
                v &= (__ldg(words) << -j0) | ((1u << -j0) - 1u);
              }
            }
            if (bad) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int key = k0 + 16 * h;
                if (key >= sg.L.len_kv) continue;
                const int pg = __ldg(pages + key / p.c.page_size);
                if (pg < 0 || pg >= p.c.num_pages) v &= h ? 0x0000FFFFu : 0xFFFF0000u;
              }
            }
            vis[w] = v;
          }
        }
        // The row's 128 scores come in halves of 64 columns: the second for its maximum, then the
        // first, which stays for its exponentials, then the second again.  P takes the columns of
        // the first quarter and then of the second, both read by then.
        uint32_t sv[64];
        auto load_half = [&](int h) {
          tmem_ld32(s_addr + h * 64, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
          tmem_ld32(s_addr + h * 64 + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
          tmem_ld_wait();
          reg_fence32(&sv[0]);
          reg_fence32(&sv[32]);
          if (need) {
#pragma unroll
            for (int c = 0; c < 64; ++c)
              if (!(((h ? vis[2 + c / 32] : vis[c / 32]) >> (c % 32)) & 1u)) sv[c] = __float_as_uint(-INFINITY);
          }
        };
        float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
        for (int h = 1; h >= 0; --h) {
          load_half(h);
#pragma unroll
          for (int c = 0; c < 64; c += 8) {
            mx0 = max3(mx0, __uint_as_float(sv[c]), __uint_as_float(sv[c + 1]));
            mx1 = max3(mx1, __uint_as_float(sv[c + 2]), __uint_as_float(sv[c + 3]));
            mx2 = max3(mx2, __uint_as_float(sv[c + 4]), __uint_as_float(sv[c + 5]));
            mx3 = max3(mx3, __uint_as_float(sv[c + 6]), __uint_as_float(sv[c + 7]));
          }
        }
        const float m_cand = fmaf(max3(mx0, mx1, fmaxf(mx2, mx3)), cst, ev);
        float alpha = 1.f;
        if (m_cand > m_ref + C::THRESH) {
          alpha = ex2(m_ref - m_cand);
          m_ref = m_cand;
        }
        const float nm = m_ref == -INFINITY ? 0.f : C::P_OFF - m_ref + ev;
        const float2 cs2 = make_float2(cst, cst), nm2 = make_float2(nm, nm);
        float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h == 1) load_half(1);
          uint32_t pk[32];
#pragma unroll
          for (int c = 0; c < 64; c += 4) {
            const float2 x01 = fma2(make_float2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])), cs2, nm2);
            const float2 x23 = fma2(make_float2(__uint_as_float(sv[c + 2]), __uint_as_float(sv[c + 3])), cs2, nm2);
            const float2 p01 = make_float2(ex2(x01.x), ex2(x01.y)), p23 = make_float2(ex2(x23.x), ex2(x23.y));
            acc0 = add2(acc0, p01);
            acc1 = add2(acc1, p23);
            pk[c / 2] = pack_pair<BF>(p01.x, p01.y);
            pk[c / 2 + 1] = pack_pair<BF>(p23.x, p23.y);
          }
          tmem_st32(s_addr + h * 32, pk);
        }
        l = l * alpha + ((acc0.x + acc0.y) + (acc1.x + acc1.y)) * back;
        // The block before has added to O already: its P V was issued ahead of this block's S.
        if (j > sg.tile0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t ov[32];
            tmem_ld32(o_addr + c * 32, ov);
            tmem_ld_wait();
            reg_fence32(ov);
#pragma unroll
            for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
            tmem_st32(o_addr + c * 32, ov);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bars.p_full[t]);
      }
      if (!ok) break;
      // ---- the next segment's Q, so that its first S runs while this one's results leave ----------
      Segment next;
      more = advance(next, skip_tiles, skip_segs);
      cs = more ? load_q(next) : 0.f;
      // ---- the segment's result: this thread's row ------------------------------------------------
      if (!mbar_wait_warp(&bars.o_full[t], on & 1, wt)) { ok = false; break; }
      ++on;
      tc_fence_after();
      const bool whole = sg.tile0 == 0 && sg.tile1 == sg.n_tiles;
      const int64_t part = 2 * blockIdx.x + (sg.tile0 == 0 ? 1 : 0);
      const bool none = !live || l == 0.f;
      const float inv = none ? 0.f : 1.f / l;
      const bool fix = live && s_found[n_seg % 8] == n_seg + 1;
      const int64_t out = row < p.rows ? row_offset(p, p.o_st, sg.bi, sg.hk, row) : 0;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t ov[32];
        tmem_ld32(o_addr + c * 32, ov);
        tmem_ld_wait();
        reg_fence32(ov);
        if (row >= p.rows) continue;
        if (fix) {
          for (int i = 0; i < 32; ++i)
            ov[i] = __float_as_uint(add_nonfinite<D, CT>(p, sg.bi, sg.hk, sg.L, row, c * 32 + i, sg.tile0 * kKeys,
                                                         min(sg.tile1 * kKeys, sg.L.len_kv), __uint_as_float(ov[i])));
        }
        if (!whole) {
          float4* dst = reinterpret_cast<float4*>(p.part_o) + (part * (D / 4) + c * 8) * 256 + t * 128 + r;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            dst[i * 256] = make_float4(__uint_as_float(ov[4 * i]), __uint_as_float(ov[4 * i + 1]), __uint_as_float(ov[4 * i + 2]),
                                 __uint_as_float(ov[4 * i + 3]));
        } else {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + out + c * 32);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float a = __uint_as_float(ov[8 * i + 2 * e]), b = __uint_as_float(ov[8 * i + 2 * e + 1]);
              w[e] = none ? 0u : pack_pair<QT == kBF16>(a * inv, b * inv);
            }
            dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      if (row < p.rows) {
        if (!whole)
          *reinterpret_cast<float2*>(p.part_ml + 2 * (part * 256 + t * 128 + r)) = make_float2(m_ref, l);
        else if (p.lse)
          p.lse[lse_offset(p, sg.bi, sg.hk, row)] = none ? -INFINITY : natural_lse(m_ref - C::P_OFF, l);
      }
      tc_fence_before();     // O has been read: the next segment's first P V follows a later arrival
      ++n_seg;
      sg = next;
    }
  }

  tc_fence_before();
  __syncthreads();
  // If a role gave up, copies may still be in flight: let them land before the CTA ends.
  if (producer && *abort_flag) {
    constexpr int N = E4 ? C::NRAW : NS;
    for (int k = (kv_issued > N ? kv_issued - N : 0); k < kv_issued; ++k)
      mbar_wait_drain(E4 ? &bars.raw_full[k % N] : &bars.kv_full[k % N], (k / N) & 1);
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of blocks that more than one CTA worked on, and writes the rows that no key
// reaches: 32 rows (lanes) by 32 elements (a warp has four) a CTA, in the parts' order.
template <int D, int QT>
__global__ void __launch_bounds__(256) decode_wide_combine_kernel(const __grid_constant__ DecodeParams p, float p_off) {
  __shared__ uint2 s_out[32][9];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int groups = (min(p.rows, 256) + 31) / 32;
  const Parts u = find_parts(p, blockIdx.x / groups, lane);
  const int r = blockIdx.x % groups * 32 + lane, row = u.r0 + r, chunk = blockIdx.y * 8 + warp;
  griddep_wait();   // (by every CTA, so that this grid never ends before the one it follows)
  if (u.n == 1) return;
  const bool on = row < p.rows;
  float m = -INFINITY, l = 0.f;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  if (on) {
#pragma unroll 4
    for (int k = 0; k < u.n; ++k) {
      const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + 2 * (u.part(k) * 256 + r));
      if (ml.y != 0.f) m = fmaxf(m, ml.x);
    }
#pragma unroll 4
    for (int k = 0; k < u.n; ++k) {
      const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + 2 * (u.part(k) * 256 + r));
      const float4 v = reinterpret_cast<const float4*>(p.part_o)[(u.part(k) * (D / 4) + chunk) * 256 + r];
      const float f = part_weight(ml, m);
      l += ml.y * f;
      x.x += f == 0.f ? 0.f : v.x * f;
      x.y += f == 0.f ? 0.f : v.y * f;
      x.z += f == 0.f ? 0.f : v.z * f;
      x.w += f == 0.f ? 0.f : v.w * f;
    }
    const bool none = row / p.group >= u.L.len_q || l == 0.f;
    const float inv = none ? 0.f : 1.f / l;
    s_out[lane][warp] = none ? make_uint2(0, 0)
                             : make_uint2(pack_pair<QT == kBF16>(x.x * inv, x.y * inv), pack_pair<QT == kBF16>(x.z * inv, x.w * inv));
    if (p.lse && chunk == 0) p.lse[lse_offset(p, u.bi, u.hk, row)] = none ? -INFINITY : natural_lse(m - p_off, l);
  }
  __syncthreads();
  // 64 bytes of a row by 8 neighbouring threads.
  const int r2 = threadIdx.x / 8, row2 = blockIdx.x % groups * 32 + r2 + u.r0;
  if (row2 < p.rows)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + row_offset(p, p.o_st, u.bi, u.hk, row2) + blockIdx.y * 32 +
                              threadIdx.x % 8 * 4) = s_out[r2][threadIdx.x % 8];
}

template <int D, int CT, int QT>
cudaError_t launch_t(const WideParams& wp, cudaStream_t st) {
  auto kern = decode_wide_kernel<D, CT, QT>;
  cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kern), WideCfg<D, CT>::SMEM);
  if (e != cudaSuccess) return e;
  const DecodeParams& p = wp.d;
  kern<<<p.ctas, WideCfg<D, CT>::THREADS, WideCfg<D, CT>::SMEM, st>>>(wp);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int groups = ((p.rows < 256 ? p.rows : 256) + 31) / 32;
  return launch_after(decode_wide_combine_kernel<D, QT>,
                      dim3(static_cast<unsigned>(p.c.b) * p.c.h_kv * p.row_tiles * groups, D / 32), dim3(256), st, p,
                      WideCfg<D, CT>::P_OFF);
}

template <int D>
cudaError_t launch_d(const WideParams& wp, int qt, int ct, cudaStream_t st) {
  if (qt == kBF16) return ct == kE4M3 ? launch_t<D, kE4M3, kBF16>(wp, st) : launch_t<D, kBF16, kBF16>(wp, st);
  return ct == kE4M3 ? launch_t<D, kE4M3, kF16>(wp, st) : launch_t<D, kF16, kF16>(wp, st);
}

}  // namespace

int decode_wide_box(int page_size) {
  int box = 128;
  while (page_size % box != 0) box /= 2;
  return box;
}

int decode_wide_swizzle(int d, int cache_dtype) { return cache_dtype == kE4M3 && d == 64 ? 64 : 128; }

cudaError_t launch_decode_wide(const DecodeParams& p, const CUtensorMap& tm_k, const CUtensorMap& tm_v, long long wait_limit,
                               int d, int qt, int ct, cudaStream_t st) {
  WideParams wp;
  wp.d = p;
  wp.tm_k = tm_k;
  wp.tm_v = tm_v;
  wp.box = decode_wide_box(p.c.page_size);
  wp.negate = p.scale_log2 < 0.f ? 1 : 0;
  // A scale of zero: every visible key weighs the same (and hidden ones still come out as -inf).
  wp.abs_scale_log2 = p.scale_log2 == 0.f ? 1e-30f : fabsf(p.scale_log2);
  wp.wait_limit = wait_limit;
  if (d == 64) return launch_d<64>(wp, qt, ct, st);
  if (d == 128) return launch_d<128>(wp, qt, ct, st);
  return cudaErrorInvalidValue;
}

uint32_t decode_take_device_error() {
  uint32_t v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, ptx::g_device_error, sizeof(v)) != cudaSuccess) return 0;
  if (v) cudaMemcpyToSymbol(ptx::g_device_error, &z, sizeof(z));
  return v;
}

}  // namespace sdpa
