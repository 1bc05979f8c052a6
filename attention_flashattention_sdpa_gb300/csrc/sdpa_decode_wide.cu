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
//   warps 12-15  E4M3 caches: every tile is widened to F16 on its way from the TMA's stage to the
//                ring; 16-bit caches: only V tiles that end behind the sequence or hold drafted
//                tokens are touched (rows that do not exist and values that are not finite are
//                cleared: a weight of zero does not hide a NaN in a product).
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

constexpr int kThreads = 512;
constexpr int kKeys = 128;
constexpr int kLog2Keys = 7;

template <int D, int CT>
struct WideCfg {
  static constexpr bool E4 = CT == kE4M3;
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
__global__ void __launch_bounds__(kThreads, 1) decode_wide_kernel(const __grid_constant__ WideParams wp) {
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

  // Registers (512 threads, 128 each at launch): 64 + 80 + 2 x 184 = 4 x 128.
  if (warp < 4) {
    regs_dec<64>();
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
    regs_dec<80>();
    // ============================ widening / clearing =========================================
    const int w4 = warp - 12;
    const bool masked = p.causal != 0 || p.tree_mask != nullptr;
    bool ok = true;
    int it = 0, n_seg = 0, n_tile = 0;
    while (ok && walk.next(p, sg)) {
      bool found = false;
      if constexpr (E4) {
        const int32_t* pages = p.c.page_table + sg.bi * p.c.page_table_stride;
        // Scales of a tile: lane's own row (32 w4 + lane), and four of the 128 for the maximum.
        struct Scales {
          float own[2];
          float4 four[2];
          bool on_own;
          int left;         // existing keys from this lane's first of four on
        };
        auto page_at = [&](int key) -> int {
          if (key >= sg.L.len_kv) return -1;
          const int pg = __ldg(pages + key / p.c.page_size);
          return pg < p.c.num_pages ? pg : -1;
        };
        auto fetch = [&](int j, int pg_own, int pg_four) {
          Scales s;
          const int own = j * kKeys + w4 * 32 + lane, four = j * kKeys + lane * 4;
          s.on_own = pg_own >= 0;
          s.left = pg_four >= 0 ? sg.L.len_kv - four : 0;
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const float* base = kv ? p.c.v_scale : p.c.k_scale;
            s.own[kv] = 0.f;
            s.four[kv] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (pg_own >= 0)
              s.own[kv] = __ldg(base + (static_cast<int64_t>(pg_own) * p.c.h_kv + sg.hk) * p.c.page_size + own % p.c.page_size);
            if (pg_four >= 0)
              s.four[kv] = __ldg(reinterpret_cast<const float4*>(
                  base + (static_cast<int64_t>(pg_four) * p.c.h_kv + sg.hk) * p.c.page_size + four % p.c.page_size));
          }
          return s;
        };
        Scales nxt = fetch(sg.tile0, page_at(sg.tile0 * kKeys + w4 * 32 + lane), page_at(sg.tile0 * kKeys + lane * 4));
        int pg_own = -1, pg_four = -1;
        if (sg.tile0 + 1 < sg.tile1) {
          pg_own = page_at((sg.tile0 + 1) * kKeys + w4 * 32 + lane);
          pg_four = page_at((sg.tile0 + 1) * kKeys + lane * 4);
        }
        for (int j = sg.tile0; ok && j < sg.tile1; ++j) {
          const Scales cur = nxt;
          if (j + 1 < sg.tile1) nxt = fetch(j + 1, pg_own, pg_four);
          if (j + 2 < sg.tile1) {
            pg_own = page_at((j + 2) * kKeys + w4 * 32 + lane);
            pg_four = page_at((j + 2) * kKeys + lane * 4);
          }
          int ex[2];
          uint32_t fh[2], fl[2];      // scale / 2^E of the lane's own row as two F16, each twice in a word
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const float4 f = cur.four[kv];
            uint32_t m = max(max(scale_bits(f.x, cur.left > 0), scale_bits(f.y, cur.left > 1)),
                             max(scale_bits(f.z, cur.left > 2), scale_bits(f.w, cur.left > 3)));
            m = __reduce_max_sync(0xffffffffu, m);
            ex[kv] = exponent_of(m);
            const float s = cur.on_own ? cur.own[kv] * pow2(-ex[kv]) : 0.f;
            const __half h = __float2half_rn(s);
            const __half l = __float2half_rn(s - __half2float(h));
            fh[kv] = __half_as_ushort(h) * 0x10001u;
            fl[kv] = __half_as_ushort(l) * 0x10001u;
          }
          if (threadIdx.x == 12 * 32) {
            s_ek[n_tile % 8] = ex[0];
            s_ev[n_tile % 8] = ex[1];
          }
          ++n_tile;
          const bool tail = masked && (j + 1) * kKeys > sg.off;
          const int rows_on = min(max(sg.L.len_kv - j * kKeys - w4 * 32, 0), 32);
#pragma unroll 1
          for (int kv = 0; ok && kv < 2; ++kv) {
            const int rs = it % C::NRAW, s = it % NS;
            ok = mbar_wait_warp(&bars.raw_full[rs], (it / C::NRAW) & 1, wt) &&
                 mbar_wait_warp(&bars.kv_empty[s], ((it / NS) & 1) ^ 1, wt);
            if (!ok) break;
            // A lane takes 8 codes at a time: rows of D / 8 lanes, 256 bytes of codes a warp.
            constexpr int LR = D / 8, RI = 32 / LR;      // lanes of a row, rows of an instruction
            const uint8_t* src = sRaw + rs * C::RAW + w4 * 32 * D + lane * 8;
            uint8_t* dst = sRing + s * C::TILE;
            const int u = lane % LR;                      // 16-byte unit of the 16-bit row
            const uint32_t my_h = kv ? fh[1] : fh[0], my_l = kv ? fl[1] : fl[0];
#pragma unroll 4
            for (int i = 0; i < 32 / RI; ++i) {
              const int lr = i * RI + lane / LR, r = w4 * 32 + lr;
              const uint2 in = *reinterpret_cast<const uint2*>(src + i * 256);
              const uint32_t h = __shfl_sync(0xffffffffu, my_h, lr), l = __shfl_sync(0xffffffffu, my_l, lr);
              const __half2 h2 = *reinterpret_cast<const __half2*>(&h), l2 = *reinterpret_cast<const __half2*>(&l);
              uint32_t out[4] = {e4m3x2_to_f16x2(in.x & 0xFFFFu), e4m3x2_to_f16x2(in.x >> 16),
                                 e4m3x2_to_f16x2(in.y & 0xFFFFu), e4m3x2_to_f16x2(in.y >> 16)};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const __half2 x = *reinterpret_cast<const __half2*>(&out[e]);
                const __half2 y = __hfma2(x, h2, __hmul2(x, l2));
                out[e] = *reinterpret_cast<const uint32_t*>(&y);
              }
              if (kv && lr >= rows_on) out[0] = out[1] = out[2] = out[3] = 0u;
              if (kv && tail) {
#pragma unroll
                for (int e = 0; e < 4; ++e) out[e] = finite_pair<false>(out[e], found);
              }
              *reinterpret_cast<uint4*>(dst + (u / 8) * 16384 + r * 128 + ((u % 8) ^ (r & 7)) * 16) =
                  make_uint4(out[0], out[1], out[2], out[3]);
            }
            if (kv && found) s_found[n_seg % 8] = n_seg + 1;
            fence_proxy_async_smem();
            mbar_arrive(&bars.kv_full[s]);
            mbar_arrive(&bars.raw_empty[rs]);
            ++it;
          }
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
    regs_inc<184>();
    // ============================ softmax, results ==============================================
    const int t = (warp - 4) / 4, quad = warp % 4;
    const int r = quad * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t s_addr = tmem + lane_off + t * 128, o_addr = tmem + lane_off + C::O_COL0 + t * D;
    const bool masked = p.causal != 0 || p.tree_mask != nullptr;
    bool ok = true;
    int n_seg = 0, n_tile = 0;
    uint32_t blk = 0, on = 0;      // blocks and segments of this tile so far
    while (ok && walk.next(p, sg)) {
      const int n_blk = sg.tile1 - sg.tile0;
      if (t == 1 && p.rows - sg.r0 <= 128) {   // no rows for the second tile
        n_tile += n_blk;
        ++n_seg;
        continue;
      }
      const int row = sg.r0 + t * 128 + r, token = row / p.group;
      const bool live = row < p.rows && token < sg.L.len_q;
      // ---- Q: this thread's row (the last S of the segment before has been read) -------------------
      float cs = wp.abs_scale_log2;
      {
        const uint16_t* src = static_cast<const uint16_t*>(p.q) + (live ? row_offset(p, p.q_st, sg.bi, sg.hk, row) : 0);
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
        uint32_t sv[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(s_addr + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[c * 32]));
        float cst = cs, ev = 0.f, back = 1.f;
        if constexpr (E4) {
          cst = cs * pow2(s_ek[n_tile % 8]);
          const int e = s_ev[n_tile % 8];
          ev = static_cast<float>(e);
          back = pow2(-e);
        }
        ++n_tile;
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 4; ++c) reg_fence32(&sv[c * 32]);
        const int key0 = j * kKeys;
        if (key0 + kKeys > sg.L.len_kv || (masked && key0 + kKeys > sg.off) || bad) {
          // Visible columns as four words.
          int lim = sg.L.len_kv - 1;
          if (p.causal) lim = min(lim, sg.off + token);
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int k0 = key0 + 32 * w, n = lim - k0 + 1;
            uint32_t vis = n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u;
            const int j0 = k0 - sg.off;
            if (p.tree_mask && j0 > -32 && live) {
              const uint32_t* words = p.tree_mask + sg.bi * p.tree_mask_stride + static_cast<int64_t>(token) * p.tree_words;
              if (j0 >= 0) {
                const uint32_t lo = j0 / 32 < p.tree_words ? __ldg(words + j0 / 32) : 0u;
                const uint32_t hi = j0 / 32 + 1 < p.tree_words ? __ldg(words + j0 / 32 + 1) : 0u;
                vis &= __funnelshift_r(lo, hi, j0 % 32);
              } else {
                vis &= (__ldg(words) << -j0) | ((1u << -j0) - 1u);
              }
            }
            if (bad) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int key = k0 + 16 * h;
                if (key >= sg.L.len_kv) continue;
                const int pg = __ldg(pages + key / p.c.page_size);
                if (pg < 0 || pg >= p.c.num_pages) vis &= h ? 0x0000FFFFu : 0xFFFF0000u;
              }
            }
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!((vis >> c) & 1u)) sv[32 * w + c] = __float_as_uint(-INFINITY);
          }
        }
        float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
        for (int c = 0; c < 128; c += 8) {
          mx0 = max3(mx0, __uint_as_float(sv[c]), __uint_as_float(sv[c + 1]));
          mx1 = max3(mx1, __uint_as_float(sv[c + 2]), __uint_as_float(sv[c + 3]));
          mx2 = max3(mx2, __uint_as_float(sv[c + 4]), __uint_as_float(sv[c + 5]));
          mx3 = max3(mx3, __uint_as_float(sv[c + 6]), __uint_as_float(sv[c + 7]));
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
        uint32_t pk[64];
#pragma unroll
        for (int c = 0; c < 128; c += 4) {
          const float2 x01 = fma2(make_float2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])), cs2, nm2);
          const float2 x23 = fma2(make_float2(__uint_as_float(sv[c + 2]), __uint_as_float(sv[c + 3])), cs2, nm2);
          const float2 p01 = make_float2(ex2(x01.x), ex2(x01.y)), p23 = make_float2(ex2(x23.x), ex2(x23.y));
          acc0 = add2(acc0, p01);
          acc1 = add2(acc1, p23);
          pk[c / 2] = pack_pair<BF>(p01.x, p01.y);
          pk[c / 2 + 1] = pack_pair<BF>(p23.x, p23.y);
        }
        tmem_st32(s_addr, *reinterpret_cast<uint32_t(*)[32]>(&pk[0]));
        tmem_st32(s_addr + 32, *reinterpret_cast<uint32_t(*)[32]>(&pk[32]));
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
      // ---- the segment's result: this thread's row ------------------------------------------------
      if (!mbar_wait_warp(&bars.o_full[t], on & 1, wt)) { ok = false; break; }
      ++on;
      tc_fence_after();
      const bool whole = sg.tile0 == 0 && sg.tile1 == sg.n_tiles;
      const int64_t part = static_cast<int64_t>(2 * blockIdx.x + (sg.tile0 == 0 ? 1 : 0)) * 256 + t * 128 + r;
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
          float4* dst = reinterpret_cast<float4*>(p.part_o + part * D + c * 32);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            dst[i] = make_float4(__uint_as_float(ov[4 * i]), __uint_as_float(ov[4 * i + 1]), __uint_as_float(ov[4 * i + 2]),
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
          *reinterpret_cast<float2*>(p.part_ml + 2 * part) = make_float2(m_ref, l);
        else if (p.lse)
          p.lse[(static_cast<int64_t>(sg.bi) * p.h_q + sg.hk * p.group + row % p.group) * p.s_q + token] =
              none ? -INFINITY : (m_ref - C::P_OFF + __log2f(l)) * 0.6931471805599453f;
      }
      tc_fence_before();     // O has been read: the next segment's first P V follows a later arrival
      ++n_seg;
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

template <int D, int CT, int QT>
cudaError_t launch_t(const WideParams& wp, cudaStream_t st) {
  auto kern = decode_wide_kernel<D, CT, QT>;
  cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kern), WideCfg<D, CT>::SMEM);
  if (e != cudaSuccess) return e;
  kern<<<wp.d.ctas, kThreads, WideCfg<D, CT>::SMEM, st>>>(wp);
  return cudaGetLastError();
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
