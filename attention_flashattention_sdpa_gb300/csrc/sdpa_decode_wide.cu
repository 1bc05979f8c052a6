// sdpa_decode_wide.cu — attention over a paged cache for many query rows a KV head: drafted trees
// and short chunks whose s_q tokens times the heads of a group fill tcgen05 tiles.
//
// The split of the batch is that of sdpa_decode.cu with tiles of 128 keys and blocks of 256 rows:
// one persistent CTA an SM walks a run of tiles for its KV head and block of rows, segment by segment
// (a segment: the part of the run in one sequence).  Roles:
//   warps 0, 2   pages and TMA of K and of V, box by box (a box lies in one page), a lane a box; boxes
//                of missing pages and behind the sequence are filled with zeros.  (One thread for all of
//                them took 4200 cycles a tile.)
//   warp 1       MMA issuer: S = Q K^T into TMEM, O += P V with P read from TMEM.
//   warp 3       E4M3: V's scales.
//   warps 4-11   two softmax warpgroups; thread r owns a row: loads it into shared memory, the
//                running max and sum, P, and the segment's results.  A block of more than 128 rows
//                has a 128-row tile for each; in a smaller one both take the same rows and every
//                second tile of keys, so that one computes while the other's products run.
//   warps 12-15  E4M3: widen K to F16 on its way from the TMA's stage to the ring (and warps 16-19 V), and
//                fetch K's scales;
//                16-bit: clear, in V tiles that end behind the sequence or hold drafted tokens, rows
//                that do not exist and values that are not finite (a weight of zero does not hide a
//                NaN in a product).
//
// E4M3: codes become F16 as they are.  S of codes is exact up to the fp32 sums, and the softmax warps multiply
// each of its columns by the key's scale in fp32; the scale of its value joins the weight, over 2^v of the row, as
// in sdpa_decode.cu: weights are rounded once, V not at all, l and LSE know nothing of V's scales, and a hidden
// key's scale touches no other row.  (V times scale over a power of two of the tile, in F16, instead: two roundings,
// and rows lost the keys beside a drafted one with a scale 2^20 times theirs, hidden or not.  K times
// its scale in F16 left the scores off by 2^-12 of themselves, which the LSE shows.)
//
// Weights are rounded once, to the type of the products (BF16 8 bits: O of a BF16 cache is off by 0.0023 of itself
// where its store alone gives 0.0017): a second term, as blocks of 8 rows in sdpa_decode.cu have it, would be half
// as many tensor instructions again.
//
// Bound: the tensor cores (4 x 128 x 128 x d MMAs a block of two tiles) and the exponentials, as
// the prompt's forward pass; reading the cache once bounds it for few rows.  Measured, 8 sequences of 4000
// to 8192 tokens, trees of 64 tokens, 64 heads over 8 of 128: BF16 105 us (990 TFLOP/s), E4M3 153 (677; F16 results 137).  128
// keys by 256 rows take 1.9 us over BF16, 2.5 to 2.6 over E4M3, of 1.13 of MMA (the warps that widen and the
// scales, 64 reads of 16 bytes a row and tile, share the schedulers and the shared memory with the softmax,
// and K has one slot where BF16 has two); 28 us of a call over BF16, 35 (F16 Q) and 47 (BF16 Q) over E4M3, are
// the first fetch of the code, Q, the last results and the parts.
#include <type_traits>

#include "sdpa_decode.cuh"

namespace sdpa {
namespace {

constexpr int kKeys = 128;

template <int D, int CT>
struct WideCfg {
  static constexpr bool E4 = CT == kE4M3;
  static constexpr int THREADS = E4 ? 640 : 512;
  // Registers of the producers', the softmax and the widening or clearing warpgroups, out of 96
  // (E4M3) or 128 a thread at launch: 64 + 2 x 152 + 2 x 56 = 5 x 96, 96 + 2 x 168 + 80 = 4 x 128.
  static constexpr int REGS0 = E4 ? 64 : 96, REGS_SOFTMAX = E4 ? 152 : 168, REGS_WIDEN = E4 ? 56 : 80;
  static constexpr int TILE = 128 * D * 2;                // a 16-bit tile of 128 rows
  static constexpr int RAW = 128 * 128;                   // an E4M3 tile: rows of 128 bytes (d = 64: half zeros)
  static constexpr int NCHUNK = D / 64;                   // 128-byte columns of a 16-bit tile
  // Slots of 16-bit K and V tiles, and stages of E4M3 K and V tiles with their scales.  K and V have
  // slots of their own: a wait for a parity may not skip phases, and in a ring of three that they
  // shared, each would follow only every second phase of a slot.
  static constexpr int NK = D == 128 ? (E4 ? 1 : 2) : (E4 ? 2 : 3), NV = D == 128 ? 2 : 3;
  static constexpr int RK = E4 ? 2 : 0, RV = E4 ? 2 : 0;
  static constexpr int OFF_K = 2 * TILE, OFF_V = OFF_K + NK * TILE, OFF_RAW = OFF_V + NV * TILE;
  // Scales, in rings that the softmax warps read, written when the tile's slot is free.  A slot of K is
  // free once S of the tile NK back is done, and that S followed the weights of the tile before it, or (split)
  // two before it: NK + 2 tiles' scales never meet.  A slot of V is free once P V of the tile NV back is
  // done, which its weights preceded: NV tiles'.
  static constexpr int KS = E4 ? NK + 2 : 0, VS = E4 ? NV : 0;
  static constexpr int OFF_KS = OFF_RAW + (RK + RV) * RAW, OFF_VS = OFF_KS + KS * 512, OFF_CTL = OFF_VS + VS * 512;
  static constexpr int SMEM = OFF_CTL + 512;
  static constexpr int KSTEPS = D / 16;
  static constexpr int O_COL0 = 256;
  static constexpr float P_OFF = CT == kBF16 ? 0.f : 6.f;
  static constexpr float THRESH = 8.f;
  static_assert(SMEM <= 232448, "shared memory");
  static_assert(O_COL0 + 2 * D <= 512, "TMEM");
};

struct alignas(8) WideBarriers {
  uint64_t q_full[2];
  uint64_t full[6], empty[6], clean[6];     // 16-bit tiles: K's slots, then V's
  uint64_t raw_full[4], raw_empty[4];       // E4M3 tiles: K's stages, then V's
  uint64_t s_full[2], p_full[2], o_full[2];
  uint64_t ml_full, o1_free;                // split: the second warpgroup's maxima and sums are there; its O is read
  uint64_t sc_full[4];                      // E4M3: a tile's scales are there
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

// A part of this CTA's run: tiles [tile0, tile1) of one sequence.
struct Segment {
  int bi, n_tiles, tile0, tile1, off;
  SeqLens L;
};

// The run's position; every role walks it by itself.
struct Walk : Run {
  __device__ __forceinline__ bool next(const DecodeParams& p, Segment& g) {
    while (t < t_end) {
      const int n = seq_tiles(p, bi);
      if (t >= base + n) {
        base += n;
        ++bi;
        continue;
      }
      g.bi = bi;
      g.n_tiles = n;
      g.tile0 = static_cast<int>(t - base);
      g.tile1 = static_cast<int>(min(static_cast<long long>(n), t_end - base));
      g.L = seq_lens(p, bi);
      g.off = g.L.len_kv - g.L.len_q;
      t = base + g.tile1;
      return true;
    }
    return false;
  }
};

// What the roles share besides tiles.
struct Control {
  WideBarriers bars;
  Walk walk;
  int ev[4];             // E4M3: v that a tile's V scales need, by tile count (as sc_full)
  int found[8];          // segment count + 1 of a segment with cleared values
};
static_assert(sizeof(Control) <= 512);

// Whether V's tile of a 16-bit cache has to be cleared of what no row may meet.
__device__ __forceinline__ bool needs_cleaning(const DecodeParams& p, const Segment& g, int tile) {
  const int end = (tile + 1) * kKeys;
  return end > g.L.len_kv || ((p.causal || p.tree_mask) && end > g.off);
}

// What a tile's V scales are divided by (log2) as they are stored, v_tile being the v that they need: nothing, unless
// that is far from 0.  They are then below 2^68, and a weight times vs / 2^v, below 2^15, is a product of two fp32
// values, one of them the exponential with the rest of 2^-v in its argument.
__device__ __forceinline__ int scale_exponent(int v_tile) { return v_tile > kNearV ? kNearV : v_tile < -kNearV ? -kNearV : 0; }

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
  constexpr bool BF = CT == kBF16;     // type of the 16-bit operands
  // Slot or stage of tile n of K or V, and the turn it is in there.
  struct Place {
    int at, turn;
  };
  auto slot_of = [](bool is_v, int n) { return is_v ? Place{C::NK + n % C::NV, n / C::NV} : Place{n % C::NK, n / C::NK}; };
  auto stage_of = [](bool is_v, int n) {
    if constexpr (E4) return is_v ? Place{C::RK + n % C::RV, n / C::RV} : Place{n % C::RK, n / C::RK};
    else return Place{0, 0};
  };
  const DecodeParams& p = wp.d;

  // All of it dynamic, without static arrays: it then begins on the 1024-byte boundary that the
  // swizzled tiles need (checked), with no room lost to alignment.
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) % 1024 != 0) {
    if (threadIdx.x == 0) atomicOr(&g_device_error, kErrSmemAlign);
    return;
  }
  uint8_t* sQ = smem;
  uint8_t* sRing = smem + C::OFF_K;
  uint8_t* sRaw = smem + C::OFF_RAW;
  float* sKs = reinterpret_cast<float*>(smem + C::OFF_KS);   // K's scales [tile % KS][128]
  float* sVs = reinterpret_cast<float*>(smem + C::OFF_VS);   // V's scales [tile % VS][128]
  // Split: the second warpgroup's maximum, sum and (E4M3) v of each row (the second tile of Q is not used).
  float2* s_ml = reinterpret_cast<float2*>(smem + C::TILE);
  int* s_v = reinterpret_cast<int*>(smem + C::TILE + 128 * 8);
  Control& ctl = *reinterpret_cast<Control*>(smem + C::OFF_CTL);
  WideBarriers& bars = ctl.bars;
  volatile int* s_ev = ctl.ev;
  volatile int* s_found = ctl.found;

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  // ---- set-up: this CTA's block of rows, the same of every sequence, and its team's run ----------
  const int blocks = p.c.h_kv * p.row_tiles, blk = blockIdx.x % blocks;
  const int hk = blk / p.row_tiles, r0 = blk % p.row_tiles * 256;
  const bool split = p.rows - r0 <= 128;   // at most 128 rows: the warpgroups take every second tile of keys
  if (warp == 0) {
    Walk w;
    static_cast<Run&>(w) = find_run(p, blockIdx.x / blocks, lane);
    if (lane == 0) ctl.walk = w;
  }
  if (threadIdx.x == 32) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars.q_full[t], 128);
      mbar_init(&bars.s_full[t], 1);
      mbar_init(&bars.p_full[t], 128);
      mbar_init(&bars.o_full[t], 1);
    }
    for (int i = 0; i < 6; ++i) {
      mbar_init(&bars.full[i], E4 ? 128 : 1);
      mbar_init(&bars.empty[i], E4 ? 1 : 1 + 4);     // the MMAs that read the slot, and the clearing warps
      mbar_init(&bars.clean[i], 128);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bars.raw_full[i], 1);
      mbar_init(&bars.raw_empty[i], 128);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&bars.sc_full[i], 4 + 1);
    mbar_init(&bars.ml_full, 128);
    mbar_init(&bars.o1_free, 128);
    mbar_init(&bars.drain, 1);
    bars.abort = 0;
    fence_mbar_init();
    for (int i = 0; i < 8; ++i) s_found[i] = 0;
  }
  if (warp == 1) {
    __syncwarp();
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
  Walk walk = ctl.walk;
  Segment sg;

  bool producer = false;
  int issued = 0;          // tiles whose copies this producer issued

  if (warp < 4) {
    regs_dec<C::REGS0>();
    if (warp == 0 || warp == 2) {
      // ================================ pages and TMA =====================================
      const bool is_v = warp == 2;
      producer = lane == 0;
      const CUtensorMap* map = is_v ? &wp.tm_v : &wp.tm_k;
      if (lane == 0) tma_prefetch_desc(map);
      const int boxes = kKeys / wp.box;     // boxes of a tile: 1, 2, 4 or 8
      // Lane x + 8 y issues copy y of box x: of 16-bit tiles the 128-byte columns, of E4M3 ones the codes.
      const int bx = lane % 8, by = lane / 8;
      constexpr int kCopies = E4 ? 1 : C::NCHUNK;
      bool ok = true;
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
        for (int b0 = 0; b0 < n_box; b0 += boxes) {
          if (b0 % 32 == 0) {
            page = next_page;
            slot = next_slot;
            look_up(b0 + 32, next_page, next_slot);
          }
          const int pg = __shfl_sync(0xffffffffu, page, (b0 + bx) % 32), sl = __shfl_sync(0xffffffffu, slot, (b0 + bx) % 32);
          const Place at = E4 ? stage_of(is_v, issued) : slot_of(is_v, issued);
          const int s = at.at;
          if (!mbar_wait_warp(E4 ? &bars.raw_empty[s] : &bars.empty[s], (at.turn & 1) ^ 1, wt)) { ok = false; break; }
          uint64_t* full = E4 ? &bars.raw_full[s] : &bars.full[s];
          uint8_t* dst = E4 ? sRaw + s * C::RAW : sRing + s * C::TILE;
          if (lane == 0) mbar_arrive_expect_tx(full, E4 ? C::RAW : C::TILE);
          ++issued;
          __syncwarp();
          if (bx < boxes && by < kCopies) {
            if constexpr (E4) {
              tma_load_4d(dst + bx * wp.box * 128, map, full, 0, sl, hk, pg);
            } else {
              tma_load_4d(dst + by * 16384 + bx * wp.box * 128, map, full, by * 64, sl, hk, pg);
            }
          }
          __syncwarp();
        }
      }
    } else if (warp == 1) {
      // ================================ MMA issuer ========================================
      if (elect_one_sync()) {
        const uint32_t idesc_s = make_idesc(BF ? 1u : 0u, 128, 128, false, false);
        const uint32_t idesc_pv = make_idesc(BF ? 1u : 0u, 128, D, false, true);
        bool ok = true;
        int nk = 0, nv = 0;               // tiles of K and V so far
        uint32_t clean_par = 0;           // by slot: parity of its next cleaning
        uint32_t q_par = 0, p_par = 0;    // by tile
        // Slots of the next tile of K and of V.
        auto wait_tile = [&](Place x) -> int {
          if (!mbar_wait(&bars.full[x.at], x.turn & 1, wt)) return -1;
          tc_fence_after();
          return x.at;
        };
        auto wait_k = [&]() -> int { return wait_tile(slot_of(false, nk++)); };
        auto wait_v = [&](bool cleaned) -> int {
          const int s = wait_tile(slot_of(true, nv++));
          if (!E4 && cleaned && s >= 0) {
            if (!mbar_wait(&bars.clean[s], (clean_par >> s) & 1, wt)) return -1;
            clean_par ^= 1u << s;
            tc_fence_after();
          }
          return s;
        };
        auto wait_p = [&](int t) {
          if (!mbar_wait(&bars.p_full[t], (p_par >> t) & 1, wt)) return false;
          p_par ^= 1u << t;
          tc_fence_after();
          return true;
        };
        // S of slot t from tile `tq` of Q.
        auto issue_s = [&](int t, int tq, int s) {
          const uint32_t qa = smem_u32(sQ + tq * C::TILE), kb = smem_u32(sRing + s * C::TILE);
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
          const int n = sg.tile1 - sg.tile0;
          for (int t = 0; t < (split ? 1 : 2) && ok; ++t) {
            ok = mbar_wait(&bars.q_full[t], (q_par >> t) & 1, wt);
            q_par ^= 1u << t;
          }
          if (!ok) break;
          tc_fence_after();
          if (split) {
            // Slot i % 2 for tile i: S runs two tiles ahead of P V.
            for (int i = 0; i < 2 && i < n; ++i) {
              const int s = wait_k();
              if (s < 0) { ok = false; break; }
              issue_s(i, 0, s);
              tc_commit(&bars.empty[s]);
            }
            for (int i = 0; ok && i < n; ++i) {
              const int t = i & 1, vs = wait_v(needs_cleaning(p, sg, sg.tile0 + i));
              if (vs < 0 || !wait_p(t)) { ok = false; break; }
              issue_pv(t, vs, i < 2);
              if (i + 2 >= n) tc_commit(&bars.o_full[t]);
              tc_commit(&bars.empty[vs]);
              if (i + 2 < n) {
                const int s = wait_k();
                if (s < 0) { ok = false; break; }
                issue_s(t, 0, s);
                tc_commit(&bars.empty[s]);
              }
            }
          } else {
            const int k0 = wait_k();
            if (k0 < 0) { ok = false; break; }
            for (int t = 0; t < 2; ++t) issue_s(t, t, k0);
            tc_commit(&bars.empty[k0]);
            for (int i = 0; ok && i < n; ++i) {
              const int vs = wait_v(needs_cleaning(p, sg, sg.tile0 + i));
              if (vs < 0) { ok = false; break; }
              int s = -1;
              for (int t = 0; t < 2; ++t) {
                if (!wait_p(t)) { ok = false; break; }
                issue_pv(t, vs, i == 0);
                if (i + 1 == n) tc_commit(&bars.o_full[t]);
                if (t == 1) tc_commit(&bars.empty[vs]);
                if (i + 1 < n) {
                  if (t == 0) s = wait_k();
                  if (s < 0) { ok = false; break; }
                  issue_s(t, t, s);
                  if (t == 1) tc_commit(&bars.empty[s]);
                }
              }
            }
          }
        }
        tc_commit(&bars.drain);
        mbar_wait_drain(&bars.drain, 0);
      }
    } else if (E4) {
      // ================================ V's scales ========================================
      bool ok = true;
      int n_seg = 0, n_tile = 0;
      while (ok && walk.next(p, sg)) {
        // Lane l: page of keys 4 l .. 4 l + 3 of a tile (-1: none; pages hold multiples of 16), and their
        // scales (0 where there is no key); both are asked for ahead.
        auto page_of = [&](int j) {
          const int key = j * kKeys + 4 * lane;
          return key < sg.L.len_kv ? __ldg(p.c.page_table + sg.bi * p.c.page_table_stride + key / p.c.page_size) : -1;
        };
        auto scales_of = [&](int j, int page) {
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
          if (page < 0 || page >= p.c.num_pages) return x;
          const int key = j * kKeys + 4 * lane, left = sg.L.len_kv - key;
          x = __ldg(reinterpret_cast<const float4*>(p.c.v_scale + (static_cast<int64_t>(page) * p.c.h_kv + hk) * p.c.page_size +
                                                    key % p.c.page_size));
          if (left < 2) x.y = 0.f;
          if (left < 3) x.z = 0.f;
          if (left < 4) x.w = 0.f;
          return x;
        };
        float4 scales = scales_of(sg.tile0, page_of(sg.tile0));
        int page1 = sg.tile0 + 1 < sg.tile1 ? page_of(sg.tile0 + 1) : -1;
        for (int j = sg.tile0; j < sg.tile1; ++j, ++n_tile) {
          auto magnitude = [](float x) {
            const uint32_t b = __float_as_uint(fabsf(x));
            return b < 0x7F800000u ? b : 0u;
          };
          const int need = needed_v(__reduce_max_sync(0xffffffffu, max(max(magnitude(scales.x), magnitude(scales.y)),
                                                                       max(magnitude(scales.z), magnitude(scales.w)))));
          const float by = pow2(-scale_exponent(need));
          float x[4] = {scales.x * by, scales.y * by, scales.z * by, scales.w * by};
          if ((p.causal || p.tree_mask) && (j + 1) * kKeys > sg.off) {
            // A scale that is not finite, times the weight of zero of a row that does not see its key, would be
            // NaN: rows that do see it get its values afterwards.
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (!(fabsf(x[i]) < INFINITY)) {
                x[i] = 0.f;
                s_found[n_seg % 8] = n_seg + 1;
              }
          }
          const Place to = slot_of(true, n_tile);
          ok = mbar_wait_warp(&bars.empty[to.at], (to.turn & 1) ^ 1, wt);
          if (!ok) break;
          *reinterpret_cast<float4*>(sVs + n_tile % (C::VS > 0 ? C::VS : 1) * 128 + 4 * lane) = make_float4(x[0], x[1], x[2], x[3]);
          if (lane == 0) s_ev[n_tile % 4] = need;
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.sc_full[n_tile % 4]);
          scales = scales_of(j + 1, page1);
          page1 = j + 2 < sg.tile1 ? page_of(j + 2) : -1;
        }
        ++n_seg;
      }
    }
  } else if (warp >= 12) {
    regs_dec<C::REGS_WIDEN>();
    // ============================ widening / clearing =========================================
    const int w4 = warp % 4, r = w4 * 32 + lane;
    const bool masked = p.causal != 0 || p.tree_mask != nullptr;
    bool ok = true;
    int n_seg = 0, n_tile = 0;
    while (ok && walk.next(p, sg)) {
      bool found = false;
      // K's widening warps: page of the lane's key in a tile of this segment (-1: none), and its scale
      // (0 where there is no key); both are asked for ahead.
      auto page_of = [&](int j) {
        const int key = j * kKeys + r;
        return key < sg.L.len_kv ? __ldg(p.c.page_table + sg.bi * p.c.page_table_stride + key / p.c.page_size) : -1;
      };
      auto scale_of = [&](int j, int page) {
        if (page < 0 || page >= p.c.num_pages) return 0.f;
        return __ldg(p.c.k_scale + (static_cast<int64_t>(page) * p.c.h_kv + hk) * p.c.page_size + (j * kKeys + r) % p.c.page_size);
      };
      int page1 = -1;          // of the next tile
      float scale0 = 0.f;      // of this one
      if (E4 && warp < 16) {
        scale0 = scale_of(sg.tile0, page_of(sg.tile0));
        page1 = sg.tile0 + 1 < sg.tile1 ? page_of(sg.tile0 + 1) : -1;
      }
      for (int j = sg.tile0; ok && j < sg.tile1; ++j, ++n_tile) {
        const bool tail = masked && (j + 1) * kKeys > sg.off;
        const bool on = j * kKeys + r < sg.L.len_kv;
        if constexpr (E4) {
          const bool is_v = warp >= 16;
          const Place from = stage_of(is_v, n_tile), to = slot_of(is_v, n_tile);
          const int rs = from.at, s = to.at, left = sg.L.len_kv - j * kKeys;
          ok = mbar_wait_warp(&bars.raw_full[rs], from.turn & 1, wt);
          if (!ok) break;
          ok = mbar_wait_warp(&bars.empty[s], (to.turn & 1) ^ 1, wt);
          if (!ok) break;
          if (!is_v) {
            sKs[n_tile % (C::KS > 0 ? C::KS : 1) * 128 + r] = scale0;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.sc_full[n_tile % 4]);
            scale0 = scale_of(j + 1, page1);
            page1 = j + 2 < sg.tile1 ? page_of(j + 2) : -1;
          }
          // A lane takes its row, 16 codes at a time; the swizzles of both tiles put the 8 rows of a
          // quarter-warp into 8 different 16-byte columns.
          const uint8_t* src = sRaw + rs * C::RAW + r * 128;
          uint8_t* dst = sRing + s * C::TILE + r * 128;
          auto widen = [&](auto clear) {
#pragma unroll
            for (int ch = 0; ch < D / 16; ++ch) {
              const uint4 in = *reinterpret_cast<const uint4*>(src + (ch ^ (r & 7)) * 16);
              const uint32_t w[4] = {in.x, in.y, in.z, in.w};
              uint32_t out[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                out[e] = e4m3x2_to_f16x2(e % 2 ? w[e / 2] >> 16 : w[e / 2] & 0xFFFFu);
                if constexpr (decltype(clear)::value) out[e] = on ? finite_pair<false>(out[e], found) : 0u;
              }
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int u = 2 * ch + h;          // 16-byte unit of the 16-bit row
                *reinterpret_cast<uint4*>(dst + (u / 8) * 16384 + ((u % 8) ^ (r & 7)) * 16) =
                    make_uint4(out[4 * h], out[4 * h + 1], out[4 * h + 2], out[4 * h + 3]);
              }
            }
          };
          if (is_v && (tail || left < kKeys)) widen(std::true_type{});
          else widen(std::false_type{});
          if (found) s_found[n_seg % 8] = n_seg + 1;
          fence_proxy_async_smem();
          mbar_arrive(&bars.full[s]);
          mbar_arrive(&bars.raw_empty[rs]);
        } else {
          // Every tile's phase is followed, and its slot returned, by these warps too: a parity says
          // nothing about a phase that lies further back or ahead.
#pragma unroll 1
          for (int kv = 0; ok && kv < 2; ++kv) {
            const Place x = slot_of(kv != 0, n_tile);
            const int s = x.at;
            ok = mbar_wait_warp(&bars.full[s], x.turn & 1, wt);
            if (!ok) break;
            if (kv && needs_cleaning(p, sg, j)) {
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
              mbar_arrive(&bars.clean[s]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.empty[s]);
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
    uint32_t n_own = 0, n_other = 0;   // S of this warpgroup's slot and of the other so far
    uint32_t n_o[2] = {0, 0};      // results of each slot so far
    bool o1_pending = false;       // split, second warpgroup: its O of the segment before may still be read
    // This warp's 32 rows of Q of a segment to shared memory (one warpgroup's where both take the same
    // rows), a row by D / 8 lanes; returns the factor on the scores of this thread's row.  To be
    // called when the last S of the segment before has been read.  (A row a thread took 8-10 thousand
    // cycles: 32 rows for each warp instruction.)
    const int my_row = r0 + (split ? 0 : t * 128) + r, my_token = my_row / p.group;
    const int64_t q_row = (static_cast<int64_t>(hk) * p.group + my_row % p.group) * p.q_st[1] + my_token * p.q_st[2];
    auto load_q = [&](const Segment& g) -> float {
      constexpr int LR = D / 8, RI = 32 / LR;        // lanes of a row, rows of an instruction
      const bool store = !split || t == 0;
      const int u = lane % LR;
      float cs = wp.abs_scale_log2;
      const uint16_t* q = static_cast<const uint16_t*>(p.q) + g.bi * p.q_st[0] + u * 8;
      const unsigned live = __ballot_sync(0xffffffffu, my_row < p.rows && my_token < g.L.len_q);
#pragma unroll 1
      for (int i0 = 0; i0 < 32; i0 += 8 * RI) {
        uint4 x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int lr = i0 + i * RI + lane / LR;
          const int64_t at = __shfl_sync(0xffffffffu, q_row, lr);
          x[i] = make_uint4(0, 0, 0, 0);
          if ((live >> lr) & 1u) x[i] = *reinterpret_cast<const uint4*>(q + at);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int lr = i0 + i * RI + lane / LR, rr = quad * 32 + lr;
          uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] ^= wp.negate ? 0x80008000u : 0u;
          if constexpr (E4 && QT == kBF16) {
            // To F16 by a power of two that brings the row's largest element to [256, 512).
            uint32_t m = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) m = max(m, max(w[e] & 0x7FFFu, (w[e] >> 16) & 0x7FFFu));
#pragma unroll
            for (int o = 1; o < LR; o *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
            const int ex = static_cast<int>(m >> 7);
            const int sh = (ex == 0 || ex == 255) ? 0 : min(127 + 8 - ex, 126);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 f = unpack_pair<true>(w[e]);
              w[e] = pack_pair<false>(f.x * pow2(sh), f.y * pow2(sh));
            }
            // The row's own thread is lane lr.
            const int mine = __shfl_sync(0xffffffffu, sh, lane % RI * LR);
            if (lane / RI == i0 / RI + i) cs *= pow2(-mine);
          }
          if (store)
            *reinterpret_cast<uint4*>(sQ + t * C::TILE + (u / 8) * 16384 + rr * 128 + ((u % 8) ^ (rr & 7)) * 16) =
                make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      if (store) {
        fence_proxy_async_smem();
        mbar_arrive(&bars.q_full[t]);
      }
      // Not 0, for a scale and a row of next to nothing: hidden scores of -inf would become NaN.
      return fmaxf(cs, 0x1p-149f);
    };
    // O of this thread's row times a factor; by a whole warp, when the products so far are done.
    auto rescale_o = [&](float by) {
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t ov[32];
        tmem_ld32(o_addr + c * 32, ov);
        tmem_ld_wait();
        reg_fence32(ov);
#pragma unroll
        for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * by);
        tmem_st32(o_addr + c * 32, ov);
      }
    };
    bool more = walk.next(p, sg);
    float cs = more ? load_q(sg) : 0.f;
    while (ok && more) {
      const int row = my_row, token = my_token;
      const bool live = row < p.rows && token < sg.L.len_q;
      const int n = sg.tile1 - sg.tile0;
      const int step = split ? 2 : 1, first = split ? t : 0;
      Segment next;
      more = walk.next(p, next);
      if (more && row < p.rows) {      // its Q starts towards L2
        const uint16_t* q = static_cast<const uint16_t*>(p.q) + next.bi * p.q_st[0] + q_row;
        prefetch_l2(q);
        if (D > 64) prefetch_l2(q + 64);
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
      int v = kMinV;              // E4M3
      for (int i = first; i < n; i += step, ++n_own) {
        if (!mbar_wait_warp(&bars.s_full[t], n_own & 1, wt)) { ok = false; break; }
        tc_fence_after();
        const int key0 = (sg.tile0 + i) * kKeys;
        int v_tile = 0;             // E4M3: the v that the tile's values need; scales of K and V
        const float *ks = nullptr, *vs = nullptr;
        if constexpr (E4) {
          const int tile = n_tile + i;
          if (!mbar_wait_warp(&bars.sc_full[tile % 4], (tile / 4) & 1, wt)) { ok = false; break; }
          v_tile = s_ev[tile % 4];
          ks = sKs + tile % C::KS * 128;
          vs = sVs + tile % C::VS * 128;
        }
        const bool need = key0 + kKeys > sg.L.len_kv || (masked && key0 + kKeys > sg.off) || bad;
        uint32_t vis[4];       // visible columns
        if (need) {
          int lim = sg.L.len_kv - 1;
          if (p.causal) lim = min(lim, sg.off + token);
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int k0 = key0 + 32 * w, in = lim - k0 + 1;
            uint32_t v = in <= 0 ? 0u : in >= 32 ? 0xFFFFFFFFu : (1u << in) - 1u;
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
                if (key < sg.L.len_kv) {
                  const int pg = __ldg(pages + key / p.c.page_size);
                  if (pg < 0 || pg >= p.c.num_pages) v &= h ? 0x0000FFFFu : 0xFFFF0000u;
                }
              }
            }
            vis[w] = v;
          }
          __syncwarp();
        }
        // The row's 128 scores come in halves of 64 columns, each with its own step of the running
        // maximum; P takes the columns of the first quarter and then of the second, both read by then.
        // The reference m_ref is an integer, so the rare step between the halves scales the first
        // half's P, already rounded, exactly.  (One body for both: instruction fetch, not registers,
        // limits an unrolled one.)
        float alpha = 1.f, alpha_v = 1.f;
        int shift = 0;              // E4M3: log2 of what vs / 2^v takes beyond the scales as they are stored
        if constexpr (E4) {
          const int s0 = scale_exponent(v_tile);
          if (v_tile > v) {
            int least = v_tile;
            if (need) {      // keys that the row does not see may not move it: looked through one by one, being rare
              uint32_t top = 0;
#pragma unroll 1
              for (int c = 0; c < 32; ++c) {
#pragma unroll
                for (int w = 0; w < 4; ++w)
                  if ((vis[w] >> c) & 1u) top = max(top, __float_as_uint(fabsf(vs[32 * w + c])));
              }
              least = top == 0 ? v : needed_v(top) + s0;
            }
            if (least > v) {
              const int now = min(least + 1, kMaxV);      // (one more, so that it seldom moves again)
              alpha_v = pow2(max(v - now, -126));
              v = now;
            }
          }
          __syncwarp();
          // At -70 nothing is left of the weights in F16 (their scales are below 1 then); above 80 are rows that see
          // scales of next to nothing beside a hidden one of over 2^60.
          shift = min(max(s0 - v, -70), 80);
        }
        const float2 cs2 = make_float2(cs, cs);
        float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          uint32_t sv[64];
          tmem_ld32(s_addr + h * 64, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
          tmem_ld32(s_addr + h * 64 + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
          tmem_ld_wait();
          reg_fence32(&sv[0]);
          reg_fence32(&sv[32]);
          if constexpr (E4) {
#pragma unroll
            for (int c = 0; c < 64; c += 4) {
              const float4 k = *reinterpret_cast<const float4*>(ks + h * 64 + c);
              const float2 a = mul2(make_float2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])), make_float2(k.x, k.y));
              const float2 b = mul2(make_float2(__uint_as_float(sv[c + 2]), __uint_as_float(sv[c + 3])), make_float2(k.z, k.w));
              sv[c] = __float_as_uint(a.x);
              sv[c + 1] = __float_as_uint(a.y);
              sv[c + 2] = __float_as_uint(b.x);
              sv[c + 3] = __float_as_uint(b.y);
            }
          }
          if (need) {
            const uint32_t v0 = h ? vis[2] : vis[0], v1 = h ? vis[3] : vis[1];
#pragma unroll
            for (int c = 0; c < 64; ++c)
              if (!(((c < 32 ? v0 : v1) >> (c % 32)) & 1u)) sv[c] = __float_as_uint(-INFINITY);
          }
          float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
          for (int c = 0; c < 64; c += 8) {
            mx0 = max3(mx0, __uint_as_float(sv[c]), __uint_as_float(sv[c + 1]));
            mx1 = max3(mx1, __uint_as_float(sv[c + 2]), __uint_as_float(sv[c + 3]));
            mx2 = max3(mx2, __uint_as_float(sv[c + 4]), __uint_as_float(sv[c + 5]));
            mx3 = max3(mx3, __uint_as_float(sv[c + 6]), __uint_as_float(sv[c + 7]));
          }
          const float m_cand = max3(mx0, mx1, fmaxf(mx2, mx3)) * cs;
          const bool up = m_cand > m_ref + C::THRESH;
          if (__any_sync(0xffffffffu, up)) {
            const float m_new = up ? ceilf(m_cand) : m_ref, a = up ? ex2(m_ref - m_new) : 1.f;
            m_ref = m_new;
            alpha *= a;
            if (h == 1) {
              acc0 = mul2(acc0, make_float2(a, a));
              acc1 = mul2(acc1, make_float2(a, a));
              uint32_t pv[32];
              tmem_st_wait();
              tmem_ld32(s_addr, pv);
              tmem_ld_wait();
              reg_fence32(pv);
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const float2 f = unpack_pair<BF>(pv[e]);
                pv[e] = pack_pair<BF>(f.x * a, f.y * a);
              }
              tmem_st32(s_addr, pv);
            }
          }
          const float nm = m_ref == -INFINITY ? 0.f : C::P_OFF - m_ref + (E4 ? static_cast<float>(shift) : 0.f);
          const float2 nm2 = make_float2(nm, nm);
          uint32_t pk[32];
#pragma unroll
          for (int c = 0; c < 64; c += 4) {
            const float2 x01 = fma2(make_float2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])), cs2, nm2);
            const float2 x23 = fma2(make_float2(__uint_as_float(sv[c + 2]), __uint_as_float(sv[c + 3])), cs2, nm2);
            float2 p01 = make_float2(ex2(x01.x), ex2(x01.y)), p23 = make_float2(ex2(x23.x), ex2(x23.y));
            acc0 = add2(acc0, p01);
            acc1 = add2(acc1, p23);
            if constexpr (E4) {
              const float4 f = *reinterpret_cast<const float4*>(vs + h * 64 + c);
              p01 = mul2(p01, make_float2(f.x, f.y));
              p23 = mul2(p23, make_float2(f.z, f.w));
            }
            pk[c / 2] = pack_pair<BF>(p01.x, p01.y);
            pk[c / 2 + 1] = pack_pair<BF>(p23.x, p23.y);
          }
          __syncwarp();
          tmem_st32(s_addr + h * 32, pk);
        }
        l = l * alpha + ((acc0.x + acc0.y) + (acc1.x + acc1.y)) * (E4 ? pow2(-shift) : 1.f);
        // The block before has added to O already: its P V was issued ahead of this block's S.
        alpha *= alpha_v;
        if (i > first && __any_sync(0xffffffffu, alpha != 1.f)) rescale_o(alpha);
        tmem_st_wait();
        tc_fence_before();
        if (o1_pending) {              // this tile's P V overwrites O
          if (!mbar_wait_warp(&bars.o1_free, (n_seg - 1) & 1, wt)) { ok = false; break; }
          o1_pending = false;
        }
        mbar_arrive(&bars.p_full[t]);
      }
      if (!ok) break;
      n_other += split ? (n + t) / 2 : n;
      n_tile += n;
      // ---- the next segment's Q, so that its first S runs while this one's results leave ----------
      if (more) {
        // Where both warpgroups shared the rows, the other slot's last S has to be done with Q too.
        if (split && t == 0 && n > 1 && !mbar_wait_warp(&bars.s_full[1], (n_other - 1) & 1, wt)) { ok = false; break; }
        cs = load_q(next);
      }
      // ---- the segment's result: this thread's row ------------------------------------------------
      // Split, second warpgroup: its part of a row's keys goes to the first one's thread of that row,
      // the O of both lying in the same TMEM lane.
      if (split && t == 1) {
        if (o1_pending && !mbar_wait_warp(&bars.o1_free, (n_seg - 1) & 1, wt)) { ok = false; break; }
        s_ml[r] = make_float2(m_ref, l);
        if constexpr (E4) s_v[r] = v;
        mbar_arrive(&bars.ml_full);
        o1_pending = true;
        ++n_seg;
        sg = next;
        continue;
      }
      if (!mbar_wait_warp(&bars.o_full[t], n_o[0] & 1, wt)) { ok = false; break; }
      ++n_o[0];
      const bool two = split && n > 1;
      float f0 = 1.f, f1 = 0.f;
      if (split) {
        if (!mbar_wait_warp(&bars.ml_full, n_seg & 1, wt)) { ok = false; break; }
        if (two) {
          if (!mbar_wait_warp(&bars.o_full[1], n_o[1] & 1, wt)) { ok = false; break; }
          ++n_o[1];
          const float2 ml0 = make_float2(m_ref, l), ml1 = s_ml[r];
          const float m = fmaxf(l != 0.f ? m_ref : -INFINITY, ml1.y != 0.f ? ml1.x : -INFINITY);
          f0 = part_weight(ml0, m);
          f1 = part_weight(ml1, m);
          l = (f0 == 0.f ? 0.f : l * f0) + (f1 == 0.f ? 0.f : ml1.y * f1);
          m_ref = m;
          if constexpr (E4) {
            const int v0 = v, v1 = s_v[r];
            v = max(v0, v1);
            f0 *= pow2(max(v0 - v, -126));
            f1 *= pow2(max(v1 - v, -126));
          }
        }
      }
      // E4M3: 2^v joins O (and see sdpa_decode.cu on values near fp32's end).
      float up = 1.f;
      if constexpr (E4) {
        up = pow2(v);
        if (v > kNearV && l > 0.f && l < INFINITY) {
          const int e = static_cast<int>(__float_as_uint(l) >> 23) - 127 + 12;
          up *= pow2(-e);
          l *= pow2(-e);
          m_ref += static_cast<float>(e);
        }
      }
      tc_fence_after();
      const bool whole = sg.tile0 == 0 && sg.tile1 == sg.n_tiles;
      const int64_t part = 2 * static_cast<int64_t>(blockIdx.x) + (sg.tile0 == 0 ? 1 : 0);
      const bool none = !live || l == 0.f;
      const float inv = none ? 0.f : 1.f / l;
      const bool fix = live && s_found[n_seg % 8] == n_seg + 1;
      const int64_t out = row < p.rows ? row_offset(p, p.o_st, sg.bi, hk, row) : 0;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t ov[32];
        __syncwarp();          // (the TMEM loads are the whole warp's)
        tmem_ld32(o_addr + c * 32, ov);
        if (two) {
          uint32_t o1[32];
          tmem_ld32(o_addr + D + c * 32, o1);
          tmem_ld_wait();
          reg_fence32(ov);
          reg_fence32(o1);
#pragma unroll
          for (int e = 0; e < 32; ++e)
            ov[e] = __float_as_uint((f0 == 0.f ? 0.f : __uint_as_float(ov[e]) * f0) + (f1 == 0.f ? 0.f : __uint_as_float(o1[e]) * f1));
        } else {
          tmem_ld_wait();
          reg_fence32(ov);
        }
        if constexpr (E4) {
#pragma unroll
          for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * up);
        }
        if (row < p.rows) {
          if (fix) {
            for (int e = 0; e < 32; ++e)
              ov[e] = __float_as_uint(add_nonfinite<D, CT>(p, sg.bi, hk, sg.L, row, c * 32 + e, sg.tile0 * kKeys,
                                                           min(sg.tile1 * kKeys, sg.L.len_kv), __uint_as_float(ov[e])));
          }
          if (!whole) {
            float4* dst = reinterpret_cast<float4*>(p.part_o) + (part * (D / 4) + c * 8) * 256 + t * 128 + r;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              dst[e * 256] = make_float4(__uint_as_float(ov[4 * e]), __uint_as_float(ov[4 * e + 1]),
                                         __uint_as_float(ov[4 * e + 2]), __uint_as_float(ov[4 * e + 3]));
          } else {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + out + c * 32);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t w[4];
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const float a = __uint_as_float(ov[8 * e + 2 * x]), b = __uint_as_float(ov[8 * e + 2 * x + 1]);
                w[x] = none ? 0u : pack_pair<QT == kBF16>(a * inv, b * inv);
              }
              dst[e] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
        __syncwarp();
      }
      if (row < p.rows) {
        if (!whole)
          *reinterpret_cast<float2*>(p.part_ml + 2 * (part * 256 + t * 128 + r)) = make_float2(m_ref, l);
        else if (p.lse)
          p.lse[lse_offset(p, sg.bi, hk, row)] = none ? -INFINITY : natural_lse(m_ref - C::P_OFF, l);
      }
      tc_fence_before();     // O has been read: the next segment's first P V follows a later arrival
      if (split) mbar_arrive(&bars.o1_free);
      ++n_seg;
      sg = next;
    }
  }

  tc_fence_before();
  __syncthreads();
  // If a role gave up, copies may still be in flight: let them land before the CTA ends.
  if (producer && *abort_flag) {
    const int n = warp == 2 ? (E4 ? C::RV : C::NV) : (E4 ? C::RK : C::NK);
    for (int k = max(issued - n, 0); k < issued; ++k) {
      const Place x = E4 ? stage_of(warp == 2, k) : slot_of(warp == 2, k);
      mbar_wait_drain(E4 ? &bars.raw_full[x.at] : &bars.full[x.at], x.turn & 1);
    }
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of sequences that more than one team worked on, and writes the rows that no key
// reaches: 32 rows a CTA, a lane a row, every warp D / 32 groups of four elements, in the parts' order.
template <int D, int QT>
__global__ void __launch_bounds__(256) decode_wide_combine_kernel(const __grid_constant__ DecodeParams p, float p_off) {
  constexpr int NG = D / 32;
  __shared__ uint2 s_out[32][D / 4 + 1];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int groups = (min(p.rows, 256) + 31) / 32;
  const Parts u = find_parts(p, blockIdx.x / groups, lane);
  const int r = blockIdx.x % groups * 32 + lane, row = u.r0 + r;
  griddep_wait();   // (by every CTA, so that this grid never ends before the one it follows)
  if (u.n == 1) return;
  float m = -INFINITY, l = 0.f;
  float4 x[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) x[g] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (row < p.rows) {
#pragma unroll 4
    for (int k = 0; k < u.n; ++k) {
      const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + 2 * (u.part(k) * 256 + r));
      if (ml.y != 0.f) m = fmaxf(m, ml.x);
    }
#pragma unroll 4
    for (int k = 0; k < u.n; ++k) {
      const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + 2 * (u.part(k) * 256 + r));
      const float f = part_weight(ml, m);
      l += ml.y * f;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const float4 v = reinterpret_cast<const float4*>(p.part_o)[(u.part(k) * (D / 4) + g * 8 + warp) * 256 + r];
        x[g].x += f == 0.f ? 0.f : v.x * f;
        x[g].y += f == 0.f ? 0.f : v.y * f;
        x[g].z += f == 0.f ? 0.f : v.z * f;
        x[g].w += f == 0.f ? 0.f : v.w * f;
      }
    }
    const bool none = row / p.group >= u.L.len_q || l == 0.f;
    const float inv = none ? 0.f : 1.f / l;
#pragma unroll
    for (int g = 0; g < NG; ++g)
      s_out[lane][g * 8 + warp] = none ? make_uint2(0, 0)
                                       : make_uint2(pack_pair<QT == kBF16>(x[g].x * inv, x[g].y * inv),
                                                    pack_pair<QT == kBF16>(x[g].z * inv, x[g].w * inv));
    if (p.lse && warp == 0) p.lse[lse_offset(p, u.bi, u.hk, row)] = none ? -INFINITY : natural_lse(m - p_off, l);
  }
  __syncthreads();
  // A row of D / 4 words by as many neighbouring threads.
  for (int i = threadIdx.x; i < 32 * (D / 4); i += 256) {
    const int r2 = i / (D / 4), row2 = u.r0 + blockIdx.x % groups * 32 + r2;
    if (row2 < p.rows)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + row_offset(p, p.o_st, u.bi, u.hk, row2) + i % (D / 4) * 4) =
          s_out[r2][i % (D / 4)];
  }
}

template <int D, int CT, int QT>
cudaError_t launch_t(const WideParams& wp, cudaStream_t st) {
  using C = WideCfg<D, CT>;
  auto kern = decode_wide_kernel<D, CT, QT>;
  cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kern), C::SMEM);
  if (e != cudaSuccess) return e;
  const DecodeParams& p = wp.d;
  kern<<<p.ctas, C::THREADS, C::SMEM, st>>>(wp);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int groups = ((p.rows < 256 ? p.rows : 256) + 31) / 32;
  return launch_after(decode_wide_combine_kernel<D, QT>,
                      dim3(static_cast<unsigned>(p.c.b) * p.c.h_kv * p.row_tiles * groups), dim3(256), st, p, C::P_OFF);
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
  // A scale of zero as the least above it: products up to fp32's largest come to 2^-21, so every visible key weighs
  // the same, and hidden ones still come out as -inf.
  wp.abs_scale_log2 = p.scale_log2 == 0.f ? 0x1p-149f : fabsf(p.scale_log2);
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
