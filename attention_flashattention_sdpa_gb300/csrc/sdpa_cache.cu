// sdpa_cache.cu — a paged key/value cache, written and read.
//
// Write: row i of a sequence's new rows goes to position len_kv - len_q + i, K rotated on the way
// if asked.  E4M3: s = max(amax, 2^-60) / 448 for each token and head, code = x / s rounded to the
// nearest of E4M3's values.  Read: code * s, dense, zeros behind the sequence.
//
// Bound: memory.  A row of d elements is spread over d / 16 lanes of 16 elements each, which find
// the row's largest value by shuffles; a thread walks heads of one token, so that its angles and
// its page are looked up once.  Measured, 8 heads of 128, E4M3 from or to BF16: 4 prompts of 5001 to
// 8192 tokens written, K rotated, 36.4 us (4.9 TB/s, 73% of a copy: the roundings of a row wait for
// its largest value), 32 single tokens 2.9 us; 2 x 8192 tokens read 17.5 us (5.6 TB/s, 83%).
#include <cuda_fp8.h>

#include <type_traits>

#include "sdpa_rope.cuh"

namespace sdpa {
namespace {

constexpr int kThreads = 128;
constexpr int kSlots = 4;           // heads of a thread in shared memory: one worked on, the others on their way
constexpr float kE4M3Max = 448.f;
constexpr float kAmaxMin = 8.673617379884035e-19f;  // 2^-60

__device__ __forceinline__ uint32_t pack4_e4m3(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return (lo & 0xFFFFu) | (hi << 16);
}

// Scales of a row of K and of one of V held 16 elements a lane by the LANES lanes from m = 0 on, and
// what multiplies the elements, for both rows in every lane.  The lanes of even m find K's largest
// magnitude and divide, those of odd m V's.
struct RowScales {
  float k, v, k_inv, v_inv;
};

template <int LANES>
__device__ __forceinline__ RowScales row_scales(const float (&x)[16], const float (&y)[16], int m) {
  auto lane_max = [](const float (&e)[16]) {
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      a = ptx::max3_abs_nan(a, e[i], e[i + 1]);
      b = ptx::max3_abs_nan(b, e[i + 2], e[i + 3]);
    }
    return ptx::max3_abs_nan(a, b, 0.f);
  };
  const float ak = lane_max(x), av = lane_max(y);
  const bool odd = m & 1;
  float a = odd ? av : ak;
  a = ptx::max3_abs_nan(a, __shfl_xor_sync(0xffffffffu, odd ? ak : av, 1), 0.f);
#pragma unroll
  for (int o = 2; o < LANES; o *= 2) a = ptx::max3_abs_nan(a, __shfl_xor_sync(0xffffffffu, a, o), 0.f);
  const float scale = (a < kAmaxMin ? kAmaxMin : a) / kE4M3Max, inv = 1.f / scale;   // a NaN stays one
  const float other = __shfl_xor_sync(0xffffffffu, scale, 1), other_inv = __shfl_xor_sync(0xffffffffu, inv, 1);
  return odd ? RowScales{other, scale, other_inv, inv} : RowScales{scale, other, inv, other_inv};
}

__device__ __forceinline__ void cp_async16(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_u32(to)), "l"(from) : "memory");
}

struct Slot {
  int64_t page;   // -1: none
  int slot;
};

__device__ __forceinline__ Slot find_slot(const CacheArgs& c, int bi, int pos) {
  Slot r{-1, 0};
  if (pos >= 0 && pos < c.max_len) {
    const int col = pos / c.page_size;
    const int page = __ldg(c.page_table + bi * c.page_table_stride + col);
    if (page >= 0 && page < c.num_pages) r.page = page;
    r.slot = pos - col * c.page_size;
  }
  return r;
}

__device__ __forceinline__ int clamp_len(const int32_t* lens, int i, int top) {
  return lens ? min(max(__ldg(lens + i), 0), top) : top;
}

// An item of a row as it lies in memory, and widened.
struct Raw {
  uint4 u[2];
};

__device__ __forceinline__ Raw load_raw(const void* base, int64_t row, int lo, int hi) {
  const uint16_t* p = static_cast<const uint16_t*>(base) + row;
  return Raw{{*reinterpret_cast<const uint4*>(p + lo), *reinterpret_cast<const uint4*>(p + hi)}};
}

template <int DT>
__device__ __forceinline__ void unpack_item(const Raw& r, float (&x)[16]) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(r.u);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = unpack16<DT>(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

// Stores an item (16 values, runs at lo and hi) of one row; lane 0 of the row stores its scale.
template <int D, int CT>
__device__ __forceinline__ void store_item(uint8_t* row, float* scale_at, int m, int lo, int hi, const float (&x)[16],
                                           float scale, float inv, bool live) {
  if (!live) return;
  if constexpr (CT == kE4M3) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = make_float2(inv, inv), a = ptx::mul2(make_float2(x[4 * i], x[4 * i + 1]), f),
                   b = ptx::mul2(make_float2(x[4 * i + 2], x[4 * i + 3]), f);
      w[i] = pack4_e4m3(a.x, a.y, b.x, b.y);
    }
    if (hi == lo + 8) {
      *reinterpret_cast<uint4*>(row + lo) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      *reinterpret_cast<uint2*>(row + lo) = make_uint2(w[0], w[1]);
      *reinterpret_cast<uint2*>(row + hi) = make_uint2(w[2], w[3]);
    }
    if (m == 0) *scale_at = scale;
  } else {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack16<CT>(x[2 * i], x[2 * i + 1]);
    *reinterpret_cast<uint4*>(row + 2 * lo) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(row + 2 * hi) = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// ROPE: 0 none, 1 rot a multiple of 16; any even rot, 2 with the angles computed once for all heads, 3 for each head anew (walks of few heads).
// (A floor of one block an SM leaves the compiler the registers it wants, for rotated rows to E4M3 112 with RING and 123 without, four
// blocks an SM either way: 4 x 8192 tokens of 8 heads of 128 41.0 -> 40.1 us.)
// AXES: K has several positions a token.  RING: a thread's next heads come through shared memory, each thread's in slots of
// its own (it waits for its own copies alone), where whole heads are rotated and a thread has four or more: 4 x 4096 tokens of 8 heads to E4M3
// 25.3 -> 23.2 us, 4 x 8192 40.8 -> 40.1, to BF16 50.2 -> 48.4 (with 3 slots or 6 about 5% more).  Otherwise the next one comes into registers:
// with too little arithmetic between its loads a thread waits for the copies (4 x 4096 tokens to E4M3, half of each head rotated, 24.5 us
// against 26.2; none 20.2 against 30.4).
template <int D, int DT, int CT, int ROPE, bool AXES, bool RING>
__global__ void __launch_bounds__(kThreads, 1) cache_write_kernel(const __grid_constant__ CacheRowsParams p, int per,
                                                            bool small) {
  constexpr int LANES = D / 16;
  const Spot who = find_spot(static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x, LANES, p.c.b, p.s, small);
  const int m = who.m, grp = who.grp, bi = who.bi, si = who.si;
  const int len_q = clamp_len(p.seq_lens_q, bi, p.s);
  const int len_kv = clamp_len(p.c.seq_lens_kv, bi, p.c.max_len);
  const int pos = len_kv - len_q + si;
  Slot at{-1, 0};
  if (grp * per < p.c.h_kv && si < len_q) at = find_slot(p.c, bi, pos);
  const bool live = at.page >= 0;
  // The lanes of a row leave together; a warp stays while any of its rows is live.
  if (!__any_sync(0xffffffffu, live)) return;

  // (V as eight elements of each half of the row, whose loads lie closer: 36.6 -> 37.7 us, its codes then
  // leave 8 bytes at a time.)
  RopeItem it{m * 16, m * 16 + 8, false};
  if constexpr (ROPE == 1) it = rope_item(p.r, m);
  const int h0 = grp * per, h_end = min(p.c.h_kv, h0 + per);
  // A head's K and V are loaded while the one before it is worked on, the first while the angles
  // are computed.
  Raw k_next, v_next;
  __shared__ uint4 ring[RING ? kSlots : 1][4][RING ? kThreads : 1];
  auto fetch = [&](int h) {
    const bool there = live && h < h_end;
    if constexpr (RING) {
      if (there) {
        auto& to = ring[(h - h0) % kSlots];
        const uint16_t* a = static_cast<const uint16_t*>(p.k) + bi * p.k_st[0] + h * p.k_st[1] + si * p.k_st[2];
        const uint16_t* b = static_cast<const uint16_t*>(p.v) + bi * p.v_st[0] + h * p.v_st[1] + si * p.v_st[2] + m * 16;
        cp_async16(&to[0][threadIdx.x], a + it.lo);
        cp_async16(&to[1][threadIdx.x], a + it.hi);
        cp_async16(&to[2][threadIdx.x], b);
        cp_async16(&to[3][threadIdx.x], b + 8);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    } else if (there) {
      k_next = load_raw(p.k, bi * p.k_st[0] + h * p.k_st[1] + si * p.k_st[2], it.lo, it.hi);
      v_next = load_raw(p.v, bi * p.v_st[0] + h * p.v_st[1] + si * p.v_st[2], m * 16, m * 16 + 8);
    }
  };
#pragma unroll
  for (int j = 0; j < (RING ? kSlots - 1 : 1); ++j) fetch(h0 + j);
  if constexpr (CT == kE4M3 && !RING) {
    // The row's other heads start towards L2, a line a lane: 4 x 8192 tokens of 8 heads, half of each rotated, 44.3 -> 41.1 us; not rotated
    // 4 x 4096 21.0 -> 20.2, 4 x 8192 36.9 -> 37.9.  (16-bit caches, copied without that much work between, were slower so: 44.6 -> 47.8.)
    constexpr int LINES = D / 64;
    for (int i = m; live && i < (h_end - h0 - 1) * LINES; i += LANES) {
      const int h = h0 + 1 + i / LINES, e = i % LINES * 64;
      ptx::prefetch_l2(static_cast<const uint16_t*>(p.k) + bi * p.k_st[0] + h * p.k_st[1] + si * p.k_st[2] + e);
      ptx::prefetch_l2(static_cast<const uint16_t*>(p.v) + bi * p.v_st[0] + h * p.v_st[1] + si * p.v_st[2] + e);
    }
  }
  RopePos<AXES> rpos = {};
  float c[ROPE == 2 ? 16 : 8], s[ROPE == 2 ? 16 : 8];
  if constexpr (ROPE != 0) {
    if (live) rpos = rope_pos<AXES>(p.r, bi, si, pos);
  }
  if constexpr (ROPE == 1) {
    if (it.turned && live) {
      // (Interleaved pairs as 16 neighbours instead: 48.8 us against 40.3 for 4 x 8192 tokens to E4M3, 66 against 49 in BF16.)
      const int far = p.r.interleaved ? p.r.rot / 4 + m * 4 : m * 8 + 4, near = p.r.interleaved ? m * 4 : m * 8;   // pairs 4..7, 0..3
      const uint32_t axes = (axes_from<AXES>(p.r, near) & 0xFFu) | axes_from<AXES>(p.r, far) << 8;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        rope_angle(p.r, __ldg(p.r.table + (i < 4 ? near + i : far + i - 4)), rpos.of(axes >> (2 * i)), c[i], s[i]);
    }
  }
  // 16 neighbours, each with an angle and a partner of its own, `other` elements away.
  const int half = p.r.rot / 2, turns = ROPE >= 2 ? min(16, p.r.rot - m * 16) : 0;
  auto is_first = [&](int i) { return p.r.interleaved ? i % 2 == 0 : m * 16 + i < half; };
  auto pair_of = [&](int i) { return p.r.interleaved ? (m * 16 + i) / 2 : m * 16 + i - (is_first(i) ? 0 : half); };
  if constexpr (ROPE == 2) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int pair = pair_of(i);
      if (live && i < turns) rope_angle(p.r, __ldg(p.r.table + pair), rpos.of(axes_from<AXES>(p.r, pair)), c[i], s[i]);
    }
  }
  // Every lane of the warp runs the same number of turns (the shuffles need them all).
  for (int j = 0; j < per; ++j) {
    const int h = h0 + j;
    const bool on = live && h < h_end;
    float x[16], y[16];
    Raw k_now, v_now;
    if constexpr (RING) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kSlots - 2) : "memory");
      const auto& from = ring[j % kSlots];
      k_now = Raw{{from[0][threadIdx.x], from[1][threadIdx.x]}};
      v_now = Raw{{from[2][threadIdx.x], from[3][threadIdx.x]}};
      fetch(h + kSlots - 1);        // into the slot of the head before this one
    } else {
      k_now = k_next;
      v_now = v_next;
      if (j + 1 < per) fetch(h + 1);
    }
    if (on) {
      unpack_item<DT>(k_now, x);
      unpack_item<DT>(v_now, y);
      if constexpr (ROPE == 1) {
        if (it.turned) {
          if (p.r.interleaved) rope_turn(true, x, c, s);
          else rope_turn(false, x, c, s);
        }
      }
      if constexpr (ROPE == 2) {
        const int64_t krow = bi * p.k_st[0] + h * p.k_st[1] + si * p.k_st[2] + m * 16;
        float a[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) a[i] = x[i];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (i >= turns) continue;
          const bool first = is_first(i);
          const float b = p.r.interleaved ? a[i ^ 1] : load16<DT>(p.k, krow + i + (first ? half : -half));
          x[i] = first ? a[i] * c[i] - b * s[i] : b * s[i] + a[i] * c[i];
        }
      }
      if constexpr (ROPE == 3) {
        const int64_t krow = bi * p.k_st[0] + h * p.k_st[1] + si * p.k_st[2];
#pragma unroll 1
        for (int i = 0; i < 16; ++i) {
          const int e = m * 16 + i;
          if (e >= p.r.rot) break;
          const bool first = is_first(i);
          const int pair = pair_of(i), other = p.r.interleaved ? e ^ 1 : first ? e + half : e - half;
          float cc, ss;
          rope_angle(p.r, __ldg(p.r.table + pair), rpos.of(axes_from<AXES>(p.r, pair)), cc, ss);
          const float a = load16<DT>(p.k, krow + e), b = load16<DT>(p.k, krow + other);
          x[i] = first ? a * cc - b * ss : b * ss + a * cc;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = y[i] = 0.f;
    }
    RowScales rs{0.f, 0.f, 0.f, 0.f};
    if constexpr (CT == kE4M3) rs = row_scales<LANES>(x, y, m);
    const int64_t sc = (at.page * p.c.h_kv + h) * p.c.page_size + at.slot;
    store_item<D, CT>(p.c.k + at.page * p.c.k_st[0] + h * p.c.k_st[1] + at.slot * p.c.k_st[2], p.c.k_scale + sc, m,
                      it.lo, it.hi, x, rs.k, rs.k_inv, on);
    store_item<D, CT>(p.c.v + at.page * p.c.v_st[0] + h * p.c.v_st[1] + at.slot * p.c.v_st[2], p.c.v_scale + sc, m,
                      m * 16, m * 16 + 8, y, rs.v, rs.v_inv, on);
  }
}

// One thread: 16 elements of K and of V of one row, eight of each half of it, so that neighbouring
// lanes write neighbouring 16 bytes (16 neighbouring elements: 19.2 us against 17.5 for 2 x 8192 tokens of
// 8 heads).  Two or four heads a thread, their loads in flight together, are no faster: 17.8 and 17.5 us.
template <int D, int DT, int CT>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const __grid_constant__ CacheRowsParams p, bool small) {
  constexpr int LANES = D / 16, ES = CT == kE4M3 ? 1 : 2;
  const Spot who = find_spot(static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x, LANES * p.c.h_kv, p.c.b, p.s, small);
  const int m = who.m % LANES, h = who.m / LANES, bi = who.bi, si = who.si;
  if (who.grp > 0) return;
  Slot at{-1, 0};
  if (si < clamp_len(p.c.seq_lens_kv, bi, p.c.max_len)) at = find_slot(p.c, bi, si);
  using Half = std::conditional_t<CT == kE4M3, uint2, uint4>;      // eight elements as stored
  Half in[2][2];
  float scale[2] = {0.f, 0.f};
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    in[t][0] = in[t][1] = Half{};
    if (at.page >= 0) {
      const int64_t* st = t ? p.c.v_st : p.c.k_st;
      const uint8_t* src = (t ? p.c.v : p.c.k) + at.page * st[0] + h * st[1] + at.slot * st[2] + m * 8 * ES;
#pragma unroll
      for (int i = 0; i < 2; ++i) in[t][i] = __ldg(reinterpret_cast<const Half*>(src + i * (D / 2) * ES));
      if constexpr (CT == kE4M3)
        scale[t] = __ldg((t ? p.c.v_scale : p.c.k_scale) + (at.page * p.c.h_kv + h) * p.c.page_size + at.slot);
    }
  }
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int64_t* st = t ? p.v_st : p.k_st;
    uint16_t* dst = static_cast<uint16_t*>(t ? p.v : p.k) + bi * st[0] + h * st[1] + si * st[2] + m * 8;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint4 out;
      if constexpr (CT == kE4M3) {
        const uint32_t iw[2] = {in[t][i].x, in[t][i].y};
        uint32_t ow[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(iw[e / 2] >> (16 * (e % 2))), __NV_E4M3);
          const float2 f = ptx::mul2(__half22float2(__half2(hr)), make_float2(scale[t], scale[t]));
          ow[e] = pack16<DT>(f.x, f.y);
        }
        out = make_uint4(ow[0], ow[1], ow[2], ow[3]);
      } else {
        out = in[t][i];
      }
      *reinterpret_cast<uint4*>(dst + i * (D / 2)) = out;
    }
  }
}

template <int D, int DT, int CT>
cudaError_t write_t(const CacheRowsParams& p, int num_sms, cudaStream_t st) {
  const int64_t tokens = static_cast<int64_t>(p.c.b) * p.s;
  const bool vec = p.r.rot % 16 == 0, whole = p.rope && p.r.rot == D;
  // Heads a thread walks: as many as leave 512 threads an SM (with 1024, 4096 tokens of 8 heads, rotated, to E4M3: 14.1 us against 10.5).
  // Walks of `cheap` heads and more, which are mostly copied, need more threads, 1024: 4 and 8 that are not rotated (16384 tokens of 8 heads to
  // E4M3: 19.8 us, 22.0 with 512), 8 that are rotated in part.
  auto walk = [&](int per, int cheap) {
    while (per > 1 && tokens * (D / 16) * ((p.c.h_kv + per - 1) / per) < static_cast<int64_t>(num_sms) * (per >= cheap ? 1024 : 512)) per /= 2;
    return per;
  };
  const int longest = p.c.h_kv > 4 ? 8 : p.c.h_kv > 2 ? 4 : p.c.h_kv;
  int per;
  bool each = false;
  if (p.rope && !vec) {
    // Angles computed once for all heads cost 168 to 186 registers a thread.  They pay for walks of 2 heads and more of adjacent pairs in 16 bits
    // (16384 tokens of 2 heads 19.3 us, with each head's anew 21.1), of 4 of halves (4096 of 16: 31.9 against 38) and of adjacent pairs to
    // E4M3 (34.6 against 36.5), of 8 of halves to E4M3 (16384 of 8: 67 against 70).  One less: 16384 of 1 in 16 bits, pairs 16.5 against 13.7;
    // to E4M3 16384 of 2, pairs 25.4 against 20.8, halves (4096 of 16) 42.3 against 35.6.
    per = walk(longest, 16);
    each = per < (CT == kE4M3 ? 2 : 1) * (p.r.interleaved ? 2 : 4);
    if (each) per = walk(longest, 1);
  } else {
    // (12 heads to E4M3 as three walks of 4, not as one of 8 and half a one: 16384 tokens of 64 elements, rotated, 19.7 us against 21.1.)
    const bool thirds = CT == kE4M3 && p.c.h_kv > 8 && (p.c.h_kv - 1) % 8 < 4;
    per = walk(thirds ? 4 : longest, !p.rope ? 4 : whole ? 16 : 8);
  }
  const int groups = (p.c.h_kv + per - 1) / per;
  const int64_t blocks = (tokens * (D / 16) * groups + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const unsigned grid = static_cast<unsigned>(blocks);
  const bool small = blocks * kThreads < (int64_t(1) << 31);
  auto run = [&](auto kernel) { kernel<<<grid, kThreads, 0, st>>>(p, per, small); };
  const bool ring = whole && per >= 4;
  if (!p.rope) run(cache_write_kernel<D, DT, CT, 0, false, false>);
  else if (vec && p.r.axes) run(ring ? cache_write_kernel<D, DT, CT, 1, true, true> : cache_write_kernel<D, DT, CT, 1, true, false>);
  else if (vec) run(ring ? cache_write_kernel<D, DT, CT, 1, false, true> : cache_write_kernel<D, DT, CT, 1, false, false>);
  else if (each) run(p.r.axes ? cache_write_kernel<D, DT, CT, 3, true, false> : cache_write_kernel<D, DT, CT, 3, false, false>);
  else run(p.r.axes ? cache_write_kernel<D, DT, CT, 2, true, false> : cache_write_kernel<D, DT, CT, 2, false, false>);
  return cudaGetLastError();
}

template <int D, int DT, int CT>
cudaError_t read_t(const CacheRowsParams& p, cudaStream_t st) {
  const int64_t blocks = (static_cast<int64_t>(p.c.b) * p.s * p.c.h_kv * (D / 16) + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  cache_read_kernel<D, DT, CT><<<static_cast<unsigned>(blocks), kThreads, 0, st>>>(p, blocks * kThreads < (int64_t(1) << 31));
  return cudaGetLastError();
}

template <int D>
cudaError_t write_d(const CacheRowsParams& p, int dt, int ct, int sms, cudaStream_t st) {
  if (dt == kBF16) return ct == kE4M3 ? write_t<D, kBF16, kE4M3>(p, sms, st) : write_t<D, kBF16, kBF16>(p, sms, st);
  return ct == kE4M3 ? write_t<D, kF16, kE4M3>(p, sms, st) : write_t<D, kF16, kF16>(p, sms, st);
}

template <int D>
cudaError_t read_d(const CacheRowsParams& p, int dt, int ct, cudaStream_t st) {
  if (dt == kBF16) return ct == kE4M3 ? read_t<D, kBF16, kE4M3>(p, st) : read_t<D, kBF16, kBF16>(p, st);
  return ct == kE4M3 ? read_t<D, kF16, kE4M3>(p, st) : read_t<D, kF16, kF16>(p, st);
}

}  // namespace

cudaError_t launch_cache_write(const CacheRowsParams& p, int dt, int ct, int num_sms, cudaStream_t st) {
  if (p.d == 64) return write_d<64>(p, dt, ct, num_sms, st);
  if (p.d == 128) return write_d<128>(p, dt, ct, num_sms, st);
  if (p.d == 256) return write_d<256>(p, dt, ct, num_sms, st);
  return cudaErrorInvalidValue;
}

cudaError_t launch_cache_read(const CacheRowsParams& p, int dt, int ct, cudaStream_t st) {
  if (p.d == 64) return read_d<64>(p, dt, ct, st);
  if (p.d == 128) return read_d<128>(p, dt, ct, st);
  if (p.d == 256) return read_d<256>(p, dt, ct, st);
  return cudaErrorInvalidValue;
}

}  // namespace sdpa
