// sdpa_cache.cu — a paged key/value cache, written and read.
//
// Write: row i of a sequence's new rows goes to position len_kv - len_q + i, K rotated on the way
// if asked.  E4M3: s = max(amax, 2^-60) / 448 for each token and head, code = x / s rounded to the
// nearest of E4M3's values.  Read: code * s, dense, zeros behind the sequence.
//
// Bound: memory.  A row of d elements is spread over d / 16 lanes of 16 elements each, which find
// the row's largest value by shuffles; a thread walks heads of one token, so that its angles and
// its page are looked up once.  Measured, 8 heads of 128, E4M3 from or to BF16: 4 prompts of 5001 to
// 8192 tokens written, K rotated, 36.5 us (4.9 TB/s, 73% of a copy: the roundings of a row wait for
// its largest value), 32 single tokens 3.0 us; 2 x 8192 tokens read 17.5 us (5.6 TB/s, 83%).
#include <cuda_fp8.h>

#include <type_traits>

#include "sdpa_rope.cuh"

namespace sdpa {
namespace {

constexpr int kThreads = 128;
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

// ROPE: 0 none, 1 rot a multiple of 16, 2 any even rot.
// (A floor of one block an SM lets the compiler hold a few more registers, 122, still four blocks: 38.5 ->
// 36.5 us.)
template <int D, int DT, int CT, int ROPE>
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
  auto fetch = [&](int h) {
    if (live && h < h_end) {
      k_next = load_raw(p.k, bi * p.k_st[0] + h * p.k_st[1] + si * p.k_st[2], it.lo, it.hi);
      v_next = load_raw(p.v, bi * p.v_st[0] + h * p.v_st[1] + si * p.v_st[2], m * 16, m * 16 + 8);
    }
  };
  fetch(h0);
  if constexpr (CT == kE4M3) {
    // The row's other heads start towards L2, a line a lane: 38.3 -> 36.5 us for the prompts above, 16 heads
    // 44.0 -> 41.0.  (16-bit caches, copied without that much work between, were slower so: 44.6 -> 47.8.)
    constexpr int LINES = D / 64;
    for (int i = m; live && i < (h_end - h0 - 1) * LINES; i += LANES) {
      const int h = h0 + 1 + i / LINES, e = i % LINES * 64;
      ptx::prefetch_l2(static_cast<const uint16_t*>(p.k) + bi * p.k_st[0] + h * p.k_st[1] + si * p.k_st[2] + e);
      ptx::prefetch_l2(static_cast<const uint16_t*>(p.v) + bi * p.v_st[0] + h * p.v_st[1] + si * p.v_st[2] + e);
    }
  }
  int rpos = pos;
  float c[8], s[8];
  if constexpr (ROPE != 0) {
    if (p.r.positions && live) rpos = p.r.positions[bi * p.r.positions_stride + si];
  }
  if constexpr (ROPE == 1) {
    if (it.turned && live) {
#pragma unroll
      for (int i = 0; i < 8; ++i) rope_angle(p.r, __ldg(p.r.table + m * 8 + i), rpos, c[i], s[i]);
    }
  }
  // Every lane of the warp runs the same number of turns (the shuffles need them all).
  for (int j = 0; j < per; ++j) {
    const int h = h0 + j;
    const bool on = live && h < h_end;
    float x[16], y[16];
    const Raw k_now = k_next, v_now = v_next;
    if (j + 1 < per) fetch(h + 1);
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
        // 16 neighbours; each finds its own partner and angle.
        const int64_t krow = bi * p.k_st[0] + h * p.k_st[1] + si * p.k_st[2];
        const int half = p.r.rot / 2;
#pragma unroll 1
        for (int i = 0; i < 16; ++i) {
          const int e = m * 16 + i;
          if (e >= p.r.rot) break;
          const int pair = p.r.interleaved ? e / 2 : e % half;
          const bool first = p.r.interleaved ? e % 2 == 0 : e < half;
          const int other = p.r.interleaved ? e ^ 1 : (first ? e + half : e - half);
          float cc, ss;
          rope_angle(p.r, __ldg(p.r.table + pair), rpos, cc, ss);
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
  int per = 8;   // heads a thread walks: as many as leave the GPU full
  while (per > 1 && tokens * (D / 16) * ((p.c.h_kv + per - 1) / per) < static_cast<int64_t>(num_sms) * 1024) per /= 2;
  const int groups = (p.c.h_kv + per - 1) / per;
  const int64_t blocks = (tokens * (D / 16) * groups + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const unsigned grid = static_cast<unsigned>(blocks);
  const bool small = blocks * kThreads < (int64_t(1) << 31);
  if (!p.rope) cache_write_kernel<D, DT, CT, 0><<<grid, kThreads, 0, st>>>(p, per, small);
  else if (p.r.rot % 16 == 0) cache_write_kernel<D, DT, CT, 1><<<grid, kThreads, 0, st>>>(p, per, small);
  else cache_write_kernel<D, DT, CT, 2><<<grid, kThreads, 0, st>>>(p, per, small);
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
