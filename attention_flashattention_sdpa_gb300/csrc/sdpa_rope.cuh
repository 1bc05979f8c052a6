// sdpa_rope.cuh — rotary positions: the angle of a pair, and 16-bit packing, shared by the
// rotation kernels and the cache write.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx.cuh"
#include "sdpa_internal.h"

namespace sdpa {

// cos and sin (times the factor) of one pair at position `pos`.  The table holds the turns per
// position as 64-bit binary fractions, so pos * table[i] modulo 2^64 is the angle's fraction of a turn, with
// nothing lost to its size (what an entry, computed in fp64, lacks counts pos times: 5e-7 radians at 2^30
// radians); its upper 32 bits, 1.5e-9 radians each, go on.  The nearest quarter turn is taken off in whole
// numbers as well.  The rest, at most pi/4, is x + dx: what the conversion to fp32 rounds off joins
// again by sin(x + dx) = sin x + dx cos x.  The Taylor series end after x^9 (sin, off by 2e-9) and
// x^10 (cos, off by 2e-10); the factor multiplies the 1 of cos and the x of sin without a rounding of
// its own, so that both results are off by little more than their last rounding.
__device__ __forceinline__ void rope_angle(const RopeArgs& r, int64_t turns, int pos, float& c, float& s) {
  const uint64_t phase = static_cast<uint64_t>(turns) * static_cast<uint64_t>(static_cast<int64_t>(pos));
  const uint32_t top = static_cast<uint32_t>(phase >> 32);
  const uint32_t quarter = (top + (1u << 29)) >> 30;                   // 0..3: a sum of 2^32 is 0 again
  const int32_t rest = static_cast<int32_t>(top - (quarter << 30));    // [-2^29, 2^29) of 2^32 a turn
  constexpr float kHi = 1.4629180792671596e-9f;                        // 2 pi / 2^32 as fp32, and what that leaves
  constexpr float kLo = static_cast<float>(1.4629180792671596e-9 - static_cast<double>(kHi));
  const float n = static_cast<float>(rest);
  const float x = n * kHi;
  const float dx = fmaf(n, kHi, -x) + fmaf(n, kLo, static_cast<float>(rest - static_cast<int32_t>(n)) * kHi);
  const float y = x * x;
  float sp = fmaf(y, 1.f / 362880.f, -1.f / 5040.f);
  sp = fmaf(y, sp, 1.f / 120.f);
  sp = fmaf(y, sp, -1.f / 6.f);
  float cp = fmaf(y, -1.f / 3628800.f, 1.f / 40320.f);
  cp = fmaf(y, cp, -1.f / 720.f);
  cp = fmaf(y, cp, 1.f / 24.f);
  cp = fmaf(y, cp, -0.5f);
  const float f = r.factor, fx = f * x;
  const float cr = fmaf(f, fmaf(y, cp, -x * dx), f);
  const float sr = fx + fmaf(f, fmaf(x * y, sp, dx), fmaf(f, x, -fx));
  const float sw = quarter & 1 ? cr : sr, cw = quarter & 1 ? sr : cr;
  c = (quarter + 1) & 2 ? -cw : cw;
  s = ((quarter & 2) != 0) != (r.sign < 0) ? -sw : sw;
}

// The positions of a token, one for each axis (axes that there are not: 0).
template <bool AXES>
struct RopePos;

template <>
struct RopePos<false> {
  int p;
  __device__ __forceinline__ int of(uint32_t) const { return p; }
};

template <>
struct RopePos<true> {
  int p[kMaxAxes];
  // The position on axis a & 3: two selections by its bits (an index into registers would go through memory).
  __device__ __forceinline__ int of(uint32_t a) const {
    const int lo = a & 1u ? p[1] : p[0], hi = a & 1u ? p[3] : p[2];
    return a & 2u ? hi : lo;
  }
};

template <bool AXES>
__device__ __forceinline__ RopePos<AXES> rope_pos(const RopeArgs& r, int bi, int si, int plain) {
  RopePos<AXES> x;
  if constexpr (AXES) {
    const int32_t* at = r.positions + bi * r.positions_stride + si;
#pragma unroll
    for (int a = 0; a < kMaxAxes; ++a) x.p[a] = a < r.axes ? __ldg(at + a * r.axis_stride) : 0;
  } else {
    x.p = r.positions ? r.positions[bi * r.positions_stride + si] : plain;
  }
  return x;
}

// Axes of the pairs from `pair` on, two bits each, the first in the lowest; 16 - pair % 16 of them.
template <bool AXES>
__device__ __forceinline__ uint32_t axes_from(const RopeArgs& r, int pair) {
  return AXES ? r.axis_of[pair >> 4] >> (2 * (pair & 15)) : 0u;
}

template <int DT>
__device__ __forceinline__ float2 unpack16(uint32_t w) {
  if (DT == kBF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

template <int DT>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  if (DT == kBF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int DT>
__device__ __forceinline__ float load16(const void* p, int64_t i) {
  const uint16_t w = static_cast<const uint16_t*>(p)[i];
  if (DT == kBF16) return __uint_as_float(static_cast<uint32_t>(w) << 16);
  return __half2float(*reinterpret_cast<const __half*>(&w));
}

template <int DT>
__device__ __forceinline__ void store16(void* p, int64_t i, float x) {
  static_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(pack16<DT>(x, 0.f) & 0xFFFFu);
}

// Thread idx of a launch over (group of heads, token of b x s, item), the item fastest.  Where the
// count fits (all but the largest calls) the divisions are of 32 bits, a quarter of the work.
struct Spot {
  int m, grp, bi, si;
};

__device__ __forceinline__ Spot find_spot(int64_t idx, int items, int b, int s, bool small) {
  Spot x;
  if (small) {
    const uint32_t i = static_cast<uint32_t>(idx), r = i / items, tokens = static_cast<uint32_t>(b) * s, tok = r % tokens;
    x.m = i - r * items;
    x.grp = r / tokens;
    x.bi = tok / s;
    x.si = tok - x.bi * s;
  } else {
    const int64_t r = idx / items, tokens = static_cast<int64_t>(b) * s, tok = r % tokens;
    x.m = static_cast<int>(idx - r * items);
    x.grp = static_cast<int>(r / tokens);
    x.bi = static_cast<int>(tok / s);
    x.si = static_cast<int>(tok - static_cast<int64_t>(x.bi) * s);
  }
  return x;
}

// A work item of 16 elements of a head, as two runs of 8: inside the rotated part of each half of it (the halves of 8 pairs, or 4
// adjacent pairs of each), so that neighbouring lanes read neighbouring 16 bytes; behind it 16 neighbours.  rot and d are
// multiples of 16.
struct RopeItem {
  int lo, hi;      // first element of each run
  bool turned;
};

__device__ __forceinline__ RopeItem rope_item(const RopeArgs& r, int m) {
  RopeItem it;
  it.turned = m * 16 < r.rot;
  it.lo = it.turned ? m * 8 : m * 16;
  it.hi = it.turned ? r.rot / 2 + m * 8 : m * 16 + 8;
  return it;
}

// Rotates 16 values of an item (x[0..8) at lo, x[8..16) at hi) by its 8 angles, two at a time.
__device__ __forceinline__ void rope_turn(bool interleaved, float (&x)[16], const float (&c)[8], const float (&s)[8]) {
  const int step = interleaved ? 2 : 1, b0 = interleaved ? 1 : 8;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    float &a0 = x[i * step], &a1 = x[(i + 1) * step], &b0r = x[i * step + b0], &b1r = x[(i + 1) * step + b0];
    const float2 a = make_float2(a0, a1), b = make_float2(b0r, b1r);
    const float2 cc = make_float2(c[i], c[i + 1]), ss = make_float2(s[i], s[i + 1]);
    const float2 y = ptx::fma2(b, make_float2(-ss.x, -ss.y), ptx::mul2(a, cc)), z = ptx::fma2(a, ss, ptx::mul2(b, cc));
    a0 = y.x;
    a1 = y.y;
    b0r = z.x;
    b1r = z.y;
  }
}

}  // namespace sdpa
