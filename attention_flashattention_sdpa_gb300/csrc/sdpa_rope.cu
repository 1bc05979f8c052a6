// sdpa_rope.cu — rotary positions of Q and K: every pair (a, b) of the rotated part of a head
// becomes factor * (a cos t - b sin t, a sin t + b cos t), t = position * frequency (the
// backward pass turns the other way).
//
// Bound: memory, 4 bytes an element.  A thread owns 16 elements of a token's head (8 pairs:
// two 16-byte loads and stores) and walks 8 heads of that token, so that the 8 angles are computed
// once for all of them.  Measured at 2 x 8192 tokens, 16 + 16 heads of 128: 43.6 us, 6.15 TB/s, 91% of
// a copy's 6.77; 4 or 2 heads a thread 46-55 us, the first loads ahead of the angles 46-52.
#include <type_traits>

#include "sdpa_rope.cuh"

namespace sdpa {
namespace {

constexpr int kThreads = 128;
constexpr int kUnroll = 4;     // heads whose loads are in flight together

// rot and d multiples of 2 W.  One thread: item m of token (bi, si), heads [h0, h0 + per).  W = 8, or 4 where rot or d is a
// multiple of 8 alone (8 bytes an access; 2 x 8192 tokens of 16 + 16 heads of 72: 28 us, a pair a thread as below 73).
// AXES: several positions a token; a thread's pairs are neighbours, so that their axes come as 2 W bits of the
// parameters (two runs of W where pairs are interleaved).  16384 tokens, 32 + 8 heads of 128, 3 axes: 53.2 us, 6.3 TB/s.
template <int W, int DT, bool INTER, bool AXES>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p, int per, int groups, bool small) {
  using Run = std::conditional_t<W == 8, uint4, uint2>;      // W elements
  const int items = p.d / (2 * W);
  const Spot at = find_spot(static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x, items, p.b, p.s, small);
  const int m = at.m, grp = at.grp, bi = at.bi, si = at.si;
  if (grp >= groups) return;
  // W elements of each half of the rotated part, or of what lies behind it, so that neighbouring
  // lanes read and write neighbouring bytes (16 neighbouring elements of interleaved pairs: 31.5 us
  // against 31.1 for the backward pass of 4999 tokens, 64 + 8 heads, half of each rotated).
  const bool turned = m * 2 * W < p.r.rot;
  const int start = turned ? 0 : p.r.rot, m8 = m * W - start / 2, width = turned ? p.r.rot : p.d - p.r.rot;
  const RopeItem it{start + m8, start + width / 2 + m8, turned};
  const int h1 = min(p.h_all, (grp + 1) * per);
  auto row_of = [&](int h, bool out) {
    const int t = h >= p.h_q;
    const int64_t(&st)[3] = out ? p.out_st[t] : p.in_st[t];
    const int64_t at = bi * st[0] + (h - (t ? p.h_q : 0)) * st[1] + si * st[2];
    return static_cast<uint16_t*>(out ? p.out[t] : const_cast<void*>(p.in[t])) + at;
  };
  Run u[kUnroll][2];
  auto load = [&](int h0) {
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      if (h0 + j >= h1) continue;
      const uint16_t* row = row_of(h0 + j, false);
      u[j][0] = *reinterpret_cast<const Run*>(row + it.lo);
      u[j][1] = *reinterpret_cast<const Run*>(row + it.hi);
    }
  };
  float c[W], s[W];
  if (it.turned) {
    const RopePos<AXES> pos = rope_pos<AXES>(p.r, bi, si, si);
    uint32_t axes = axes_from<AXES>(p.r, INTER ? m * (W / 2) : m * W);
    if (INTER) axes = (axes & ((1u << W) - 1)) | axes_from<AXES>(p.r, p.r.rot / 4 + m * (W / 2)) << W;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const int pair = !INTER ? m * W + i : i < W / 2 ? m * (W / 2) + i : p.r.rot / 4 + m * (W / 2) + i - W / 2;
      rope_angle(p.r, __ldg(p.r.table + pair), pos.of(axes >> (2 * i)), c[i], s[i]);
    }
  }
  for (int h0 = grp * per; h0 < h1; h0 += kUnroll) {
    load(h0);
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const int h = h0 + j;
      if (h >= h1 || (!it.turned && p.in_place[h >= p.h_q])) continue;
      uint32_t* w = reinterpret_cast<uint32_t*>(u[j]);
      if (it.turned) {
        float x[2 * W];
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const float2 f = unpack16<DT>(w[i]);
          x[2 * i] = f.x;
          x[2 * i + 1] = f.y;
        }
        if constexpr (W == 8) {
          rope_turn(INTER, x, c, s);
        } else {
#pragma unroll
          for (int i = 0; i < W; ++i) {
            float &first = x[INTER ? 2 * i : i], &second = x[INTER ? 2 * i + 1 : i + W];
            const float a = first, b = second;
            first = a * c[i] - b * s[i];
            second = a * s[i] + b * c[i];
          }
        }
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = pack16<DT>(x[2 * i], x[2 * i + 1]);
      }
      uint16_t* row = row_of(h, true);
      *reinterpret_cast<Run*>(row + it.lo) = u[j][0];
      *reinterpret_cast<Run*>(row + it.hi) = u[j][1];
    }
  }
}

// Any even rot and any d: one thread takes one pair (or two elements behind the rotated part).
template <int DT, bool INTER, bool AXES>
__global__ void __launch_bounds__(kThreads) rope_any_kernel(const __grid_constant__ RopeParams p, int per, int groups, bool small) {
  const int items = p.d / 2, half = p.r.rot / 2;
  const Spot at = find_spot(static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x, items, p.b, p.s, small);
  const int m = at.m, grp = at.grp, bi = at.bi, si = at.si;
  if (grp >= groups) return;
  const bool turned = m < half;
  const int ia = turned && !INTER ? m : 2 * m, ib = turned && !INTER ? m + half : 2 * m + 1;
  float c = 1.f, s = 0.f;
  if (turned) {
    rope_angle(p.r, __ldg(p.r.table + m), rope_pos<AXES>(p.r, bi, si, si).of(axes_from<AXES>(p.r, m)), c, s);
  }
  const int h1 = min(p.h_all, (grp + 1) * per);
  for (int h = grp * per; h < h1; ++h) {
    const int t = h >= p.h_q;
    if (!turned && p.in_place[t]) continue;
    const int hh = h - (t ? p.h_q : 0);
    const uint16_t* in = static_cast<const uint16_t*>(p.in[t]) + bi * p.in_st[t][0] + hh * p.in_st[t][1] + si * p.in_st[t][2];
    uint16_t* out = static_cast<uint16_t*>(p.out[t]) + bi * p.out_st[t][0] + hh * p.out_st[t][1] + si * p.out_st[t][2];
    if (turned) {
      const float a = load16<DT>(in, ia), b = load16<DT>(in, ib);
      store16<DT>(out, ia, a * c - b * s);
      store16<DT>(out, ib, a * s + b * c);
    } else {
      out[ia] = in[ia];
      out[ib] = in[ib];
    }
  }
}

template <int DT, bool INTER, bool AXES>
cudaError_t launch_t(const RopeParams& p, int num_sms, cudaStream_t st) {
  const int all = p.d | p.r.rot, run = all % 16 == 0 ? 16 : all % 8 == 0 ? 8 : 2;     // elements of an item
  const int64_t tokens = static_cast<int64_t>(p.b) * p.s, items = p.d / run;
  // Heads a thread walks: as many as leave the GPU full (1024 threads an SM).
  int per = 2 * kUnroll;
  while (per > 1 && tokens * items * ((p.h_all + per - 1) / per) < static_cast<int64_t>(num_sms) * 1024) per /= 2;
  const int groups = (p.h_all + per - 1) / per;
  const int64_t blocks = (tokens * items * groups + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const bool small = blocks * kThreads < (int64_t(1) << 31);
  if (run == 16)
    rope_kernel<8, DT, INTER, AXES><<<static_cast<unsigned>(blocks), kThreads, 0, st>>>(p, per, groups, small);
  else if (run == 8)
    rope_kernel<4, DT, INTER, AXES><<<static_cast<unsigned>(blocks), kThreads, 0, st>>>(p, per, groups, small);
  else
    rope_any_kernel<DT, INTER, AXES><<<static_cast<unsigned>(blocks), kThreads, 0, st>>>(p, per, groups, small);
  return cudaGetLastError();
}

template <int DT, bool INTER>
cudaError_t launch_a(const RopeParams& p, int num_sms, cudaStream_t st) {
  return p.r.axes ? launch_t<DT, INTER, true>(p, num_sms, st) : launch_t<DT, INTER, false>(p, num_sms, st);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int dtype, int num_sms, cudaStream_t st) {
  if (dtype == kBF16) return p.r.interleaved ? launch_a<kBF16, true>(p, num_sms, st) : launch_a<kBF16, false>(p, num_sms, st);
  return p.r.interleaved ? launch_a<kF16, true>(p, num_sms, st) : launch_a<kF16, false>(p, num_sms, st);
}

}  // namespace sdpa
