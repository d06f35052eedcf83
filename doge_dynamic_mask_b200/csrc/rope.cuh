// Rotary angles and head-row helpers shared by the kernels that rotate query and key rows.
//
// Channel i < d/2 of a head row pairs with channel i + d/2 and turns by
// pos * theta^(-2i/d).  The angle is formed in double precision as turns (the
// angle over 2 pi; a position of 10^5 times a frequency near 1 would lose about
// 2^-7 rad in float32, the size of a bf16 rounding), reduced to its fractional
// part, and its cosine and sine are taken in float32.
#pragma once

#include <cmath>

#include "common.cuh"

namespace dma {

// theta^(-2i/d) / (2 pi) for i < d/2: each angle in turns is pos times one of
// these, formed once per call in double precision by the launcher
struct RopeTurns {
  double t[64];
};

// (the last table is kept per host thread: its 64 exponentials cost as much as
// a third of a launch)
inline const RopeTurns& make_rope_turns(float theta, int d) {
  static thread_local RopeTurns turns{};
  static thread_local float last_theta = 0.0f;
  static thread_local int last_d = 0;
  if (theta != last_theta || d != last_d) {
    const double log_theta = log(static_cast<double>(theta));
    for (int i = 0; i < d / 2; ++i) turns.t[i] = exp(-2.0 * i / d * log_theta) * 0.15915494309189535;   // / (2 pi)
    last_theta = theta;
    last_d = d;
  }
  return turns;
}

// cosine and sine of 2 pi * pos * turn; the reduced turn r in [-1/2, 1/2] is
// exact in float32 to 2^-25
__device__ __forceinline__ void rope_cos_sin(double pos, double turn, float& cs, float& sn) {
  const double u = pos * turn;
  const float r = static_cast<float>(u - rint(u));
  sincospif(2.0f * r, &sn, &cs);
}

__device__ __forceinline__ unsigned long long mul_f32x2(unsigned long long a, unsigned long long b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// two bf16 channels (one 32-bit word, low channel first) as packed float32
__device__ __forceinline__ unsigned long long widen_bf16x2(uint32_t w) {
  return f32x2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t pack_f32x2_bf16(unsigned long long v) {
  float a, b;
  f32x2_split(v, a, b);
  return pack_bf16x2(a, b);
}

// Sixteen channels of one head row: a lane's low chunk (channels 8l .. 8l+7)
// and high chunk (d/2 + 8l ..), the rotation's partners, as packed float32.
// d/16 adjacent lanes hold a row.
struct RowChunk {
  unsigned long long lo[4], hi[4];
};

struct RawChunk {
  uint4 lo, hi;
};

__device__ __forceinline__ RowChunk widen_row(const RawChunk& r) {
  RowChunk x;
  x.lo[0] = widen_bf16x2(r.lo.x);
  x.lo[1] = widen_bf16x2(r.lo.y);
  x.lo[2] = widen_bf16x2(r.lo.z);
  x.lo[3] = widen_bf16x2(r.lo.w);
  x.hi[0] = widen_bf16x2(r.hi.x);
  x.hi[1] = widen_bf16x2(r.hi.y);
  x.hi[2] = widen_bf16x2(r.hi.z);
  x.hi[3] = widen_bf16x2(r.hi.w);
  return x;
}

__device__ __forceinline__ RawChunk round_row(const RowChunk& x) {
  RawChunk r;
  r.lo = make_uint4(pack_f32x2_bf16(x.lo[0]), pack_f32x2_bf16(x.lo[1]), pack_f32x2_bf16(x.lo[2]),
                    pack_f32x2_bf16(x.lo[3]));
  r.hi = make_uint4(pack_f32x2_bf16(x.hi[0]), pack_f32x2_bf16(x.hi[1]), pack_f32x2_bf16(x.hi[2]),
                    pack_f32x2_bf16(x.hi[3]));
  return r;
}

__device__ __forceinline__ void store_row(uint16_t* row, int half, const RawChunk& r) {
  *reinterpret_cast<uint4*>(row) = r.lo;
  *reinterpret_cast<uint4*>(row + half) = r.hi;
}

// Sum over the LPR adjacent lanes that hold a row (every lane of the warp calls it).
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o >= 1; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// sum over a lane's sixteen channels of a * b
__device__ __forceinline__ float chunk_dot(const RowChunk& a, const RowChunk& b) {
  unsigned long long acc = mul_f32x2(a.lo[0], b.lo[0]);
#pragma unroll
  for (int e = 1; e < 4; ++e) acc = fma_f32x2(a.lo[e], b.lo[e], acc);
#pragma unroll
  for (int e = 0; e < 4; ++e) acc = fma_f32x2(a.hi[e], b.hi[e], acc);
  float x, y;
  f32x2_split(acc, x, y);
  return x + y;
}

// The eight angles of a lane's channel pairs at a position.
struct RowAngles {
  unsigned long long cs[4], sn[4];
};

// How a grid's warps share the head rows of q and of k.  A warp step takes 128 /
// d tokens and four consecutive heads of each, so a token's step is 4 d
// contiguous channels; a token has ceil(Hq / 4) steps in q, then ceil(Hkv / 4) in
// k.  An item is the steps of one group of tokens, or a part of them when there
// are fewer groups than warps.  Items are dealt to the warps in turn: what the
// grid touches at any time is one window of memory (a contiguous share per warp
// instead cost 12% at 32768 tokens of 16 + 8 heads of 128).
struct RowShare {
  int T, heads[2];
  int q_steps, steps;   // of a token: in q, in both
  int parts, items;
};

inline RowShare share_rows(int T, int Hq, int Hkv, int d, long long warps) {
  RowShare s;
  s.T = T;
  s.heads[0] = Hq;
  s.heads[1] = Hkv;
  s.q_steps = (Hq + 3) / 4;
  s.steps = s.q_steps + (Hkv + 3) / 4;
  const long long groups = (static_cast<long long>(T) * d + 127) / 128;
  const long long parts = warps / groups;
  s.parts = static_cast<int>(parts < 1 ? 1 : parts > s.steps ? s.steps : parts);
  s.items = static_cast<int>(groups * s.parts);   // 32 bits hold it: several parts only while groups are few
  return s;
}

// An item as a lane sees it: its token, its steps, and its row in a step (head
// 4 (step within the tensor) + row of the token's tensor).
template <int D>
struct RowItem {
  static constexpr int kTokens = 128 / D;          // tokens per warp
  static constexpr int kLanes = 32 / kTokens;      // lanes per token
  static constexpr int LPR = D / 16;               // lanes per row
  int token, s0, s1;
  bool there;                                      // the token exists

  static __device__ __forceinline__ int row() { return (threadIdx.x & 31) / LPR % 4; }
  __device__ __forceinline__ void enter(const RowShare& s, int item) {
    int group = item;
    s0 = 0;
    s1 = s.steps;
    if (s.parts > 1) {
      group = item / s.parts;
      const int part = item - group * s.parts;
      s0 = part * s.steps / s.parts;
      s1 = (part + 1) * s.steps / s.parts;
    }
    token = group * kTokens + static_cast<int>(threadIdx.x & 31) / kLanes;
    there = item < s.items && token < s.T;
  }
};

// The eight angles of a lane's channel pairs at its token's position: each lane
// of a token forms two of the d/2 and the lanes exchange them.
template <int D>
__device__ __forceinline__ RowAngles token_angles(double pos, const double* turns) {
  constexpr int UL = RowItem<D>::kLanes, LPR = RowItem<D>::LPR;
  const int lane = threadIdx.x & 31, l = lane % LPR;
  float c[2], s[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) rope_cos_sin(pos, turns[2 * (lane % UL) + i], c[i], s[i]);
  RowAngles a;
#pragma unroll
  for (int e = 0; e < 4; ++e) {   // angles 8 l + 2 e and the next sit in lane 4 l + e
    a.cs[e] = f32x2(__shfl_sync(0xFFFFFFFFu, c[0], 4 * l + e, UL), __shfl_sync(0xFFFFFFFFu, c[1], 4 * l + e, UL));
    a.sn[e] = f32x2(__shfl_sync(0xFFFFFFFFu, s[0], 4 * l + e, UL), __shfl_sync(0xFFFFFFFFu, s[1], 4 * l + e, UL));
  }
  return a;
}

// The rotation of a weighted row, (lo, hi) -> (w_lo lo cos - w_hi hi sin, w_hi hi
// cos + w_lo lo sin), as the four products that a token's rows share.
struct RowTurn {
  unsigned long long lc[4], hs[4], hc[4], ls[4];
};

__device__ __forceinline__ RowTurn row_turn(const RowAngles& a, const RowChunk& w) {
  RowTurn t;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    t.lc[e] = mul_f32x2(w.lo[e], a.cs[e]);
    t.hs[e] = mul_f32x2(w.hi[e], a.sn[e]);
    t.hc[e] = mul_f32x2(w.hi[e], a.cs[e]);
    t.ls[e] = mul_f32x2(w.lo[e], a.sn[e]);
  }
  return t;
}

__device__ __forceinline__ RowChunk turn_row(const RowChunk& x, const RowTurn& t) {
  RowChunk o;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    o.lo[e] = sub_f32x2(mul_f32x2(x.lo[e], t.lc[e]), mul_f32x2(x.hi[e], t.hs[e]));
    o.hi[e] = fma_f32x2(x.lo[e], t.ls[e], mul_f32x2(x.hi[e], t.hc[e]));
  }
  return o;
}

// the rotation undone: (lo, hi) -> (lo cos + hi sin, hi cos - lo sin)
__device__ __forceinline__ RowChunk rotate_row_back(const RowChunk& y, const RowAngles& a) {
  RowChunk o;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    o.lo[e] = fma_f32x2(y.hi[e], a.sn[e], mul_f32x2(y.lo[e], a.cs[e]));
    o.hi[e] = sub_f32x2(mul_f32x2(y.hi[e], a.cs[e]), mul_f32x2(y.lo[e], a.sn[e]));
  }
  return o;
}

// sixteen float32 weights of a lane's chunks (w points at channel 8l)
__device__ __forceinline__ RowChunk load_weights(const float* w, int half) {
  const float4 a = *reinterpret_cast<const float4*>(w), b = *reinterpret_cast<const float4*>(w + 4);
  const float4 c = *reinterpret_cast<const float4*>(w + half), e = *reinterpret_cast<const float4*>(w + half + 4);
  RowChunk r;
  r.lo[0] = f32x2(a.x, a.y);
  r.lo[1] = f32x2(a.z, a.w);
  r.lo[2] = f32x2(b.x, b.y);
  r.lo[3] = f32x2(b.z, b.w);
  r.hi[0] = f32x2(c.x, c.y);
  r.hi[1] = f32x2(c.z, c.w);
  r.hi[2] = f32x2(e.x, e.y);
  r.hi[3] = f32x2(e.z, e.w);
  return r;
}

}  // namespace dma
