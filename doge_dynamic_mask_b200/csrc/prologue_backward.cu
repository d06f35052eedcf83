// Backward of the prologue's q_norm / k_norm and rotary embedding.
//
// Method: page "Transformers 中的 Doge 小语言模型完全指南", section
// "动态掩码注意力（DMA）：从缓存 value states 生成稀疏掩码", forward-chain step 1
// (per-head RMSNorm of Q and K, then the rotary embedding); its gradients, for
// a head row x of d channels with weight w, angles a of the token's position
// and the gradient g of the rotated row:
//
//   r    = (mean_c(x^2) + eps)^(-1/2),  xh = x r
//   dy   = R(-a) g          (the rotation is orthogonal: its transpose undoes it)
//   dw  += dy xh            (summed over every row of q, or of k)
//   u    = dy w
//   dx   = r (u - xh mean_c(u xh))
//
// Design.  Memory-bound: x and g are read once and dx written once, about 4
// flops per byte.  A row's channels sit in d/16 adjacent lanes, each with a
// 16-byte chunk of channels i and the chunk of their partners i + d/2, so the
// rotation needs no exchange and the two row sums are three shuffles or fewer.
// A warp takes 32/(d/16) tokens at once, one per lane group, and walks over
// the heads: the eight angles a lane needs are formed once per token and stay
// in registers for all of its rows.  When there are fewer tokens than warps
// the heads are split over warps too.  A lane always holds the same
// channels, so its share of dw accumulates in float32 registers over
// everything the warp does; the shares are added in a fixed order (lane
// groups, then warps, then, in a second kernel, blocks), so the result does
// not depend on timing.
#include <algorithm>

#include "rope.cuh"

namespace dma {
namespace {

constexpr int kPbThreads = 256;
constexpr int kPbWarps = kPbThreads / 32;
constexpr int kPbMinBlocks = 2;
constexpr int kPbReduceThreads = 256;

struct PbArgs {
  const uint16_t *q, *k, *gq, *gk;
  long long q_stride, k_stride, dq_stride, dk_stride;   // elements between tokens
  const float *q_w, *k_w;
  const int32_t* positions;
  uint16_t *dq, *dk;
  float* part;         // [blocks][2][d]
  float eps;
  int T, L, Hq, Hkv;
  int splits;          // head splits per token group
};

template <int D>
__global__ void __launch_bounds__(kPbThreads, kPbMinBlocks)
    prologue_bwd_kernel(const __grid_constant__ PbArgs a, const __grid_constant__ RopeTurns turns) {
  constexpr int LPR = D / 16;          // lanes per row
  constexpr int GPW = 32 / LPR;        // rows (tokens) per warp step
  constexpr int H = D / 2;
  __shared__ __align__(16) float s_w[2][D];
  __shared__ __align__(16) double s_turn[H];
  __shared__ float s_dw[kPbWarps][2][D];
  pdl_wait();
  pdl_trigger();
  for (int c = threadIdx.x; c < D; c += kPbThreads) {
    s_w[0][c] = a.q_w[c];
    s_w[1][c] = a.k_w[c];
    if (c < H) s_turn[c] = turns.t[c];
  }
  __syncthreads();

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int l = lane % LPR, grp = lane / LPR;
  const int c0 = 8 * l;
  const int rows = a.Hq + a.Hkv;
  const int groups = (a.T + GPW - 1) / GPW;
  const long long items = static_cast<long long>(groups) * a.splits;
  RowChunk dw[2];
#pragma unroll
  for (int e = 0; e < 4; ++e) dw[0].lo[e] = dw[0].hi[e] = dw[1].lo[e] = dw[1].hi[e] = 0ull;

  for (long long it = static_cast<long long>(warp) * gridDim.x + blockIdx.x; it < items;
       it += static_cast<long long>(gridDim.x) * kPbWarps) {
    const int tg = static_cast<int>(it / a.splits), part = static_cast<int>(it % a.splits);
    const int h0 = static_cast<int>(static_cast<long long>(part) * rows / a.splits);
    const int h1 = static_cast<int>(static_cast<long long>(part + 1) * rows / a.splits);
    const int token = tg * GPW + grp;
    const bool act = token < a.T;
    const int b = act ? token / a.L : 0;
    const double pos = act ? static_cast<double>(static_cast<long long>(a.positions[b]) + (token - b * a.L)) : 0.0;
    const RowAngles ang = row_angles(pos, s_turn + c0);

    // rows [ha, hb) of one tensor
    auto walk = [&](int ha, int hb, const uint16_t* x, const uint16_t* g, uint16_t* dx, const float* w_s,
                    RowChunk& acc) {
      const RowChunk w = load_weights(w_s + c0, H);
      const RawChunk zero{make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
      RawChunk xr = act ? load_row(x + ha * D, H) : zero, gr = act ? load_row(g + ha * D, H) : zero;
      for (int h = ha; h < hb; ++h) {
        const RawChunk xc = xr, gc = gr;
        if (act && h + 1 < hb) {   // the next row travels while this one is computed
          xr = load_row(x + (h + 1) * D, H);
          gr = load_row(g + (h + 1) * D, H);
        }
        RowChunk xh = widen_row(xc);
        const float r = rsqrtf(row_sum<LPR>(chunk_dot(xh, xh)) * (1.0f / D) + a.eps);
        const unsigned long long r2 = f32x2(r, r);
        const RowChunk dy = rotate_row_back(widen_row(gc), ang);
        RowChunk u;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          xh.lo[e] = mul_f32x2(xh.lo[e], r2);
          xh.hi[e] = mul_f32x2(xh.hi[e], r2);
          acc.lo[e] = fma_f32x2(dy.lo[e], xh.lo[e], acc.lo[e]);
          acc.hi[e] = fma_f32x2(dy.hi[e], xh.hi[e], acc.hi[e]);
          u.lo[e] = mul_f32x2(dy.lo[e], w.lo[e]);
          u.hi[e] = mul_f32x2(dy.hi[e], w.hi[e]);
        }
        const float m = -row_sum<LPR>(chunk_dot(u, xh)) * (1.0f / D);
        const unsigned long long m2 = f32x2(m, m);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          u.lo[e] = mul_f32x2(fma_f32x2(xh.lo[e], m2, u.lo[e]), r2);
          u.hi[e] = mul_f32x2(fma_f32x2(xh.hi[e], m2, u.hi[e]), r2);
        }
        if (act) store_row(dx + h * D, H, round_row(u));
      }
    };
    const long long t = token;
    if (h0 < a.Hq)
      walk(h0, min(h1, a.Hq), a.q + t * a.q_stride + c0, a.gq + t * a.Hq * D + c0, a.dq + t * a.dq_stride + c0,
           s_w[0], dw[0]);
    if (h1 > a.Hq)
      walk(max(h0, a.Hq) - a.Hq, h1 - a.Hq, a.k + t * a.k_stride + c0, a.gk + t * a.Hkv * D + c0,
           a.dk + t * a.dk_stride + c0, s_w[1], dw[1]);
  }

  // this block's share of the weight gradients: lane groups, then warps
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float v[4];
      f32x2_split(dw[n].lo[e], v[0], v[1]);
      f32x2_split(dw[n].hi[e], v[2], v[3]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int o = LPR; o < 32; o <<= 1) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
        if (grp == 0) s_dw[warp][n][(i >= 2 ? H : 0) + c0 + 2 * e + (i & 1)] = v[i];
      }
    }
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * D; c += kPbThreads) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kPbWarps; ++w) s += s_dw[w][c / D][c % D];
    a.part[static_cast<size_t>(blockIdx.x) * 2 * D + c] = s;
  }
}

// Sum of the blocks' shares, 32 channels per block: each warp adds every eighth
// block's row in order, then the warps' sums are added in order.
__global__ void __launch_bounds__(kPbReduceThreads)
    prologue_bwd_reduce_kernel(const float* part, int blocks, int d, float* __restrict__ dq_w,
                               float* __restrict__ dk_w) {
  constexpr int kWarps = kPbReduceThreads / 32;
  __shared__ float s[kWarps][32];
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.0f;
#pragma unroll 8
  for (int b = warp; b < blocks; b += kWarps) v += part[static_cast<size_t>(b) * 2 * d + c];
  s[warp][lane] = v;
  __syncthreads();
  if (warp == 0) {
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) t += s[w][lane];
    if (c < d)
      dq_w[c] = t;
    else
      dk_w[c - d] = t;
  }
}

}  // namespace

cudaError_t launch_prologue_backward(const PrologueBackward& p, cudaStream_t s) {
  const RopeTurns& turns = make_rope_turns(p.theta, p.d);
  const int nsm = sm_count();
  if (nsm <= 0) return cudaErrorInvalidDevice;
  PbArgs a;
  a.q = static_cast<const uint16_t*>(p.q);
  a.k = static_cast<const uint16_t*>(p.k);
  a.gq = static_cast<const uint16_t*>(p.dq_out);
  a.gk = static_cast<const uint16_t*>(p.dk_out);
  a.q_stride = p.q_stride;
  a.k_stride = p.k_stride;
  a.dq_stride = p.dq_stride;
  a.dk_stride = p.dk_stride;
  a.q_w = p.q_norm_w;
  a.k_w = p.k_norm_w;
  a.positions = p.positions;
  a.dq = static_cast<uint16_t*>(p.dq);
  a.dk = static_cast<uint16_t*>(p.dk);
  a.part = p.part;
  a.eps = p.eps;
  a.T = p.B * p.L;
  a.L = p.L;
  a.Hq = p.Hq;
  a.Hkv = p.Hkv;
  // tokens are taken in groups of 4 (d = 128) or 8 (d = 64) per warp; with
  // fewer groups than resident warps the heads of a token are split as well
  const int gpw = 32 / (p.d / 16);
  const long long groups = (static_cast<long long>(a.T) + gpw - 1) / gpw;
  const long long slots = static_cast<long long>(std::min(kPbMinBlocks * nsm, kPbMaxBlocks)) * kPbWarps;
  a.splits = static_cast<int>(std::max(1LL, std::min<long long>(p.Hq + p.Hkv, slots / groups)));
  const long long items = groups * a.splits;
  // few items spread over blocks (and SMs) before they share one
  const int blocks = static_cast<int>(std::min<long long>(items, slots / kPbWarps));
  cudaError_t e = p.d == 64 ? launch_after(prologue_bwd_kernel<64>, dim3(blocks), dim3(kPbThreads), 0, s, a, turns)
                            : launch_after(prologue_bwd_kernel<128>, dim3(blocks), dim3(kPbThreads), 0, s, a, turns);
  if (e != cudaSuccess) return e;
  return launch_after(prologue_bwd_reduce_kernel, dim3(2 * p.d / 32), dim3(kPbReduceThreads), 0, s, p.part, blocks, p.d,
                      p.dq_norm_w, p.dk_norm_w);
}

}  // namespace dma
