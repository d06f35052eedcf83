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
// A warp step takes four consecutive heads of a token (of two tokens at d = 64):
// a contiguous piece of x, of g and of dx.  The eight angles a lane needs are
// formed once per token.  The rows travel by cp.async through a ring in shared
// memory in which each lane reads back only what it copied itself, so the steps
// in flight need no registers or barriers.  A lane always holds the same
// channels, so its share of dw accumulates in float32 registers over everything
// the warp does; the shares are added in a fixed order (lane groups, warps,
// blocks), so the result does not depend on timing; the last block to finish adds
// the blocks' shares, so there is no second launch.
//
// Measured.  32768 tokens, 16 + 8 heads of 128: 115 us for 604 MB, 5.2 TB/s (94 us
// at the copy rate).  16384 tokens, 8 + 4 heads of 64: 22 us for 75 MB, of which some
// 6 us are the start and the join of the weight gradients (74 tokens take 5.6 us).  With
// one to three heads of q and one or two of k, 21852 tokens of d = 128 take 31 us (5 to 10 us
// at the copy rate): a warp step is four heads of one token, absent or not.
// Half of the issue slots are used, by four warps a scheduler, which 128 registers a
// thread allow; ten warps a block in 96 registers spilled: 165 us and 32 us.
#include <algorithm>

#include "rope.cuh"

namespace dma {
namespace {

constexpr int kPbThreads = 256;
constexpr int kPbWarps = kPbThreads / 32;
constexpr int kPbMinBlocks = 2;
constexpr int kPbStages = 4;                                     // ring steps per warp
constexpr int kPbSmemBytes = kPbWarps * kPbStages * 4 * 32 * 16;   // a step: four 16-byte chunks per lane

struct PbArgs {
  const uint16_t *q, *k, *gq, *gk;
  long long q_stride, k_stride, dq_stride, dk_stride;   // elements between tokens
  const float *q_w, *k_w;
  const int32_t* positions;
  uint16_t *dq, *dk;
  float *dq_w, *dk_w;
  float* part;         // [blocks][2][d]: the blocks' shares
  uint32_t* ticket;    // finished blocks, zero between calls
  float eps;
  int L;
  RowShare share;
};

// EPS: eps > 0
template <int D, bool EPS>
__global__ void __launch_bounds__(kPbThreads, kPbMinBlocks)
    prologue_bwd_kernel(const __grid_constant__ PbArgs a, const __grid_constant__ RopeTurns turns) {
  constexpr int LPR = D / 16;          // lanes per row
  constexpr int H = D / 2;
  __shared__ __align__(16) float s_w[2][D];
  __shared__ __align__(16) double s_turn[H];
  __shared__ __align__(16) float s_dw[kPbWarps][2][D];
  pdl_wait();
  pdl_trigger();
  for (int c = threadIdx.x; c < D; c += kPbThreads) {
    s_w[0][c] = a.q_w[c];
    s_w[1][c] = a.k_w[c];
    if (c < H) s_turn[c] = turns.t[c];
  }
  __syncthreads();

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c0 = 8 * (lane % LPR);
  const int stride = static_cast<int>(gridDim.x) * kPbWarps;
  const int it0 = warp * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x);
  const int row0 = RowItem<D>::row();

  // ---- the ring: rows of x and g on their way
  extern __shared__ __align__(16) uint4 ring_all[];
  uint4* ring = ring_all + warp * kPbStages * 128 + lane;   // [stage][x lo, x hi, g lo, g hi][lane]
  const uint32_t ring_u = smem_u32(ring);
  int f_it = it0, f_s = 0, f_h = 0, f_n = 0;
  RowItem<D> f{};
  const uint16_t *f_x = a.q, *f_g = a.gq;
  auto f_tensor = [&](int n, int s) {   // step s is in tensor n
    f_n = n;
    f_h = 4 * s + row0;
    const long long t = f.token;
    f_x = (n ? a.k + t * a.k_stride : a.q + t * a.q_stride) + f_h * D + c0;
    f_g = (n ? a.gk : a.gq) + (t * a.share.heads[n] + f_h) * D + c0;
  };
  auto f_enter = [&]() {
    f.enter(a.share, f_it);
    f_s = f.s0;
    const int n = f_s >= a.share.q_steps;
    f_tensor(n, n ? f_s - a.share.q_steps : f_s);
  };
  f_enter();
  auto issue = [&](int slot) {
    if (f_it < a.share.items) {
      const bool there = f.there && f_h < a.share.heads[f_n];
      const uint16_t *x = there ? f_x : a.q, *g = there ? f_g : a.gq;
      const uint32_t dst = ring_u + slot * 2048;
      cp_async16_zfill(dst, x, there);
      cp_async16_zfill(dst + 512, x + H, there);
      cp_async16_zfill(dst + 1024, g, there);
      cp_async16_zfill(dst + 1536, g + H, there);
      f_x += 4 * D;
      f_g += 4 * D;
      f_h += 4;
      if (++f_s == f.s1) {
        f_it += stride;
        f_enter();
      } else if (f_s == a.share.q_steps) {
        f_tensor(1, 0);
      }
    }
    cp_commit();
  };
#pragma unroll
  for (int s = 0; s < kPbStages - 1; ++s) issue(s);

  RowChunk dw[2];
#pragma unroll
  for (int e = 0; e < 4; ++e) dw[0].lo[e] = dw[0].hi[e] = dw[1].lo[e] = dw[1].hi[e] = 0ull;
  int slot = 0;
  RowItem<D> w;
  for (int it = it0; it < a.share.items; it += stride) {
    w.enter(a.share, it);
    const int b = w.there ? w.token / a.L : 0;
    const double pos =
        w.there ? static_cast<double>(static_cast<long long>(a.positions[b]) + (w.token - b * a.L)) : 0.0;
    const RowAngles ang = token_angles<D>(pos, s_turn);
    // one row: its gradient to dx, its share of dw to acc
    auto row = [&](bool act, uint16_t* dx, const float* w_s, RowChunk& acc) {
      cp_wait<kPbStages - 2>();
      const RawChunk xc{ring[slot * 128], ring[slot * 128 + 32]}, gc{ring[slot * 128 + 64], ring[slot * 128 + 96]};
      issue(slot == 0 ? kPbStages - 1 : slot - 1);   // the step read last time
      slot = slot + 1 == kPbStages ? 0 : slot + 1;
      RowChunk xh = widen_row(xc);
      // a row that is not there is zeros: its r is finite and it adds nothing, unless eps is 0
      // (kernels of their own: asking takes 1.4 us of 22.5)
      float r = rsqrtf(row_sum<LPR>(chunk_dot(xh, xh)) * (1.0f / D) + a.eps);
      if (!EPS && !act) r = 0.0f;
      const unsigned long long r2 = f32x2(r, r);
      RowChunk u = rotate_row_back(widen_row(gc), ang);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        xh.lo[e] = mul_f32x2(xh.lo[e], r2);
        xh.hi[e] = mul_f32x2(xh.hi[e], r2);
        acc.lo[e] = fma_f32x2(u.lo[e], xh.lo[e], acc.lo[e]);
        acc.hi[e] = fma_f32x2(u.hi[e], xh.hi[e], acc.hi[e]);
      }
      const RowChunk wt = load_weights(w_s, H);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        u.lo[e] = mul_f32x2(u.lo[e], wt.lo[e]);
        u.hi[e] = mul_f32x2(u.hi[e], wt.hi[e]);
      }
      const float m = -row_sum<LPR>(chunk_dot(u, xh)) * (1.0f / D);
      const unsigned long long m2 = f32x2(m, m);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        u.lo[e] = mul_f32x2(fma_f32x2(xh.lo[e], m2, u.lo[e]), r2);
        u.hi[e] = mul_f32x2(fma_f32x2(xh.hi[e], m2, u.hi[e]), r2);
      }
      if (act) store_row(dx, H, round_row(u));
    };
    const long long t = w.token;
    const int q1 = min(w.s1, a.share.q_steps), k0 = max(w.s0, a.share.q_steps);
    int h = 4 * w.s0 + row0;
    uint16_t* dx = a.dq + t * a.dq_stride + h * D + c0;
    for (int s = w.s0; s < q1; ++s, h += 4, dx += 4 * D)
      row(w.there && h < a.share.heads[0], dx, s_w[0] + c0, dw[0]);
    h = 4 * (k0 - a.share.q_steps) + row0;
    dx = a.dk + t * a.dk_stride + h * D + c0;
    for (int s = k0; s < w.s1; ++s, h += 4, dx += 4 * D)
      row(w.there && h < a.share.heads[1], dx, s_w[1] + c0, dw[1]);
  }
  cp_wait<0>();

  // this warp's share of the weight gradients: the sum over its lane groups
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
        if (lane < LPR) s_dw[warp][n][(i >= 2 ? H : 0) + c0 + 2 * e + (i & 1)] = v[i];
      }
    }

  // the block's share: its warps in order
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * D; c += kPbThreads) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kPbWarps; ++w) s += s_dw[w][c / D][c % D];
    a.part[static_cast<size_t>(blockIdx.x) * 2 * D + c] = s;
  }
  // the last block to finish adds the blocks' shares: four columns and every
  // kRows-th block per thread, then the kRows sums
  __shared__ bool s_last;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    s_last = atomicAdd(a.ticket, 1u) == gridDim.x - 1u;
    if (s_last) *a.ticket = 0u;
    __threadfence();
  }
  __syncthreads();
  if (!s_last) return;
  constexpr int kCols = 2 * D / 4, kRows = kPbThreads / kCols;
  float4* sums = reinterpret_cast<float4*>(&s_dw[0][0][0]);   // [kRows][kCols]
  const float4* part = reinterpret_cast<const float4*>(a.part);
  const int col = threadIdx.x % kCols;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 16
  for (int i = threadIdx.x / kCols; i < static_cast<int>(gridDim.x); i += kRows) {
    const float4 x = __ldcg(part + static_cast<size_t>(i) * kCols + col);
    v.x += x.x;
    v.y += x.y;
    v.z += x.z;
    v.w += x.w;
  }
  sums[threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.x >= kCols) return;
#pragma unroll
  for (int i = 1; i < kRows; ++i) {
    const float4 x = sums[i * kCols + col];
    v.x += x.x;
    v.y += x.y;
    v.z += x.z;
    v.w += x.w;
  }
  *reinterpret_cast<float4*>((col < kCols / 2 ? a.dq_w : a.dk_w) + 4 * (col % (kCols / 2))) = v;
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
  a.dq_w = p.dq_norm_w;
  a.dk_w = p.dk_norm_w;
  a.ticket = p.ticket;
  a.part = p.part;
  a.eps = p.eps;
  a.L = p.L;
  const int slots = std::min(kPbMinBlocks * nsm, kPbMaxBlocks);
  a.share = share_rows(p.B * p.L, p.Hq, p.Hkv, p.d, static_cast<long long>(slots) * kPbWarps);
  // a warp per item: few blocks, and few shares to add, when there are few items (74
  // tokens: 5.7 us, with a block in every slot 7.6 us)
  const int blocks = std::min((a.share.items + kPbWarps - 1) / kPbWarps, slots);
  auto* kernel = p.d == 64 ? (p.eps > 0.0f ? prologue_bwd_kernel<64, true> : prologue_bwd_kernel<64, false>)
                           : (p.eps > 0.0f ? prologue_bwd_kernel<128, true> : prologue_bwd_kernel<128, false>);
  const cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(kernel), kPbSmemBytes);
  if (e != cudaSuccess) return e;
  return launch_after(kernel, dim3(blocks), dim3(kPbThreads), kPbSmemBytes, s, a, turns);
}

size_t prologue_backward_scratch_bytes(int d) {
  return static_cast<size_t>(kPbMaxBlocks) * 2 * d * sizeof(float);
}

}  // namespace dma
