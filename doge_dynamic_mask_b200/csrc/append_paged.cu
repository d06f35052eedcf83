// Append to a paged cache: q_norm / k_norm, rotary embedding, K/V pages and dt rows, in one launch.
//
// Method: page "Transformers 中的 Doge 小语言模型完全指南", section
// "动态掩码注意力（DMA）：从缓存 value states 生成稀疏掩码", forward-chain steps 1-3:
// the prologue's per-head RMSNorm and rotation of Q and K, the cache update, and
// dt = exp(A softplus(dt_proj(value_states))), which is one projection per
// token and therefore needs computing only once, when the token enters the
// cache.  For token t of the packed batch, in sequence b (cu[b] <= t <
// cu[b+1]), at position pos = positions[b] + t - cu[b]:
//
//   q_out = R(pos) (w_q q / rms(q)),  K row = R(pos) (w_k k / rms(k)),  V row = v,
//   dt[g] = exp(A[g] softplus(sum_c v[c] W[c, g]))
//
// and the cache row is (page_table[b, pos / page_size], pos % page_size).
//
// Design.  Memory-bound: every projected row is read once and written once
// (about 4 flops per byte), and W is read once per block.  Blocks have one of
// two jobs.
//
// Row blocks: q and k rows.  A row's channels sit in d/16 adjacent lanes (a
// 16-byte chunk and its rotation partner's chunk each), a warp takes 4 or 8
// tokens at once, one per lane group, and walks over the heads with the token's
// angles in registers; with few tokens the heads are split over warps as well.
//
// Value blocks: v rows and dt.  Sixteen tokens are the M side of
// mma.m16n8k16, the kv heads the N side.  A dot product does not care in which
// order its channels are taken, so the A fragments are the 16-byte chunks as
// they come from memory (a quad of lanes covers 64 bytes of a row) and the same
// registers are stored to the page: V passes through without shared memory.
// W is split exactly into three bf16 terms (each the rounding of what the
// previous ones leave), whose products with bf16 values are exact, so the
// float32 accumulators hold the float32 projection; a warp keeps the
// fragments of its 128 channels in registers for all of its tokens.  The
// projection is 2 Hkv flops per byte of V: far below what tcgen05 is for, and a
// 128-row tile would leave a decode step's few tokens on one SM.
#include <algorithm>

#include "rope.cuh"

namespace dma {
namespace {

constexpr int kApCuCap = 1024;       // sequences whose offsets fit the staged copy

struct ApArgs {
  const uint16_t *q, *k, *v;
  long long q_stride, k_stride, v_stride;   // elements between tokens
  const float *q_w, *k_w, *W, *A;
  const int32_t *cu, *positions, *table;
  uint16_t *q_out, *k_out, *k_pages, *v_pages;
  float* dt_pages;
  long long page_stride;                    // elements between pages of k_pages / v_pages
  float eps;
  int T, B, max_pages, num_pages, page_size, Hq;
  int splits;                               // head splits per token group (row blocks)
  int val_blocks;                           // blocks [0, val_blocks) take the values
  uint32_t* err;
};

// Where a token of the packed batch goes.  live: it belongs to a sequence;
// page < 0: its position has no page (reported), nothing is written to the cache.
struct Where {
  long long pos;
  int page, off;
  bool live;
};

__device__ __forceinline__ Where locate(const ApArgs& a, const int32_t* cu, int token) {
  Where w{0, -1, 0, false};
  if (token >= a.T || token < cu[0] || token >= cu[a.B]) return w;
  // cu[lo] <= token < cu[hi] holds throughout
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= token)
      lo = mid;
    else
      hi = mid;
  }
  w.live = true;
  w.pos = static_cast<long long>(a.positions[lo]) + (token - cu[lo]);
  if (w.pos < 0 || w.pos >= static_cast<long long>(a.max_pages) * a.page_size) {
    raise_error(a.err, kDevErrBadPosition);
    return w;
  }
  const int slot = static_cast<int>(w.pos) / a.page_size;
  const int page = a.table[static_cast<size_t>(lo) * a.max_pages + slot];
  if (page < 0 || page >= a.num_pages) {
    raise_error(a.err, kDevErrBadPage);
    return w;
  }
  w.page = page;
  w.off = static_cast<int>(w.pos) - slot * a.page_size;
  return w;
}

__device__ __forceinline__ float softplus_f32(float x) { return fmaxf(x, 0.0f) + log1pf(expf(-fabsf(x))); }

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int D, int HKV>
struct ApCfg {
  static constexpr int C = HKV * D;
  static constexpr int kSlice = C >= 128 ? 128 : 64;        // channels of one warp
  static constexpr int kSlices = C / kSlice;
  static constexpr int kJ = kSlice / 32;                    // 64-byte steps of a slice
  static constexpr int NT = HKV > 8 ? 2 : 1;                // groups of eight heads
  static constexpr int kWarps = kSlices > 8 ? 16 : 8;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kMinBlocks = kWarps > 8 ? 1 : 2;
  static constexpr int kTiles = kWarps / kSlices;           // 16-token tiles of a block at once
  static constexpr int LPR = D / 16;
  static constexpr int GPW = 32 / LPR;
};

template <int D, int HKV>
__device__ __forceinline__ void row_blocks(const ApArgs& a, const int32_t* cu, const float (*s_w)[D],
                                           const double* s_turn) {
  using Cfg = ApCfg<D, HKV>;
  constexpr int H = D / 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int l = lane % Cfg::LPR, grp = lane / Cfg::LPR;
  const int c0 = 8 * l;
  const int rows = a.Hq + HKV;
  const int groups = (a.T + Cfg::GPW - 1) / Cfg::GPW;
  const long long items = static_cast<long long>(groups) * a.splits;
  const int nblk = gridDim.x - a.val_blocks, blk = blockIdx.x - a.val_blocks;
  for (long long it = static_cast<long long>(warp) * nblk + blk; it < items;
       it += static_cast<long long>(nblk) * Cfg::kWarps) {
    const int tg = static_cast<int>(it / a.splits), part = static_cast<int>(it % a.splits);
    const int h0 = static_cast<int>(static_cast<long long>(part) * rows / a.splits);
    const int h1 = static_cast<int>(static_cast<long long>(part + 1) * rows / a.splits);
    const int token = tg * Cfg::GPW + grp;
    const Where w = locate(a, cu, token);
    const RowAngles ang = row_angles(static_cast<double>(w.pos), s_turn + c0);
    const long long t = token;

    auto walk = [&](int ha, int hb, const uint16_t* x, const float* w_s, uint16_t* out0, uint16_t* out1) {
      const RowChunk wt = load_weights(w_s + c0, H);
      RawChunk xr{make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
      if (w.live) xr = load_row(x + ha * D, H);
      for (int h = ha; h < hb; ++h) {
        const RawChunk xc = xr;
        if (w.live && h + 1 < hb) xr = load_row(x + (h + 1) * D, H);
        RowChunk y = widen_row(xc);
        const float r = rsqrtf(row_sum<Cfg::LPR>(chunk_dot(y, y)) * (1.0f / D) + a.eps);
        const unsigned long long r2 = f32x2(r, r);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y.lo[e] = mul_f32x2(mul_f32x2(y.lo[e], wt.lo[e]), r2);
          y.hi[e] = mul_f32x2(mul_f32x2(y.hi[e], wt.hi[e]), r2);
        }
        const RawChunk o = round_row(rotate_row(y, ang));
        if (out0) store_row(out0 + h * D, H, o);
        if (out1) store_row(out1 + h * D, H, o);
      }
    };
    if (h0 < a.Hq)
      walk(h0, min(h1, a.Hq), a.q + t * a.q_stride + c0, s_w[0], w.live ? a.q_out + t * a.Hq * D + c0 : nullptr,
           nullptr);
    if (h1 > a.Hq)
      walk(max(h0, a.Hq) - a.Hq, h1 - a.Hq, a.k + t * a.k_stride + c0, s_w[1],
           w.page >= 0 ? a.k_pages + w.page * a.page_stride + static_cast<long long>(w.off) * HKV * D + c0 : nullptr,
           w.live && a.k_out ? a.k_out + t * HKV * D + c0 : nullptr);
  }
}

template <int D, int HKV>
__device__ __forceinline__ void value_blocks(const ApArgs& a, const int32_t* cu) {
  using Cfg = ApCfg<D, HKV>;
  constexpr int NT = Cfg::NT;
  __shared__ float red[2][Cfg::kWarps][16][8 * NT + 1];
  __shared__ long long s_dt[2][Cfg::kTiles][16];   // dt_pages offset of the tile's tokens, head 0 (-1: none)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, t4 = lane & 3;
  const int slice = warp % Cfg::kSlices, tl = warp / Cfg::kSlices;

  // B fragments: channel 8 t4 + e of each 32-channel step is k position
  // 2 t4 + (e & 1) + 8 ((e >> 1) & 1) of MMA e >> 2
  uint32_t bw[Cfg::kJ][2][NT][3][2];
#pragma unroll
  for (int j = 0; j < Cfg::kJ; ++j)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int g = gid + 8 * nt;
      const int ch = slice * Cfg::kSlice + 32 * j + 8 * t4;
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = g < HKV ? __ldg(a.W + static_cast<size_t>(ch + e) * HKV + g) : 0.0f;
#pragma unroll
      for (int term = 0; term < 3; ++term)
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const uint32_t u = pack_bf16x2(x[2 * p], x[2 * p + 1]);
          bw[j][p >> 1][nt][term][p & 1] = u;
          x[2 * p] -= __uint_as_float(u << 16);
          x[2 * p + 1] -= __uint_as_float(u & 0xFFFF0000u);
        }
    }

  const int ntiles = (a.T + 15) / 16;
  int buf = 0;
  for (int base = blockIdx.x * Cfg::kTiles; base < ntiles; base += a.val_blocks * Cfg::kTiles, buf ^= 1) {
    const int tile = base + tl;
    // lanes 0-15 (and again 16-31) locate the tile's tokens
    const Where w = locate(a, cu, tile < ntiles ? tile * 16 + (lane & 15) : a.T);
    if (slice == 0 && lane < 16)
      s_dt[buf][tl][lane] = w.page >= 0 ? static_cast<long long>(w.page) * HKV * a.page_size + w.off : -1;
    const long long row = w.page >= 0 ? w.page * a.page_stride + static_cast<long long>(w.off) * HKV * D : -1;
    const long long row0 = __shfl_sync(0xFFFFFFFFu, row, gid), row1 = __shfl_sync(0xFFFFFFFFu, row, gid + 8);
    const int ch = slice * Cfg::kSlice + 8 * t4;
    const uint16_t* v0 = a.v + static_cast<long long>(tile * 16 + gid) * a.v_stride + ch;
    const uint16_t* v1 = v0 + 8 * a.v_stride;
    uint4 x0[Cfg::kJ], x1[Cfg::kJ];
#pragma unroll
    for (int j = 0; j < Cfg::kJ; ++j) {
      x0[j] = row0 >= 0 ? __ldg(reinterpret_cast<const uint4*>(v0 + 32 * j)) : make_uint4(0u, 0u, 0u, 0u);
      x1[j] = row1 >= 0 ? __ldg(reinterpret_cast<const uint4*>(v1 + 32 * j)) : make_uint4(0u, 0u, 0u, 0u);
    }
    float acc[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[nt][i] = 0.0f;
#pragma unroll
    for (int j = 0; j < Cfg::kJ; ++j) {
      if (row0 >= 0) *reinterpret_cast<uint4*>(a.v_pages + row0 + ch + 32 * j) = x0[j];
      if (row1 >= 0) *reinterpret_cast<uint4*>(a.v_pages + row1 + ch + 32 * j) = x1[j];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int term = 2; term >= 0; --term) {
          mma_bf16(acc[nt], x0[j].x, x1[j].x, x0[j].y, x1[j].y, bw[j][0][nt][term][0], bw[j][0][nt][term][1]);
          mma_bf16(acc[nt], x0[j].z, x1[j].z, x0[j].w, x1[j].w, bw[j][1][nt][term][0], bw[j][1][nt][term][1]);
        }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      red[buf][warp][gid][8 * nt + 2 * t4] = acc[nt][0];
      red[buf][warp][gid][8 * nt + 2 * t4 + 1] = acc[nt][1];
      red[buf][warp][gid + 8][8 * nt + 2 * t4] = acc[nt][2];
      red[buf][warp][gid + 8][8 * nt + 2 * t4 + 1] = acc[nt][3];
    }
    __syncthreads();   // (the other buffer is read until the next one)
    for (int i = threadIdx.x; i < Cfg::kTiles * 16 * HKV; i += Cfg::kThreads) {
      const int tok = i % 16, g = i / 16 % HKV, tt = i / (16 * HKV);
      const long long at = s_dt[buf][tt][tok];
      if (at < 0) continue;
      float x = 0.0f;
#pragma unroll
      for (int sl = 0; sl < Cfg::kSlices; ++sl) x += red[buf][tt * Cfg::kSlices + sl][tok][g];
      a.dt_pages[at + static_cast<long long>(g) * a.page_size] = expf(__ldg(a.A + g) * softplus_f32(x));
    }
  }
}

template <int D, int HKV>
__global__ void __launch_bounds__(ApCfg<D, HKV>::kThreads, ApCfg<D, HKV>::kMinBlocks)
    append_paged_kernel(const __grid_constant__ ApArgs a, const __grid_constant__ RopeTurns turns) {
  constexpr int kThreads = ApCfg<D, HKV>::kThreads;
  __shared__ __align__(16) float s_w[2][D];
  __shared__ __align__(16) double s_turn[D / 2];
  __shared__ int32_t s_cu[kApCuCap + 1];
  pdl_wait();
  pdl_trigger();
  const bool staged = a.B <= kApCuCap;
  if (staged)
    for (int i = threadIdx.x; i <= a.B; i += kThreads) s_cu[i] = a.cu[i];
  for (int c = threadIdx.x; c < D; c += kThreads) {
    s_w[0][c] = a.q_w[c];
    s_w[1][c] = a.k_w[c];
    if (c < D / 2) s_turn[c] = turns.t[c];
  }
  __syncthreads();
  const int32_t* cu = staged ? s_cu : a.cu;
  if (static_cast<int>(blockIdx.x) < a.val_blocks)
    value_blocks<D, HKV>(a, cu);
  else
    row_blocks<D, HKV>(a, cu, s_w, s_turn);
}

template <int D, int HKV>
cudaError_t launch_append(ApArgs a, const RopeTurns& turns, int nsm, cudaStream_t s) {
  using Cfg = ApCfg<D, HKV>;
  const int slots = Cfg::kMinBlocks * nsm;
  const int ntiles = (a.T + 15) / 16;
  // resident blocks shared out by bytes moved: values (in and out) against q and k rows
  const int v_rows = 2 * HKV, r_rows = 2 * (a.Hq + HKV) + (a.k_out ? HKV : 0);
  const int val_want = (ntiles + Cfg::kTiles - 1) / Cfg::kTiles;
  a.val_blocks = std::max(1, std::min(val_want, slots * v_rows / (v_rows + r_rows)));
  const int row_slots = slots - a.val_blocks;
  const long long groups = (static_cast<long long>(a.T) + Cfg::GPW - 1) / Cfg::GPW;
  const long long row_warps = static_cast<long long>(row_slots) * Cfg::kWarps;
  a.splits = static_cast<int>(std::max(1LL, std::min<long long>(a.Hq + HKV, row_warps / groups)));
  const int row_blocks_n = static_cast<int>(std::min<long long>(groups * a.splits, row_slots));
  return launch_after(append_paged_kernel<D, HKV>, dim3(a.val_blocks + row_blocks_n), dim3(Cfg::kThreads), 0, s, a,
                      turns);
}

}  // namespace

cudaError_t launch_append_paged(const AppendPaged& p, uint32_t* err, cudaStream_t s) {
  const RopeTurns& turns = make_rope_turns(p.theta, p.d);
  const int nsm = sm_count();
  if (nsm <= 0) return cudaErrorInvalidDevice;
  ApArgs a;
  a.q = static_cast<const uint16_t*>(p.q);
  a.k = static_cast<const uint16_t*>(p.k);
  a.v = static_cast<const uint16_t*>(p.v);
  a.q_stride = p.q_stride;
  a.k_stride = p.k_stride;
  a.v_stride = p.v_stride;
  a.q_w = p.q_norm_w;
  a.k_w = p.k_norm_w;
  a.W = p.W_dt;
  a.A = p.A;
  a.cu = p.cu_tokens;
  a.positions = p.positions;
  a.table = p.page_table;
  a.q_out = static_cast<uint16_t*>(p.q_out);
  a.k_out = static_cast<uint16_t*>(p.k_out);
  a.k_pages = static_cast<uint16_t*>(p.k_pages);
  a.v_pages = static_cast<uint16_t*>(p.v_pages);
  a.dt_pages = p.dt_pages;
  a.page_stride = p.page_stride;
  a.eps = p.eps;
  a.T = p.T;
  a.B = p.B;
  a.max_pages = p.max_pages;
  a.num_pages = p.num_pages;
  a.page_size = p.page_size;
  a.Hq = p.Hq;
  a.splits = 1;
  a.val_blocks = 1;
  a.err = err;
#define DMA_AP_CASE(DD, HK) \
  if (p.d == DD && p.Hkv == HK) return launch_append<DD, HK>(a, turns, nsm, s);
  DMA_AP_CASE(64, 1) DMA_AP_CASE(64, 2) DMA_AP_CASE(64, 4) DMA_AP_CASE(64, 8) DMA_AP_CASE(64, 16)
  DMA_AP_CASE(128, 1) DMA_AP_CASE(128, 2) DMA_AP_CASE(128, 4) DMA_AP_CASE(128, 8) DMA_AP_CASE(128, 16)
#undef DMA_AP_CASE
  return cudaErrorInvalidValue;
}

}  // namespace dma
