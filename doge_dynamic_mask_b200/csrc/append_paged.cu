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
// (about 4 flops per byte), and W is read once per block.  A block has two jobs,
// one after the other: tiles of values, dealt to the blocks in turn, and q and k
// rows, dealt so that every block moves as many bytes in all.  (Blocks with one
// job each, shared out by bytes, ended 113 us and 85 us after the start at 32768
// tokens.)
//
// q and k rows.  A row's channels sit in d/16 adjacent lanes (a
// 16-byte chunk and its rotation partner's chunk each); a warp step takes four
// consecutive heads of a token (of two tokens at d = 64), a contiguous piece,
// and the token's angles, multiplied into the norm's weights, stay in registers
// for its rows.  The rows travel by cp.async through a ring in shared memory in
// which each lane reads back only what it copied itself: five steps in flight
// per warp without registers or barriers.
//
// v rows and dt.  Sixteen tokens are the M side of
// mma.m16n8k16, the kv heads the N side.  A dot product does not care in which
// order its channels are taken, so the A fragments are the 16-byte chunks as
// they come from memory (a quad of lanes covers 64 bytes of a row), through the
// same kind of ring, and the same registers are stored to the page.
// W is split exactly into three bf16 terms (each the rounding of what the
// previous ones leave), whose products with bf16 values are exact, so the
// float32 accumulators hold the float32 projection; a warp keeps the
// fragments of its 128 channels in registers for all of its tokens.  The
// projection is 2 Hkv flops per byte of V: far below what tcgen05 is for, and a
// 128-row tile would leave a decode step's few tokens on one SM.
//
// Measured.  32768 tokens, 16 + 8 heads of 128, K rows packed as well: 107 us for
// 605 MB, 5.7 TB/s (94 us at the copy rate).  9 prompts of up to 2047 tokens, 8 + 4
// heads of 64: 12.7 us for 43 MB, of which about 4 us are the start and W's split.
// 57 single tokens: 5.5 us, a launch and four dependent memory latencies.  One to four
// heads of each: 28 to 30 us for 21852 tokens of d = 128, whatever their number, against
// 5 to 10 us at the copy rate: a warp step is four heads of one token, and fewer leave
// its other rows empty.
#include <algorithm>

#include "rope.cuh"

namespace dma {
namespace {

constexpr int kApCuCap = 1024;       // sequences whose offsets fit the staged copy (57 tokens: 5.5 us with it, 6.6 without)

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
  RowShare share;                           // q and k rows: items below late_items are for the
  int late_items, late_block;               // blocks from late_block on, the others for those before it
  uint32_t* err;
};

// Where a token of the packed batch goes, from a look-up whose table entry may
// still be on its way.  live: the token belongs to a sequence; slot_ok: its
// position lies in the table; seq: where the search ended, a hint for the next
// token's.
struct Place {
  int pos, entry, off, seq;
  bool live, slot_ok;
};

// cu and positions: in shared memory when they fit.
struct Batch {
  const int32_t *cu, *positions;
};

__device__ __forceinline__ Place look_up(const ApArgs& a, const Batch& s, int token, int hint) {
  Place p{0, -1, 0, hint, false, false};
  if (token >= a.T || token < s.cu[0] || token >= s.cu[a.B]) return p;
  // cu[lo] <= token < cu[hi] holds throughout
  int lo = 0, hi = a.B;
  if (s.cu[hint] <= token) {
    lo = hint;
    if (token < s.cu[hint + 1]) hi = hint + 1;
  } else {
    hi = hint;
  }
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s.cu[mid] <= token)
      lo = mid;
    else
      hi = mid;
  }
  p.live = true;
  p.seq = lo;
  const long long pos = static_cast<long long>(s.positions[lo]) + (token - s.cu[lo]);
  p.slot_ok = pos >= 0 && pos < static_cast<long long>(a.max_pages) * a.page_size;
  p.pos = static_cast<int>(pos);   // (the angle of a position outside the cache is that of its low 32 bits)
  if (!p.slot_ok) {
    raise_error(a.err, kDevErrBadPosition);
    return p;
  }
  const int slot = p.pos / a.page_size;
  p.off = p.pos - slot * a.page_size;
  p.entry = __ldg(a.table + static_cast<size_t>(lo) * a.max_pages + slot);
  return p;
}

// The place's page, or -1 (reported) when it has none: nothing is written to the cache then.
__device__ __forceinline__ int page_of(const ApArgs& a, const Place& p) {
  if (!p.slot_ok) return -1;
  if (p.entry >= 0 && p.entry < a.num_pages) return p.entry;
  raise_error(a.err, kDevErrBadPage);
  return -1;
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
  static constexpr int kStages = 6;                         // ring steps per warp: two 16-byte chunks per lane each
  static constexpr int kSmemBytes = kWarps * kStages * 2 * 512;
};

template <int D, int HKV>
__device__ __forceinline__ void rows_job(const ApArgs& a, const Batch& batch, const float (*s_w)[D],
                                           const double* s_turn, uint4* dyn) {
  using Cfg = ApCfg<D, HKV>;
  constexpr int H = D / 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c0 = 8 * (lane % Cfg::LPR);
  const int late = static_cast<int>(blockIdx.x) >= a.late_block;
  const int blk = blockIdx.x - (late ? a.late_block : 0), nblk = late ? gridDim.x - a.late_block : a.late_block;
  const int stride = nblk * Cfg::kWarps, it0 = (late ? 0 : a.late_items) + warp * nblk + blk;
  const int items = late ? a.late_items : a.share.items;
  const int row0 = RowItem<D>::row();

  // ---- the ring: rows on their way
  constexpr int STG = Cfg::kStages;
  uint4* ring = dyn + warp * STG * 64 + lane;   // [stage][lo, hi][lane]
  const uint32_t ring_u = smem_u32(ring);
  int f_it = it0, f_s = 0, f_h = 0, f_n = 0;
  RowItem<D> f{};
  const uint16_t* f_x = a.q;
  auto f_tensor = [&](int n, int s) {   // step s is in tensor n
    f_n = n;
    f_h = 4 * s + row0;
    const long long t = f.token;
    f_x = (n ? a.k + t * a.k_stride : a.q + t * a.q_stride) + f_h * D + c0;
  };
  auto f_enter = [&]() {
    f.enter(a.share, f_it);
    f_s = f.s0;
    const int n = f_s >= a.share.q_steps;
    f_tensor(n, n ? f_s - a.share.q_steps : f_s);
  };
  f_enter();
  auto issue = [&](int slot) {
    if (f_it < items) {
      const bool there = f.there && f_h < a.share.heads[f_n];
      const uint16_t* x = there ? f_x : a.q;
      const uint32_t dst = ring_u + slot * 1024;
      cp_async16_zfill(dst, x, there);
      cp_async16_zfill(dst + 512, x + H, there);
      f_x += 4 * D;
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
  for (int s = 0; s < STG - 1; ++s) issue(s);

  int slot = 0;
  RowItem<D> i;
  i.enter(a.share, it0);
  Place next = look_up(a, batch, it0 < items && i.there ? i.token : a.T, 0);
  for (int it = it0; it < items; it += stride) {
    const Place w = next;
    const RowItem<D> now = i;
    i.enter(a.share, it + stride);   // the next item's place is looked up while this one's rows are computed
    next = look_up(a, batch, it + stride < items && i.there ? i.token : a.T, w.seq);
    const RowAngles ang = token_angles<D>(static_cast<double>(w.pos), s_turn);
    // one row, normalised and rotated
    auto row = [&](const RowTurn& turn) {
      cp_wait<STG - 2>();
      const RowChunk x = widen_row(RawChunk{ring[slot * 64], ring[slot * 64 + 32]});
      issue(slot == 0 ? STG - 1 : slot - 1);   // the step read last time
      slot = slot + 1 == STG ? 0 : slot + 1;
      const float r = rsqrtf(row_sum<Cfg::LPR>(chunk_dot(x, x)) * (1.0f / D) + a.eps);
      const unsigned long long r2 = f32x2(r, r);
      RowChunk y = turn_row(x, turn);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        y.lo[e] = mul_f32x2(y.lo[e], r2);
        y.hi[e] = mul_f32x2(y.hi[e], r2);
      }
      return round_row(y);
    };
    const long long t = now.token;
    if (now.s0 < a.share.q_steps) {
      const RowTurn turn = row_turn(ang, load_weights(s_w[0] + c0, H));
      int h = 4 * now.s0 + row0;
      uint16_t* out = a.q_out + (t * a.share.heads[0] + h) * D + c0;
      for (int s = now.s0; s < min(now.s1, a.share.q_steps); ++s, h += 4, out += 4 * D) {
        const RawChunk o = row(turn);
        if (w.live && h < a.share.heads[0]) store_row(out, H, o);
      }
    }
    if (now.s1 > a.share.q_steps) {
      const RowTurn turn = row_turn(ang, load_weights(s_w[1] + c0, H));
      const int k0 = max(now.s0, a.share.q_steps);
      int h = 4 * (k0 - a.share.q_steps) + row0;
      uint16_t* out = a.k_out + (t * HKV + h) * D + c0;
      const int page = page_of(a, w);
      uint16_t* cache = a.k_pages + page * a.page_stride + (static_cast<long long>(w.off) * HKV + h) * D + c0;
      for (int s = k0; s < now.s1; ++s, h += 4, out += 4 * D, cache += 4 * D) {
        const RawChunk o = row(turn);
        if (page >= 0 && h < HKV) store_row(cache, H, o);
        if (w.live && a.k_out && h < HKV) store_row(out, H, o);
      }
    }
  }
  cp_wait<0>();
}

template <int D, int HKV>
__device__ __forceinline__ void values_job(const ApArgs& a, const Batch& batch, uint4* dyn) {
  using Cfg = ApCfg<D, HKV>;
  constexpr int NT = Cfg::NT;
  __shared__ float red[2][Cfg::kWarps][16][8 * NT + 1];
  __shared__ long long s_dt[2][Cfg::kTiles][16];   // dt_pages offset of the tile's tokens, head 0 (-1: none)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, t4 = lane & 3;
  const int slice = warp % Cfg::kSlices, tl = warp / Cfg::kSlices;

  const int ntiles = (a.T + 15) / 16;
  const int base0 = blockIdx.x * Cfg::kTiles;
  if (base0 >= ntiles) return;
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

  // ---- the ring: this lane's chunks of two rows, 64 bytes of each row, per step
  constexpr int STG = Cfg::kStages;
  uint4* ring = dyn + warp * STG * 64 + lane;   // [stage][row][lane]
  const uint32_t ring_u = smem_u32(ring);
  const int step = gridDim.x * Cfg::kTiles;
  const int ch = slice * Cfg::kSlice + 8 * t4;
  int f_base = base0, f_j = 0;
  auto issue = [&](int slot) {
    if (f_base < ntiles) {
      const long long t = static_cast<long long>(f_base + tl) * 16 + gid;
      const bool there0 = t < a.T, there1 = t + 8 < a.T;
      const uint16_t* v = a.v + ch + 32 * f_j;
      cp_async16_zfill(ring_u + slot * 1024, v + (there0 ? t * a.v_stride : 0), there0);
      cp_async16_zfill(ring_u + slot * 1024 + 512, v + (there1 ? (t + 8) * a.v_stride : 0), there1);
      if (++f_j == Cfg::kJ) {
        f_j = 0;
        f_base += step;
      }
    }
    cp_commit();
  };
  // lanes 0-15 (and again 16-31) locate the tile's tokens
  auto where_of = [&](int base, int hint) {
    return look_up(a, batch, base + tl < ntiles ? (base + tl) * 16 + (lane & 15) : a.T, hint);
  };
#pragma unroll
  for (int s = 0; s < STG - 1; ++s) issue(s);
  Place next = where_of(base0, 0);
  int buf = 0, slot = 0;
  for (int base = base0; base < ntiles; base += step, buf ^= 1) {
    const Place w = next;
    const int page = page_of(a, w);
    next = where_of(base + step, w.seq);   // its loads travel while this tile is computed
    if (slice == 0 && lane < 16)
      s_dt[buf][tl][lane] = page >= 0 ? static_cast<long long>(page) * HKV * a.page_size + w.off : -1;
    const long long row = page >= 0 ? page * a.page_stride + static_cast<long long>(w.off) * HKV * D : -1;
    const long long row0 = __shfl_sync(0xFFFFFFFFu, row, gid), row1 = __shfl_sync(0xFFFFFFFFu, row, gid + 8);
    float acc[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[nt][i] = 0.0f;
#pragma unroll
    for (int j = 0; j < Cfg::kJ; ++j) {
      cp_wait<STG - 2>();
      const uint4 x0 = ring[slot * 64], x1 = ring[slot * 64 + 32];
      issue(slot == 0 ? STG - 1 : slot - 1);   // the step read last time
      slot = slot + 1 == STG ? 0 : slot + 1;
      if (row0 >= 0) *reinterpret_cast<uint4*>(a.v_pages + row0 + ch + 32 * j) = x0;
      if (row1 >= 0) *reinterpret_cast<uint4*>(a.v_pages + row1 + ch + 32 * j) = x1;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int term = 2; term >= 0; --term) {
          mma_bf16(acc[nt], x0.x, x1.x, x0.y, x1.y, bw[j][0][nt][term][0], bw[j][0][nt][term][1]);
          mma_bf16(acc[nt], x0.z, x1.z, x0.w, x1.w, bw[j][1][nt][term][0], bw[j][1][nt][term][1]);
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
  cp_wait<0>();
}

template <int D, int HKV>
__global__ void __launch_bounds__(ApCfg<D, HKV>::kThreads, ApCfg<D, HKV>::kMinBlocks)
    append_paged_kernel(const __grid_constant__ ApArgs a, const __grid_constant__ RopeTurns turns) {
  constexpr int kThreads = ApCfg<D, HKV>::kThreads;
  __shared__ __align__(16) float s_w[2][D];
  __shared__ __align__(16) double s_turn[D / 2];
  __shared__ int32_t s_cu[kApCuCap + 1], s_pos[kApCuCap];
  extern __shared__ __align__(16) uint4 dyn[];
  pdl_wait();
  pdl_trigger();
  const bool staged = a.B <= kApCuCap;
  if (staged)
    for (int i = threadIdx.x; i <= a.B; i += kThreads) {
      s_cu[i] = a.cu[i];
      if (i < a.B) s_pos[i] = a.positions[i];
    }
  for (int c = threadIdx.x; c < D; c += kThreads) {
    s_w[0][c] = a.q_w[c];
    s_w[1][c] = a.k_w[c];
    if (c < D / 2) s_turn[c] = turns.t[c];
  }
  __syncthreads();
  const Batch batch{staged ? s_cu : a.cu, staged ? s_pos : a.positions};
  values_job<D, HKV>(a, batch, dyn);
  rows_job<D, HKV>(a, batch, s_w, s_turn, dyn);
}

template <int D, int HKV>
cudaError_t launch_append(ApArgs a, const RopeTurns& turns, int nsm, cudaStream_t s) {
  using Cfg = ApCfg<D, HKV>;
  const int slots = Cfg::kMinBlocks * nsm;
  const int ntiles = (a.T + 15) / 16;
  a.share = share_rows(a.T, a.Hq, HKV, D, static_cast<long long>(slots) * Cfg::kWarps);
  // few tiles and items spread over SMs before a block gets a second one
  const int passes = (ntiles + Cfg::kTiles - 1) / Cfg::kTiles;   // a block's tiles at once
  const int blocks = static_cast<int>(std::min<long long>(slots, static_cast<long long>(passes) + a.share.items));
  // the first blocks have a pass more than the others: the others get as many
  // row items more as move the same bytes
  const double pass = 2.0 * Cfg::kTiles * 16 * HKV;   // rows in and out
  const double item = (2.0 * (a.Hq + HKV) + (a.k_out ? HKV : 0)) * (128 / D) / a.share.parts;
  const double each = (passes * pass + a.share.items * item) / blocks;
  a.late_block = passes % blocks;
  const double late = std::max(0.0, each - passes / blocks * pass) / item * (blocks - a.late_block);
  a.late_items = a.late_block == 0 ? a.share.items
                                   : static_cast<int>(std::min<double>(a.share.items, std::ceil(late)));
  if (each <= (passes / blocks + 1) * pass) a.late_items = a.share.items;
  const cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(append_paged_kernel<D, HKV>), Cfg::kSmemBytes);
  if (e != cudaSuccess) return e;
  return launch_after(append_paged_kernel<D, HKV>, dim3(blocks), dim3(Cfg::kThreads),
                      Cfg::kSmemBytes, s, a, turns);
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
  a.err = err;
#define DMA_AP_CASE(DD, HK) \
  if (p.d == DD && p.Hkv == HK) return launch_append<DD, HK>(a, turns, nsm, s);
  DMA_AP_CASE(64, 1) DMA_AP_CASE(64, 2) DMA_AP_CASE(64, 4) DMA_AP_CASE(64, 8) DMA_AP_CASE(64, 16)
  DMA_AP_CASE(128, 1) DMA_AP_CASE(128, 2) DMA_AP_CASE(128, 4) DMA_AP_CASE(128, 8) DMA_AP_CASE(128, 16)
#undef DMA_AP_CASE
  return cudaErrorInvalidValue;
}

}  // namespace dma
