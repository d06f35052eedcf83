// Decode attention over a paged cache: one new query per sequence against its kept keys.
//
// Method: page "Transformers 中的 Doge 小语言模型完全指南", section
// "动态掩码注意力（DMA）：从缓存 value states 生成稀疏掩码", step 4 (scores scaled by
// head_dim^-0.5 plus dt as an additive mask, softmax in float32) for the decode
// query.  For head h of kv group g, over the kept keys j:
//
//   s_j = scale q_h . k_j + dt_j,   o_h = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m)
//
// with a running maximum m (in log2 units), so the keys are read once.
//
// Design.  Memory-bound: every kept K and V row is read once, 4 Hq/Hkv flops
// per 2 bytes.  All rows of all sequences and kv heads form one axis of 16-key
// tiles, and the warps of the grid take equal contiguous ranges of it, so
// ragged batches and single long sequences fill the SMs alike; a warp that
// ends or begins inside a row leaves a float32 partial (o, m, l) that a second
// kernel joins, in the order of the axis.  A warp works alone: its tiles travel
// by cp.async through a ring of its own (keys that do not exist are filled with
// zeros and masked), with table entries and dt fetched further ahead.  The
// products run on mma.m16n8k16 with the keys (and, for P V, the channels) on
// the M side and the group's query heads, at most eight, on the N side: no
// row of a tile is padding, which tcgen05's 128 rows could not offer to one
// query, and the tensor work stays far below the copy time.  P is split into
// two bf16 terms, so its rounding (2^-17) does not show in the output.
#include <algorithm>

#include "paged.cuh"

namespace dma {
namespace {

constexpr int kDpWarps = 8;
constexpr int kDpThreads = 32 * kDpWarps;
constexpr int kTileKeys = 16;
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct DpCfg {
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kRowBytes = D * 2;
  static constexpr int kTileBytes = kTileKeys * kRowBytes;         // K rows (V rows follow)
  static constexpr int kStageBytes = 2 * kTileBytes + kTileKeys * 4;   // + the keys' biases
  static constexpr int kSmemBytes = kDpWarps * kStages * kStageBytes;
};

struct DpArgs {
  PagedCache c;
  PagedLists lists;
  const uint16_t *q, *k, *v;
  uint16_t* out;
  float* part;        // [workers][2][Hq / Hkv][d + 2]: o, m, l of the pieces at a range's ends
  float scale;
  int Hq, workers;
};

__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ int row_tiles(int keys) { return max(1, (keys + kTileKeys - 1) / kTileKeys); }

// Tiles of one (sequence, kv head) row of the axis; a sequence without keys has
// one empty tile, whose output is zero.
__device__ __forceinline__ int seq_tiles(const PagedCache& c, int b) { return row_tiles(min(seq_view(c, b).n, c.w)); }

// Position on the axis: row (b, g), tile t of nt, and what the row keeps.
struct Cursor {
  SeqView view;
  int b, g, t, nt, keys;
  bool listed;

  __device__ __forceinline__ void enter(const PagedCache& c) {
    view = seq_view(c, b);
    keys = min(view.n, c.w);
    listed = view.n > c.w;
    nt = row_tiles(keys);
  }
  __device__ __forceinline__ void next(const PagedCache& c) {
    if (++t < nt) return;
    t = 0;
    if (++g < c.Hkv) return;
    g = 0;
    if (++b < c.B) enter(c);
  }
};

// One key of a tile on its way to the ring, per lane (lane & 15 is the key).
struct KeyRef {
  uint32_t row;      // offset of its K / V row in 16-byte units, or kNoRow
  float bias;        // dt
};

template <int D>
__global__ void __launch_bounds__(kDpThreads, 1) decode_paged_kernel(const __grid_constant__ DpArgs a) {
  using Cfg = DpCfg<D>;
  constexpr int KS = D / 16;            // k16 steps of q.k; 16-channel tiles of o
  constexpr int CPR = D / 8;            // 16-byte chunks per row
  constexpr int RPI = 32 / CPR;         // rows per copy step of a warp
  constexpr int STG = Cfg::kStages;
  extern __shared__ __align__(128) unsigned char ring_all[];
  __shared__ uint32_t s_scan[64];
  __shared__ long long s_pref[kDpThreads + 1];
  const PagedCache& c = a.c;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // ---- this warp's range [x0, x1) of the axis
  long long total = 0;
  for (int b0 = 0; b0 < c.B; b0 += kDpThreads) {
    uint32_t n;
    block_exclusive_scan(b0 + tid < c.B ? static_cast<uint32_t>(seq_tiles(c, b0 + tid)) : 0u, s_scan, &n);
    total += n;
  }
  const long long U = total * c.Hkv;
  const long long W = min(static_cast<long long>(a.workers), U);
  const long long wk = static_cast<long long>(warp) * gridDim.x + blockIdx.x;
  const long long x0 = wk < W ? U * wk / W : 0, x1 = wk < W ? U * (wk + 1) / W : 0;
  Cursor cur{};
  {
    const long long y = x0 / c.Hkv;   // tiles of sequences before this one, rounded into it
    long long before = 0;
    for (int b0 = 0; b0 < c.B; b0 += kDpThreads) {
      uint32_t n;
      const uint32_t ex =
          block_exclusive_scan(b0 + tid < c.B ? static_cast<uint32_t>(seq_tiles(c, b0 + tid)) : 0u, s_scan, &n);
      s_pref[tid] = before + ex;
      if (tid == 0) s_pref[kDpThreads] = before + n;
      __syncthreads();
      if (y >= before && y < before + n) {
        int lo = 0, hi = kDpThreads;   // s_pref[lo] <= y < s_pref[hi]
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (s_pref[mid] <= y)
            lo = mid;
          else
            hi = mid;
        }
        cur.b = b0 + lo;
        cur.enter(c);
        const long long rem = x0 - s_pref[lo] * c.Hkv;
        cur.g = static_cast<int>(rem / cur.nt);
        cur.t = static_cast<int>(rem % cur.nt);
      }
      before += n;
      __syncthreads();
    }
  }
  const int count = static_cast<int>(x1 - x0);
  if (count == 0) return;

  // ---- the ring: fetch (table entry or list entry) -> resolve (dt) -> issue (rows)
  unsigned char* ring = ring_all + static_cast<size_t>(warp) * STG * Cfg::kStageBytes;
  const uint32_t ring_u = smem_u32(ring);
  const int kl = lane & 15;
  Cursor fc = cur;       // the fetch side's cursor
  int fetched = 0;
  // what fetch left for resolve: a page (and the key's row of it), or a list entry
  int f_page = 0, f_off = 0, f_g = 0;
  KeyRef f_ref{kNoRow, 0.0f};
  bool f_direct = false;
  auto fetch = [&]() {
    f_direct = false;
    f_ref = KeyRef{kNoRow, 0.0f};
    if (fetched < count) {
      const int i = fc.t * kTileKeys + kl;
      if (i < fc.keys) {
        if (fc.listed) {
          const size_t at = (static_cast<size_t>(fc.b) * c.Hkv + fc.g) * a.lists.cap + i;
          f_ref = KeyRef{a.lists.row[at], a.lists.bias[at]};
        } else {
          f_direct = true;
          const int slot = page_slot(c, key_position(c, fc.view, i), f_off);
          f_page = __ldg(c.table + static_cast<size_t>(fc.b) * c.max_pages + slot);
          f_g = fc.g;
        }
      }
      fc.next(c);
    }
    ++fetched;
  };
  auto resolve = [&]() {
    KeyRef r = f_ref;
    if (f_direct) {
      const int page = checked_page(c, f_page);
      if (page >= 0) {
        r.row = row_offset16(c, page, f_off, f_g);
        r.bias = __ldg(c.dt_pages + dt_offset(c, page, f_off, f_g));
      }
    }
    return r;
  };
  const int cr = lane / CPR, cc = lane % CPR;
  auto issue = [&](const KeyRef& r, int slot) {
    const uint32_t st = ring_u + slot * Cfg::kStageBytes;
#pragma unroll
    for (int i = 0; i < kTileKeys / RPI; ++i) {
      const int row = i * RPI + cr;
      const uint32_t off = __shfl_sync(0xFFFFFFFFu, r.row, row);
      const bool there = off != kNoRow;
      const size_t e = there ? (static_cast<size_t>(off) + cc) * 8 : 0;
      const uint32_t dst = st + row * Cfg::kRowBytes + ((cc ^ (row & 7)) << 4);
      cp_async16_zfill(dst, a.k + e, there);
      cp_async16_zfill(dst + Cfg::kTileBytes, a.v + e, there);
    }
    if (lane < kTileKeys)
      *reinterpret_cast<float*>(ring + slot * Cfg::kStageBytes + 2 * Cfg::kTileBytes + 4 * lane) =
          r.row != kNoRow ? r.bias * kLog2e : -INFINITY;
  };
  fetch();
  KeyRef ref = resolve();
  fetch();
#pragma unroll
  for (int s = 0; s < STG - 1; ++s) {
    if (s < count) issue(ref, s);
    cp_commit();
    ref = resolve();
    fetch();
  }

  // ---- the tiles
  const int gid = lane >> 2, t4 = lane & 3;
  const int nrep = a.Hq / c.Hkv;
  const float sl = a.scale * kLog2e;
  // ldmatrix addresses: K rows (row of the lane's 8x8 block, chunk parity), V rows transposed
  const int k_row = ((lane >> 3) & 1) * 8 + (lane & 7), k_par = lane >> 4;
  const int v_row = (lane >> 4) * 8 + (lane & 7), v_par = (lane >> 3) & 1;
  uint32_t qf[KS][2];
  float o[KS][4];
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
  bool fresh = true;        // the next tile begins this warp's piece of a row
  bool from_start = false;  // the piece begins at the row's first tile
  int slot = 0;
  for (int x = 0; x < count; ++x) {
    if (fresh) {
      fresh = false;
      from_start = cur.t == 0;
      const uint16_t* qr = a.q + (static_cast<size_t>(cur.b) * a.Hq + cur.g * nrep + gid) * D + 2 * t4;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        qf[s][0] = gid < nrep ? __ldg(reinterpret_cast<const uint32_t*>(qr + 16 * s)) : 0u;
        qf[s][1] = gid < nrep ? __ldg(reinterpret_cast<const uint32_t*>(qr + 16 * s + 8)) : 0u;
        o[s][0] = o[s][1] = o[s][2] = o[s][3] = 0.0f;
      }
      m0 = m1 = -INFINITY;
      l0 = l1 = 0.0f;
    }
    cp_wait<STG - 2>();
    __syncwarp();   // every lane's copies of this stage have landed; the previous stage has been read
    {
      const int nslot = slot == 0 ? STG - 1 : slot - 1;
      if (x + STG - 1 < count) issue(ref, nslot);
      cp_commit();
      ref = resolve();
      fetch();
    }
    const uint32_t st = ring_u + slot * Cfg::kStageBytes;
    float sa[4] = {0.0f, 0.0f, 0.0f, 0.0f}, sb[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int s = 0; s < KS; s += 2) {
      uint32_t ka[4], kb[4];
      ldsm4(ka, st + k_row * Cfg::kRowBytes + (((2 * s + k_par) ^ (k_row & 7)) << 4));
      ldsm4(kb, st + k_row * Cfg::kRowBytes + (((2 * s + 2 + k_par) ^ (k_row & 7)) << 4));
      mma16816(sa, ka, qf[s][0], qf[s][1]);
      mma16816(sb, kb, qf[s + 1][0], qf[s + 1][1]);
    }
    const float* bias = reinterpret_cast<const float*>(ring + slot * Cfg::kStageBytes + 2 * Cfg::kTileBytes);
    const float b0 = bias[gid], b1 = bias[gid + 8];
    // scores in log2 units: keys gid and gid + 8, heads 2 t4 and 2 t4 + 1
    const float s00 = b0 == -INFINITY ? -INFINITY : fmaf(sa[0] + sb[0], sl, b0);
    const float s01 = b0 == -INFINITY ? -INFINITY : fmaf(sa[1] + sb[1], sl, b0);
    const float s10 = b1 == -INFINITY ? -INFINITY : fmaf(sa[2] + sb[2], sl, b1);
    const float s11 = b1 == -INFINITY ? -INFINITY : fmaf(sa[3] + sb[3], sl, b1);
    const float t0 = fmaxf(s00, s10), t1 = fmaxf(s01, s11);
    // the maximum follows only when a score outgrows it by 2^8: the terms then
    // stay below 2^8 and the sums below 2^28
    if (__any_sync(0xFFFFFFFFu, t0 > m0 + 8.0f || t1 > m1 + 8.0f)) {
      float n0 = fmaxf(m0, t0), n1 = fmaxf(m1, t1);
#pragma unroll
      for (int d = 4; d <= 16; d <<= 1) {
        n0 = fmaxf(n0, __shfl_xor_sync(0xFFFFFFFFu, n0, d));
        n1 = fmaxf(n1, __shfl_xor_sync(0xFFFFFFFFu, n1, d));
      }
      const float f0 = m0 == n0 ? 1.0f : fast_exp2(m0 - n0), f1 = m1 == n1 ? 1.0f : fast_exp2(m1 - n1);
      m0 = n0;
      m1 = n1;
      l0 *= f0;
      l1 *= f1;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        o[s][0] *= f0;
        o[s][1] *= f1;
        o[s][2] *= f0;
        o[s][3] *= f1;
      }
    }
    const float p00 = s00 == -INFINITY ? 0.0f : fast_exp2(s00 - m0), p01 = s01 == -INFINITY ? 0.0f : fast_exp2(s01 - m1);
    const float p10 = s10 == -INFINITY ? 0.0f : fast_exp2(s10 - m0), p11 = s11 == -INFINITY ? 0.0f : fast_exp2(s11 - m1);
    l0 += p00 + p10;
    l1 += p01 + p11;
    const uint32_t h0 = pack_bf16x2(p00, p01), h1 = pack_bf16x2(p10, p11);
    const uint32_t e0 = pack_bf16x2(p00 - __uint_as_float(h0 << 16), p01 - __uint_as_float(h0 & 0xFFFF0000u));
    const uint32_t e1 = pack_bf16x2(p10 - __uint_as_float(h1 << 16), p11 - __uint_as_float(h1 & 0xFFFF0000u));
    const uint32_t ph0 = transpose8x8(h0), ph1 = transpose8x8(h1), pe0 = transpose8x8(e0), pe1 = transpose8x8(e1);
    const uint32_t sv = st + Cfg::kTileBytes;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      uint32_t va[4];
      ldsm4_t(va, sv + v_row * Cfg::kRowBytes + (((2 * s + v_par) ^ (v_row & 7)) << 4));
      mma16816(o[s], va, ph0, ph1);
      mma16816(o[s], va, pe0, pe1);
    }
    slot = slot + 1 == STG ? 0 : slot + 1;

    const bool row_end = cur.t + 1 == cur.nt;
    if (row_end || x + 1 == count) {
      float L0 = l0, L1 = l1;
#pragma unroll
      for (int d = 4; d <= 16; d <<= 1) {
        L0 += __shfl_xor_sync(0xFFFFFFFFu, L0, d);
        L1 += __shfl_xor_sync(0xFFFFFFFFu, L1, d);
      }
      const int ha = 2 * t4, hb = ha + 1;
      if (row_end && from_start) {
        const float i0 = L0 == 0.0f ? 0.0f : 1.0f / L0, i1 = L1 == 0.0f ? 0.0f : 1.0f / L1;
        __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(a.out) +
                             (static_cast<size_t>(cur.b) * a.Hq + cur.g * nrep + ha) * D + gid;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          if (ha < nrep) {
            dst[16 * s] = __float2bfloat16_rn(o[s][0] * i0);
            dst[16 * s + 8] = __float2bfloat16_rn(o[s][2] * i0);
          }
          if (hb < nrep) {
            dst[D + 16 * s] = __float2bfloat16_rn(o[s][1] * i1);
            dst[D + 16 * s + 8] = __float2bfloat16_rn(o[s][3] * i1);
          }
        }
      } else {
        // slot 1: the piece begins its row here and ends elsewhere; slot 0: the row began before
        float* dst = a.part + ((wk * 2 + (from_start ? 1 : 0)) * nrep + ha) * (D + 2);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          if (ha < nrep) {
            dst[16 * s + gid] = o[s][0];
            dst[16 * s + 8 + gid] = o[s][2];
          }
          if (hb < nrep) {
            dst[D + 2 + 16 * s + gid] = o[s][1];
            dst[D + 2 + 16 * s + 8 + gid] = o[s][3];
          }
        }
        if (gid == 0 && ha < nrep) {
          dst[D] = m0;
          dst[D + 1] = L0;
        }
        if (gid == 0 && hb < nrep) {
          dst[2 * D + 2] = m1;
          dst[2 * D + 3] = L1;
        }
      }
      fresh = true;
    }
    cur.next(c);
  }
  cp_wait<0>();
}

// Joins the pieces of rows that more than one warp worked on, in the order of
// the axis: one block per (sequence, query head), a thread per channel.
template <int D>
__global__ void __launch_bounds__(D) decode_paged_join_kernel(const __grid_constant__ DpArgs a) {
  __shared__ long long s_sum[2];
  const PagedCache& c = a.c;
  pdl_wait();
  const int b = blockIdx.x / a.Hq, h = blockIdx.x % a.Hq;
  const int nrep = a.Hq / c.Hkv, g = h / nrep;
  if (threadIdx.x < 2) s_sum[threadIdx.x] = 0;
  __syncthreads();
  long long before = 0, all = 0;
  for (int i = threadIdx.x; i < c.B; i += D) {
    const int n = seq_tiles(c, i);
    all += n;
    before += i < b ? n : 0;
  }
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) {
    all += __shfl_xor_sync(0xFFFFFFFFu, all, d);
    before += __shfl_xor_sync(0xFFFFFFFFu, before, d);
  }
  if ((threadIdx.x & 31) == 0) {
    atomicAdd(reinterpret_cast<unsigned long long*>(&s_sum[0]), static_cast<unsigned long long>(all));
    atomicAdd(reinterpret_cast<unsigned long long*>(&s_sum[1]), static_cast<unsigned long long>(before));
  }
  __syncthreads();
  const long long U = s_sum[0] * c.Hkv, W = min(static_cast<long long>(a.workers), U);
  const int nt = seq_tiles(c, b);
  const long long t0 = s_sum[1] * c.Hkv + static_cast<long long>(g) * nt, t1 = t0 + nt;   // the row on the axis
  const long long w0 = (W * (t0 + 1) - 1) / U, w1 = (W * t1 - 1) / U;                     // its first and last warp
  if (w0 == w1) return;   // one warp had it all and has written it
  const int e = threadIdx.x;
  const size_t slot = static_cast<size_t>(nrep) * (D + 2);
  const float* p0 = a.part + w0 * 2 * slot + static_cast<size_t>(h - g * nrep) * (D + 2);
  const int np = static_cast<int>(w1 - w0) + 1;
  // the first warp's piece is in slot 1 when the row begins inside or at the start of its range
  auto piece = [&](int i) { return p0 + (i == 0 ? 1 : 2 * i) * slot; };
  float M = -INFINITY;
#pragma unroll 8
  for (int i = 0; i < np; ++i) M = fmaxf(M, piece(i)[D]);
  float num = 0.0f, den = 0.0f;
#pragma unroll 8
  for (int i = 0; i < np; ++i) {
    const float* p = piece(i);
    const float wgt = p[D] == -INFINITY ? 0.0f : fast_exp2(p[D] - M);
    num = fmaf(wgt, p[e], num);
    den = fmaf(wgt, p[D + 1], den);
  }
  reinterpret_cast<__nv_bfloat16*>(a.out)[static_cast<size_t>(blockIdx.x) * D + e] =
      __float2bfloat16_rn(den == 0.0f ? 0.0f : num / den);
}

template <int D>
cudaError_t launch_dp(const DpArgs& a, int blocks, cudaStream_t s) {
  cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(decode_paged_kernel<D>), DpCfg<D>::kSmemBytes);
  if (e != cudaSuccess) return e;
  e = launch_after(decode_paged_kernel<D>, dim3(blocks), dim3(kDpThreads), DpCfg<D>::kSmemBytes, s, a);
  if (e != cudaSuccess) return e;
  return launch_after(decode_paged_join_kernel<D>, dim3(static_cast<unsigned>(a.c.B) * a.Hq), dim3(D), 0, s, a);
}

}  // namespace

cudaError_t launch_attn_paged(const PagedCache& c, const PagedLists& lists, const void* q, const void* k_pages,
                              const void* v_pages, int Hq, float scale, float* part, void* out, cudaStream_t s) {
  const int nsm = sm_count();
  if (nsm <= 0) return cudaErrorInvalidDevice;
  DpArgs a;
  a.c = c;
  a.lists = lists;
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k_pages);
  a.v = static_cast<const uint16_t*>(v_pages);
  a.out = static_cast<uint16_t*>(out);
  a.part = part;
  a.scale = scale;
  a.Hq = Hq;
  const int blocks = std::min(nsm, kPagedMaxWorkers / kDpWarps);
  a.workers = blocks * kDpWarps;
  return c.d == 64 ? launch_dp<64>(a, blocks, s) : launch_dp<128>(a, blocks, s);
}

}  // namespace dma
