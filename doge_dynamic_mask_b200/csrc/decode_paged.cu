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
// tiles, and the blocks of the grid, and their warps, take equal contiguous
// ranges of it, so ragged batches and single long sequences fill the SMs
// alike (few rows of like lengths get a block each).  A warp that begins or ends
// inside a row leaves a float32 piece (o, m, l); a block joins its warps' pieces,
// and of the blocks that share a row the last one to finish joins theirs, always
// in the order of the axis.  A warp works alone: its tiles travel by cp.async
// through a ring of its own (keys that do not exist are filled with zeros and
// masked), with positions, table entries and dt fetched further ahead.  The
// products run on mma.m16n8k16 with the keys (and, for P V, the channels) on the
// M side and the group's query heads, at most eight, on the N side: no row of a
// tile is padding, which tcgen05's 128 rows could not offer to one query, and the
// tensor work stays far below the copy time.  P is split into three bf16 terms, its
// 24 bits exactly; groups of one or two heads have the terms side by side in the eight
// columns (8 sequences of 64k to 128k keys, call after call: 484 us so, 492 us with three
// products each), and larger groups take three products.
//
// Measured.  Long rows kept whole (8 sequences of 64k to 128k keys, 8 heads of
// 128) run at the copy rate: 480 us for 3.2 GB, 6.7 TB/s.  Kept lists of 2048 of
// 32k to 64k keys, 64 sequences: about 102 us for 540 MB, 5.3 TB/s in scattered
// 256-byte rows.  Small calls are bound by the chain lengths, table, rows, pieces,
// each a memory latency: 32 ragged sequences of up to 2048 keys of 4 heads of 64,
// 14.8 us for 34 MB; one sequence of 301 keys, 6.6 us.
#include <algorithm>

#include "paged.cuh"

namespace dma {
namespace {

constexpr int kDpMaxWarps = 16;
constexpr int kTileKeys = 16;
constexpr uint32_t kRowSteps = 3;   // tiles of a warp that cost less than joining a row's blocks
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kFewWarpsLength = 4096;   // longest row (d = 64) for which blocks of eight warps are taken

// W: warps of a block.  d = 128 takes 204 registers a thread: eight, 25 KB of ring
// each.  d = 64 has room for sixteen (see the launch).
template <int D, int W>
struct DpCfg {
  static constexpr int kWarps = W;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kStages = 3;
  static constexpr int kRowBytes = D * 2;
  static constexpr int kTileBytes = kTileKeys * kRowBytes;         // K rows (V rows follow)
  static constexpr int kStageBytes = 2 * kTileBytes + kTileKeys * 8;   // + the keys' masks (0 or -inf) and dt
  static constexpr int kSmemBytes = kWarps * kStages * kStageBytes;
};

struct DpArgs {
  PagedCache c;
  PagedLists lists;
  const uint16_t *q, *k, *v;
  uint16_t* out;
  float* warp_part;   // [blocks][warps][2][Hq / Hkv][piece_floats(d)]: o, m, l of the pieces at a warp range's ends
  float* block_part;  // [blocks][2][Hq / Hkv][piece_floats(d)]: the same for the blocks' ranges
  uint32_t* finished; // [blocks] bytes, zero between calls: finished blocks of the row that begins in a block and leaves it
  float scale;
  int Hq;
};

// A head's piece: o[d], m, l, and zeros up to the next 32 bytes.  Written in whole
// sectors: reading one back that was written in part would wait for memory.
__host__ __device__ constexpr int piece_floats(int d) { return d + 8; }
__device__ __forceinline__ void write_ml(float* dst, float m, float l) {
  reinterpret_cast<float4*>(dst)[0] = make_float4(m, l, 0.0f, 0.0f);
  reinterpret_cast<float4*>(dst)[1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
}

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

// the eight leading bits of a value, and those of two as bf16 (a in the low half)
__device__ __forceinline__ float leading_bits(float x) { return __uint_as_float(__float_as_uint(x) & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_leading(float a, float b) {
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
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
struct KeyPos {
  int j, b, g;         // position in sequence b (-1: no key), kv head
  const float* dt;     // where a listed key's dt lies, else null
};
struct KeyPage {
  int page, off, g;    // table entry, row of the page (-1: no key)
  const float* dt;
};

// What a warp leaves of a row that its range cuts: slot 0 a row that began
// before the range, slot 1 one that begins in it and goes on.
struct RowCut {
  uint32_t t0;       // the row's first tile on the axis
  int nt, b, g;
};

// The axis of U tiles (32 bits hold it: the entry point refuses more) over G
// blocks: the first U % G of them have a tile more than the others.
struct Axis {
  uint32_t per, more, split;   // tiles of a late block; blocks with one more; where the late ones begin
  __device__ __forceinline__ Axis(uint32_t U, uint32_t G) : per(U / G), more(U - U / G * G) { split = more * (per + 1u); }
  __device__ __forceinline__ uint32_t begin(uint32_t block) const { return block * per + min(block, more); }
  __device__ __forceinline__ uint32_t block_of(uint32_t tile) const {
    return tile < split ? tile / (per + 1u) : more + (tile - split) / per;
  }
};

// Joins n pieces of a row for four channels of a head: piece(i) points at
// piece i's o[d], m, l of that head; e is the first channel.  Eight pieces at a
// time, so a block's or a short row's pieces cost one or two latencies.
template <int D, class F>
__device__ __forceinline__ void join_pieces(int n, int e, F&& piece, float& M, float& den, float4& num) {
  constexpr int kAtOnce = 8;
  M = -INFINITY;
  den = 0.0f;
  num = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int i0 = 0; i0 < n; i0 += kAtOnce) {
    float4 o[kAtOnce];
    float2 ml[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      o[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      ml[i] = make_float2(-INFINITY, 0.0f);
      if (i0 + i < n) {
        const float* p = piece(i0 + i);
        o[i] = __ldcg(reinterpret_cast<const float4*>(p + e));
        ml[i] = __ldcg(reinterpret_cast<const float2*>(p + D));
      }
    }
    float N = M;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) N = fmaxf(N, ml[i].x);
    const float f = M == N ? 1.0f : fast_exp2(M - N);
    M = N;
    den *= f;
    num.x *= f;
    num.y *= f;
    num.z *= f;
    num.w *= f;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const float w = ml[i].x == -INFINITY ? 0.0f : fast_exp2(ml[i].x - N);
      den = fmaf(w, ml[i].y, den);
      num.x = fmaf(w, o[i].x, num.x);
      num.y = fmaf(w, o[i].y, num.y);
      num.z = fmaf(w, o[i].z, num.z);
      num.w = fmaf(w, o[i].w, num.w);
    }
  }
}

__device__ __forceinline__ void write_out(uint16_t* out, float den, const float4& num) {
  const float inv = den == 0.0f ? 0.0f : 1.0f / den;
  *reinterpret_cast<uint2*>(out) =
      make_uint2(pack_bf16x2(num.x * inv, num.y * inv), pack_bf16x2(num.z * inv, num.w * inv));
}

// PAIR: a group has one or two query heads.  The eight columns of P then hold its three
// terms at once, term t4 of the two heads in the columns of the quad's lane t4 (every
// lane of a quad computes the same two heads), and o its three sums, joined at a row's
// end: one product per 16 channels instead of three.
template <int D, int W, bool PAIR>
__global__ void __launch_bounds__(DpCfg<D, W>::kThreads, 1) decode_paged_kernel(const __grid_constant__ DpArgs a) {
  using Cfg = DpCfg<D, W>;
  constexpr int kDpWarps = Cfg::kWarps;
  constexpr int KS = D / 16;            // k16 steps of q.k; 16-channel tiles of o
  constexpr int CPR = D / 8;            // 16-byte chunks per row
  constexpr int RPI = 32 / CPR;         // rows per copy step of a warp
  constexpr int STG = Cfg::kStages;
  extern __shared__ __align__(128) unsigned char ring_all[];
  __shared__ RowCut s_cut[kDpWarps][2];
  __shared__ bool s_left[kDpWarps][2];   // the warp left such a piece
  __shared__ int s_last[2];
  const PagedCache& c = a.c;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // ---- the axis: U tiles; G blocks take at least a tile per warp.  Every warp
  // counts for itself, four sequences per lane at a time.
  constexpr int kSeqs = 128;
  uint32_t tiles[4], upto = 0;   // of this lane's sequences of a step; of the step up to and with them
  uint32_t most = 0;             // of any of this lane's sequences
  auto count_step = [&](int b0) {   // returns the step's tiles
    upto = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int b = b0 + 4 * lane + i;
      tiles[i] = b < c.B ? static_cast<uint32_t>(seq_tiles(c, b)) : 0u;
      upto += tiles[i];
      most = max(most, tiles[i]);
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, upto, d);
      if (lane >= d) upto += y;
    }
    return __shfl_sync(0xFFFFFFFFu, upto, 31);
  };
  uint32_t total = 0;
  for (int b0 = 0; b0 < c.B; b0 += kSeqs) total += count_step(b0);
  const uint32_t U = total * static_cast<uint32_t>(c.Hkv);
  // few rows of like lengths: a block takes a row (its part of the axis begins at 0
  // then), and none joins with others.  48 sequences that see 1028 keys of 2 heads of
  // 128 take 18.8 us over equal parts, 16.9 us so; one of 301 keys of 4 heads of 64,
  // 7.2 and 6.6 us; at five tiles a warp instead of kRowSteps both are alike.
  most = __reduce_max_sync(0xFFFFFFFFu, most);
  const uint32_t rows = static_cast<uint32_t>(c.B) * static_cast<uint32_t>(c.Hkv);
  const bool by_row = rows <= gridDim.x && most * gridDim.x <= U + kRowSteps * kDpWarps * gridDim.x;
  const uint32_t G = by_row ? rows : min(gridDim.x, (U + kDpWarps - 1u) / kDpWarps);
  if (blockIdx.x >= G) return;
  const Axis axis(U, G);
  const int hshift = 31 - __clz(c.Hkv);   // (Hkv is a power of two)
  Cursor cur{};
  uint32_t xb0 = 0u, nb = 0u, before = 0u;
  auto warp_begin = [&](uint32_t w) { return xb0 + nb * w / kDpWarps; };
  if (by_row) {
    cur.b = static_cast<int>(blockIdx.x) >> hshift;
  } else {
    xb0 = axis.begin(blockIdx.x);
    nb = axis.begin(blockIdx.x + 1u) - xb0;
    const uint32_t y = warp_begin(warp) >> hshift;   // tiles of sequences before the warp's first one, rounded into it
    for (int b0 = 0; b0 < c.B; b0 += kSeqs) {
      const uint32_t next = c.B > kSeqs ? before + count_step(b0) : total;
      if (y >= next) {
        before = next;
        continue;
      }
      // the lane, then its sequence, whose tiles hold y
      const int from = __popc(__ballot_sync(0xFFFFFFFFu, before + upto <= y));
      cur.b = b0 + 4 * from;
      before += __shfl_sync(0xFFFFFFFFu, upto - tiles[0] - tiles[1] - tiles[2] - tiles[3], from);
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const uint32_t n = __shfl_sync(0xFFFFFFFFu, tiles[i], from);
        if (cur.b == b0 + 4 * from + i && y >= before + n) {
          before += n;
          ++cur.b;
        }
      }
      break;
    }
  }
  cur.enter(c);
  if (by_row) nb = static_cast<uint32_t>(cur.nt);
  const uint32_t xb1 = xb0 + nb, x0 = warp_begin(warp);
  const int count = static_cast<int>(warp_begin(warp + 1) - x0);
  if (by_row) {
    cur.g = static_cast<int>(blockIdx.x) & (c.Hkv - 1);
    cur.t = static_cast<int>(x0);
  } else {
    const uint32_t rem = x0 - before * static_cast<uint32_t>(c.Hkv);
    cur.g = static_cast<int>(rem / static_cast<uint32_t>(cur.nt));
    cur.t = static_cast<int>(rem) - cur.g * cur.nt;
  }
  if (lane < 2) s_left[warp][lane] = false;
  if (tid < 2) s_last[tid] = 0;
  const int nrep = a.Hq / c.Hkv;
  constexpr int PF = piece_floats(D);
  const size_t psize = static_cast<size_t>(nrep) * PF;
  float* my_part = a.warp_part + (static_cast<size_t>(blockIdx.x) * kDpWarps + warp) * 2 * psize;

  // ---- the ring: position -> table entry -> copies of rows and dt, a tile apart
  unsigned char* ring = ring_all + static_cast<size_t>(warp) * STG * Cfg::kStageBytes;
  const uint32_t ring_u = smem_u32(ring);
  const int kl = lane & 15;
  Cursor fc = cur;       // the fetching side's cursor
  int fetched = 0;
  auto position = [&]() {
    KeyPos p{-1, fc.b, fc.g, nullptr};
    if (fetched < count) {
      const int i = fc.t * kTileKeys + kl;
      if (i < fc.keys) {
        if (fc.listed) {
          const size_t at = (static_cast<size_t>(fc.b) * c.Hkv + fc.g) * a.lists.cap + i;
          p.j = a.lists.pos[at];
          p.dt = a.lists.bias + at;
        } else {
          p.j = key_position(c, fc.view, i);
        }
      }
      fc.next(c);
    }
    ++fetched;
    return p;
  };
  auto entry = [&](const KeyPos& p) {
    KeyPage e{0, -1, p.g, p.dt};
    if (p.j >= 0) {
      const int slot = page_slot(c, p.j, e.off);
      e.page = __ldg(c.table + static_cast<size_t>(p.b) * c.max_pages + slot);
    }
    return e;
  };
  const int cr = lane / CPR, cc = lane % CPR;
  auto issue = [&](const KeyPage& k, int slot) {
    const int page = k.off >= 0 ? checked_page(c, k.page) : -1;
    const uint32_t krow = page >= 0 ? row_offset16(c, page, k.off, k.g) : kNoRow;
    const float* dt = page < 0 ? c.dt_pages : k.dt ? k.dt : c.dt_pages + dt_offset(c, page, k.off, k.g);
    const uint32_t st = ring_u + slot * Cfg::kStageBytes;
#pragma unroll
    for (int i = 0; i < kTileKeys / RPI; ++i) {
      const int row = i * RPI + cr;
      const uint32_t off = __shfl_sync(0xFFFFFFFFu, krow, row);
      const bool there = off != kNoRow;
      const size_t e = there ? (static_cast<size_t>(off) + cc) * 8 : 0;
      const uint32_t dst = st + row * Cfg::kRowBytes + ((cc ^ (row & 7)) << 4);
      cp_async16_zfill(dst, a.k + e, there);
      cp_async16_zfill(dst + Cfg::kTileBytes, a.v + e, there);
    }
    if (lane < kTileKeys) {
      *reinterpret_cast<float*>(ring + slot * Cfg::kStageBytes + 2 * Cfg::kTileBytes + 4 * lane) =
          krow != kNoRow ? 0.0f : -INFINITY;
      cp_async4_zfill(st + 2 * Cfg::kTileBytes + 4 * kTileKeys + 4 * lane, dt, krow != kNoRow);
    }
  };
  // the first tiles' positions, then their entries, then their copies: one
  // latency each
  KeyPage next;   // of the tile to be issued next
  KeyPos npos;    // of the one after it
  {
    KeyPos p[STG + 1];
    KeyPage e[STG];
#pragma unroll
    for (int s = 0; s <= STG; ++s) p[s] = position();
#pragma unroll
    for (int s = 0; s < STG; ++s) e[s] = entry(p[s]);
#pragma unroll
    for (int s = 0; s < STG - 1; ++s) {
      if (s < count) issue(e[s], s);
      cp_commit();
    }
    next = e[STG - 1];
    npos = p[STG];
  }

  // ---- the tiles
  const int gid = lane >> 2, t4 = lane & 3;
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
      const int head = PAIR ? gid & 1 : gid;
      const uint16_t* qr = a.q + (static_cast<size_t>(cur.b) * a.Hq + cur.g * nrep + head) * D + 2 * t4;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        qf[s][0] = head < nrep ? __ldg(reinterpret_cast<const uint32_t*>(qr + 16 * s)) : 0u;
        qf[s][1] = head < nrep ? __ldg(reinterpret_cast<const uint32_t*>(qr + 16 * s + 8)) : 0u;
        o[s][0] = o[s][1] = o[s][2] = o[s][3] = 0.0f;
      }
      m0 = m1 = -INFINITY;
      l0 = l1 = 0.0f;
    }
    cp_wait<STG - 2>();
    __syncwarp();   // every lane's copies of this stage have landed; the previous stage has been read
    {
      const int nslot = slot == 0 ? STG - 1 : slot - 1;
      if (x + STG - 1 < count) issue(next, nslot);
      cp_commit();
      next = entry(npos);
      npos = position();
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
    const float b0 = fmaf(bias[kTileKeys + gid], kLog2e, bias[gid]),
                b1 = fmaf(bias[kTileKeys + gid + 8], kLog2e, bias[gid + 8]);   // -inf where there is no key
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
    // P in three terms of eight bits: its leading ones, those of what they leave, and the rest
    // (all differences are exact)
    const float r00 = p00 - leading_bits(p00), r01 = p01 - leading_bits(p01);
    const float r10 = p10 - leading_bits(p10), r11 = p11 - leading_bits(p11);
    const float u00 = r00 - leading_bits(r00), u01 = r01 - leading_bits(r01);
    const float u10 = r10 - leading_bits(r10), u11 = r11 - leading_bits(r11);
    // A tile's sums start at zero, the smallest terms first, and enter o by an addition
    // that rounds to nearest: the tensor core cuts off what it adds to an accumulator, so a
    // chain over a row's tiles loses 2^-24 of the sum each time, always the same way
    // (131072 keys a row: 5e-6 of an output's terms and more)
    const uint32_t sv = st + Cfg::kTileBytes;
    constexpr int kAtOnce = 2;   // independent products in a row: none waits for the one before it
    auto values = [&](auto&& products) {
#pragma unroll
      for (int s0 = 0; s0 < KS; s0 += kAtOnce) {
        uint32_t va[kAtOnce][4];
        float t[kAtOnce][4];
#pragma unroll
        for (int s = 0; s < kAtOnce; ++s) {
          ldsm4_t(va[s], sv + v_row * Cfg::kRowBytes + (((2 * (s0 + s) + v_par) ^ (v_row & 7)) << 4));
          t[s][0] = t[s][1] = t[s][2] = t[s][3] = 0.0f;
        }
        products(t, va);
#pragma unroll
        for (int s = 0; s < kAtOnce; ++s)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[s0 + s][i] += t[s][i];
      }
    };
    auto term = [&](float (&t)[kAtOnce][4], const uint32_t (&va)[kAtOnce][4], uint32_t p0, uint32_t p1) {
#pragma unroll
      for (int s = 0; s < kAtOnce; ++s) mma16816(t[s], va[s], p0, p1);
    };
    if constexpr (PAIR) {
      auto mine = [&](float p, float r, float u) { return t4 == 0 ? p : t4 == 1 ? r : t4 == 2 ? u : 0.0f; };
      const uint32_t pm0 = transpose8x8(pack_leading(mine(p00, r00, u00), mine(p01, r01, u01)));
      const uint32_t pm1 = transpose8x8(pack_leading(mine(p10, r10, u10), mine(p11, r11, u11)));
      values([&](auto& t, const auto& va) { term(t, va, pm0, pm1); });
    } else {
      const uint32_t ph0 = transpose8x8(pack_leading(p00, p01)), ph1 = transpose8x8(pack_leading(p10, p11));
      const uint32_t pe0 = transpose8x8(pack_leading(r00, r01)), pe1 = transpose8x8(pack_leading(r10, r11));
      const uint32_t pf0 = transpose8x8(pack_leading(u00, u01)), pf1 = transpose8x8(pack_leading(u10, u11));
      values([&](auto& t, const auto& va) {
        term(t, va, pf0, pf1);
        term(t, va, pe0, pe1);
        term(t, va, ph0, ph1);
      });
    }
    const int used = slot;
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
      // through the stage just read (its K rows' place), so that rows of o leave in
      // whole 128-byte lines: written from the accumulators as they lie, four bytes a
      // lane, a block's pieces took 1 to 2 us
      float* turn = reinterpret_cast<float*>(ring + used * Cfg::kStageBytes);   // [head][d]; PAIR: [term][2][d]
      constexpr int kTerm = 2 * D + 8;   // floats between terms: the quad's lanes write to other banks
      const bool wa = PAIR ? t4 < 3 : ha < nrep, wb = PAIR ? t4 < 3 && nrep == 2 : hb < nrep;
      float *ta = turn + (PAIR ? t4 * kTerm : ha * D) + gid, *tb = ta + D;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        if (wa) {
          ta[16 * s] = o[s][0];
          ta[16 * s + 8] = o[s][2];
        }
        if (wb) {
          tb[16 * s] = o[s][1];
          tb[16 * s + 8] = o[s][3];
        }
      }
      __syncwarp();
      static_assert(3 * kTerm * 4 <= Cfg::kTileBytes, "the terms fit the K rows' place");
      auto sums = [&](int e) {
        float4 x = *reinterpret_cast<const float4*>(turn + e);
        if constexpr (PAIR) {
          const float4 y = *reinterpret_cast<const float4*>(turn + kTerm + e);
          const float4 z = *reinterpret_cast<const float4*>(turn + 2 * kTerm + e);
          x = make_float4(x.x + (y.x + z.x), x.y + (y.y + z.y), x.z + (y.z + z.z), x.w + (y.w + z.w));
        }
        return x;
      };
      if (row_end && from_start) {
        uint16_t* dst = a.out + (static_cast<size_t>(cur.b) * a.Hq + cur.g * nrep) * D;
        for (int e = 4 * lane; e < (nrep * D + 127) / 128 * 128; e += 128) {   // the whole warp shuffles
          const int h = e / D;
          const float la = __shfl_sync(0xFFFFFFFFu, L0, h >> 1 & 3), lb = __shfl_sync(0xFFFFFFFFu, L1, h >> 1 & 3);
          if (h < nrep) write_out(dst + e, h & 1 ? lb : la, sums(e));
        }
      } else {
        // slot 0: the row began before this range; slot 1: it begins here and goes on
        const int cut = from_start ? 1 : 0;
        float* dst = my_part + cut * psize;
        for (int e = 4 * lane; e < nrep * D; e += 128)
          *reinterpret_cast<float4*>(dst + e / D * PF + e % D) = sums(e);
        if (gid == 0 && ha < nrep) write_ml(dst + ha * PF + D, m0, L0);
        if (gid == 0 && hb < nrep) write_ml(dst + hb * PF + D, m1, L1);
        if (lane == 0) {
          s_left[warp][cut] = true;
          s_cut[warp][cut] = RowCut{x0 + static_cast<uint32_t>(x) - static_cast<uint32_t>(cur.t), cur.nt, cur.b, cur.g};
        }
      }
      fresh = true;
      __syncwarp();   // the stage is free again
    }
    cur.next(c);
  }
  cp_wait<0>();
  __syncthreads();   // every warp's pieces are written

  // ---- the block's pieces, row by row.  Chain w < kDpWarps: the row that begins
  // in warp w and leaves its range; chain kDpWarps: the row that began before the
  // block.  Lane w finds chain w; the warps share out (chain, 128 channels of its
  // heads).
  const float* warp_part = a.warp_part + static_cast<size_t>(blockIdx.x) * kDpWarps * 2 * psize;
  float* my_block = a.block_part + static_cast<size_t>(blockIdx.x) * 2 * psize;
  const int parts = (nrep * D + 127) / 128;
  const uint32_t busy = __ballot_sync(0xFFFFFFFFu, lane < kDpWarps && warp_begin(lane + 1) != warp_begin(lane));   // warps with tiles
  const int first = __ffs(static_cast<int>(busy)) - 1;
  RowCut cut{};
  int w0 = 0, w1 = 0;      // the chain's warps
  bool right = false;      // it goes on past the block
  const bool mine = lane < kDpWarps ? s_left[lane][1] : lane == kDpWarps && s_left[first][0];
  if (mine) {
    w0 = lane < kDpWarps ? lane : first;
    cut = s_cut[w0][lane < kDpWarps ? 1 : 0];
    const uint32_t end = min(cut.t0 + static_cast<uint32_t>(cut.nt), xb1);
    w1 = static_cast<int>(((end - xb0) * kDpWarps - 1u) / nb);   // the warp of its last tile here
    right = cut.t0 + static_cast<uint32_t>(cut.nt) > xb1;
  }
  const uint32_t chains = __ballot_sync(0xFFFFFFFFu, mine), opens = __ballot_sync(0xFFFFFFFFu, right);
  const bool left = chains >> kDpWarps & 1u;
  for (int it = warp; it < __popc(chains) * parts; it += kDpWarps) {
    uint32_t rest = chains;
    for (int i = it / parts; i > 0; --i) rest &= rest - 1u;
    const int w = __ffs(static_cast<int>(rest)) - 1;
    const int c0 = __shfl_sync(0xFFFFFFFFu, w0, w), c1 = __shfl_sync(0xFFFFFFFFu, w1, w);
    const int cb = __shfl_sync(0xFFFFFFFFu, cut.b, w), cg = __shfl_sync(0xFFFFFFFFu, cut.g, w);
    const int e = it % parts * 128 + 4 * lane, h = e / D;
    if (h >= nrep) continue;
    uint32_t todo = busy & (0xFFFFFFFFu << c0) & (0xFFFFFFFFu >> (31 - c1));   // its warps that have tiles
    const int n = __popc(todo);
    const float* base = warp_part + static_cast<size_t>(h) * PF;
    float M, den;
    float4 num;
    join_pieces<D>(
        n, e % D,
        [&](int i) {
          const int from = __ffs(static_cast<int>(todo)) - 1;
          todo &= todo - 1u;
          return base + (2 * from + (i == 0 && w < kDpWarps ? 1 : 0)) * psize;
        },
        M, den, num);
    if (w < kDpWarps && !(opens >> w & 1u)) {
      write_out(a.out + (static_cast<size_t>(cb) * a.Hq + cg * nrep + h) * D + e % D, den, num);
    } else {
      float* dst = my_block + (w < kDpWarps ? psize : 0) + static_cast<size_t>(h) * PF;
      *reinterpret_cast<float4*>(dst + e % D) = num;
      if (e % D == 0) write_ml(dst + D, M, den);
    }
  }

  // ---- rows shared with other blocks: the one that finishes such a row's last
  // piece joins them
  const uint32_t here = opens & ((1u << kDpWarps) - 1u);   // a row that goes on and began here (else it is the left one)
  const bool two = here != 0u;
  if (!left && !two) return;
  auto row_blocks = [&](int k, uint32_t& b0, uint32_t& b1) {
    const RowCut r = k == 0 ? s_cut[first][0] : s_cut[__ffs(static_cast<int>(here)) - 1][1];
    b0 = axis.block_of(r.t0);
    b1 = axis.block_of(r.t0 + static_cast<uint32_t>(r.nt) - 1u);
    return r;
  };
  __syncthreads();
  if (lane == 0 && warp < 2 && (warp == 0 ? left : two)) {
    uint32_t b0, b1;
    row_blocks(warp, b0, b1);
    // releases this block's pieces (written before the barrier) and acquires the others'
    const uint32_t one = 1u << (8u * (b0 & 3u));
    uint32_t* word = a.finished + (b0 >> 2);
    uint32_t before;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;" : "=r"(before) : "l"(word), "r"(one) : "memory");
    if ((before / one & 255u) == b1 - b0) {
      atomicSub(word, (b1 - b0 + 1u) * one);
      s_last[warp] = 1;
    }
  }
  __syncthreads();
  for (int k = 0; k < 2; ++k) {
    if (!s_last[k]) continue;
    uint32_t b0, b1;
    const RowCut r = row_blocks(k, b0, b1);
    for (int q = warp; q < parts; q += kDpWarps) {
      const int e = q * 128 + 4 * lane, h = e / D;
      if (h >= nrep) continue;
      const float* base = a.block_part + static_cast<size_t>(b0) * 2 * psize + static_cast<size_t>(h) * PF;
      float M, den;
      float4 num;
      join_pieces<D>(
          static_cast<int>(b1 - b0) + 1, e % D, [&](int i) { return base + (i == 0 ? 1 : 2 * i) * psize; }, M, den, num);
      write_out(a.out + (static_cast<size_t>(r.b) * a.Hq + r.g * nrep + h) * D + e % D, den, num);
    }
  }
}

template <int D, int W>
cudaError_t launch_dp(const DpArgs& a, int blocks, cudaStream_t s) {
  using Cfg = DpCfg<D, W>;
  auto* kernel = a.Hq <= 2 * a.c.Hkv ? decode_paged_kernel<D, W, true> : decode_paged_kernel<D, W, false>;
  const cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(kernel), Cfg::kSmemBytes);
  if (e != cudaSuccess) return e;
  return launch_after(kernel, dim3(blocks), dim3(Cfg::kThreads), Cfg::kSmemBytes, s, a);
}

}  // namespace

cudaError_t launch_attn_paged(const PagedCache& c, const PagedLists& lists, const void* q, const void* k_pages,
                              const void* v_pages, int Hq, float scale, void* scratch, void* out, cudaStream_t s) {
  const int nsm = sm_count();
  if (nsm <= 0) return cudaErrorInvalidDevice;
  const size_t psize = static_cast<size_t>(Hq / c.Hkv) * piece_floats(c.d);
  DpArgs a;
  a.c = c;
  a.lists = lists;
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k_pages);
  a.v = static_cast<const uint16_t*>(v_pages);
  a.out = static_cast<uint16_t*>(out);
  a.finished = c.err + kHdrRowWord;
  a.block_part = static_cast<float*>(scratch);
  a.warp_part = a.block_part + kPagedMaxBlocks * 2 * psize;
  a.scale = scale;
  a.Hq = Hq;
  const int blocks = std::min(nsm, kPagedMaxBlocks);
  if (c.d == 128) return launch_dp<128, 8>(a, blocks, s);
  // d = 64: sixteen warps keep more scattered rows on their way (64 sequences with
  // lists of 2048 on 8 heads, selection included: 121 us, eight warps 145 us; 16 of 500
  // to 700 keys on 4 heads: 9.5 and 10.4 us); eight start and join sooner, which counts
  // while there are few and short rows (one sequence of 301 keys, 4 heads: 7.5 and 6.7 us;
  // of 2048: 9.6 and 8.6 us; of 4096: 10.2 and 9.8 us; of 32k: 15.9 and 16.4 us; of 512k: 94
  // and 115 us; two of 301 keys: 7.7 and 6.8 us, of 131k: 54 and 62 us)
  const bool few = lists.cap == 0 && 4 * c.B * c.Hkv <= nsm && c.longest <= kFewWarpsLength;
  return few ? launch_dp<64, 8>(a, blocks, s) : launch_dp<64, 16>(a, blocks, s);
}

size_t attn_paged_scratch_bytes(int Hq, int Hkv, int d) {
  return static_cast<size_t>(kPagedMaxBlocks) * (1 + kDpMaxWarps) * 2 * (Hq / Hkv) * piece_floats(d) * sizeof(float);
}

}  // namespace dma
