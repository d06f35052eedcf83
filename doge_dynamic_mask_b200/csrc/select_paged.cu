// Selection of the decode step over a paged cache: the kept keys of rows longer than the kept window.
//
// Method: page "Transformers 中的 Doge 小语言模型完全指南", section
// "动态掩码注意力（DMA）：从缓存 value states 生成稀疏掩码", step 3
// (prepare_dynamic_mask: of the keys a query sees, the keep_window_size best by
// dt; ties go to the lower index).  dt of every cached token lies in its page.
//
// Design.  One cluster of CTAs per (sequence, kv head).  The row is read once:
// a sample of 4096 keys (1024 quads spread over the row) gives a threshold that
// the w-th best key is above with four standard deviations to spare, every
// warp collects the keys at or above it from 128-key chunks dealt out in turn,
// and the collected keys (about 1.4 w at 64k keys) are cut to the w best: a
// histogram over the cluster finds the bin of the w-th, keys above the bin are
// kept, and the few keys inside are ranked one against another by (dt, index).
// The bound is the one read of dt plus the latency of those steps; a row is
// spread over up to eight CTAs when there are fewer rows than SMs.  Rows the
// sample misjudges (more ties at the threshold than the buffers hold, too few
// keys) are selected exactly by the cluster's first CTA in a few more passes.
// The order of the list is fixed by the row alone (chunk dealing, then rank),
// so the attention adds its terms in the same order every time.
#include <cooperative_groups.h>

#include "paged.cuh"
#include "select_common.cuh"

namespace dma {
namespace {

namespace cg = cooperative_groups;

constexpr int kSpThreads = 256;
constexpr int kSpWarps = kSpThreads / 32;
constexpr int kSpMinBlocks = 3;
constexpr int kSpRegion = 768;           // collected keys per warp
constexpr int kSpSampleQuads = 1024;
constexpr int kSpEdge = 1024;            // keys inside the w-th key's bin
constexpr int kSpChunks = 4;             // 128-key chunks in flight per warp

struct SpSmem {
  uint64_t keys[kSpWarps][kSpRegion];    // collected keys; first the sample
  uint64_t edge[kSpEdge];                // (first CTA) keys inside the w-th key's bin
  uint32_t hist[kBins];
  uint64_t vars[8];
  uint32_t red[64];
  uint32_t count[kSpWarps];              // collected per warp, then kept per warp
  uint32_t stat[8];                      // cluster exchange, see the uses
};

// A row's visible keys as quads of four positions (16 bytes of dt when the
// page size is a multiple of four): quads [0, nqa) cover the sinks, the rest the
// positions from `start` on.
struct Row {
  int b, g, sinks, start, len, nqa, nq, qb;
};

__device__ __forceinline__ Row make_row(const PagedCache& c, const SeqView& v, int b, int g) {
  Row r;
  r.b = b;
  r.g = g;
  r.len = v.len;
  r.sinks = v.shift > 0 ? c.sinks : 0;
  r.start = v.shift > 0 ? c.sinks + v.shift : 0;
  r.nqa = (r.sinks + 3) >> 2;
  r.qb = r.start >> 2;
  r.nq = r.nqa + ((r.len + 3) >> 2) - r.qb;
  return r;
}

__device__ __forceinline__ int quad_position(const Row& r, int x) { return 4 * (x < r.nqa ? x : x - r.nqa + r.qb); }

__device__ __forceinline__ bool quad_sees(const Row& r, int x, int j) {
  return x < r.nqa ? j < r.sinks : (j >= r.start && j < r.len);
}

// The quad's table entry (page size a multiple of four): x in [0, nq).
__device__ __forceinline__ int quad_page(const PagedCache& c, const Row& r, int x) {
  int off;
  const int slot = page_slot(c, quad_position(r, x), off);
  return __ldg(c.table + static_cast<size_t>(r.b) * c.max_pages + slot);
}

// dt bits of a quad and which of its positions are seen (bit e of the result)
__device__ __forceinline__ uint32_t load_quad(const PagedCache& c, const Row& r, int x, int page, uint32_t (&v)[4]) {
  const int j0 = quad_position(r, x);
  uint32_t seen = 0;
  if ((c.page_size & 3) == 0) {
    int off;
    page_slot(c, j0, off);
    page = checked_page(c, page);
    if (page < 0) return 0;
    const uint4 q = __ldg(reinterpret_cast<const uint4*>(c.dt_pages + dt_offset(c, page, off, r.g)));
    v[0] = q.x;
    v[1] = q.y;
    v[2] = q.z;
    v[3] = q.w;
#pragma unroll
    for (int e = 0; e < 4; ++e) seen |= quad_sees(r, x, j0 + e) ? 1u << e : 0u;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = 0;
      if (!quad_sees(r, x, j0 + e)) continue;
      int off;
      const int slot = page_slot(c, j0 + e, off);
      const int pg = checked_page(c, __ldg(c.table + static_cast<size_t>(r.b) * c.max_pages + slot));
      if (pg < 0) continue;
      v[e] = __float_as_uint(__ldg(c.dt_pages + dt_offset(c, pg, off, r.g)));
      seen |= 1u << e;
    }
  }
  return seen;
}

// page of a quad where one entry covers it (else looked up per position)
__device__ __forceinline__ int quad_page_or_none(const PagedCache& c, const Row& r, int x) {
  return (c.page_size & 3) == 0 && x < r.nq ? quad_page(c, r, x) : 0;
}

__device__ __forceinline__ void write_entry(const PagedCache& c, const PagedLists& o, size_t at, const Row& r, uint64_t key) {
  const int j = static_cast<int>(composite_index(key));
  int off;
  const int slot = page_slot(c, j, off);
  const int page = __ldg(c.table + static_cast<size_t>(r.b) * c.max_pages + slot);   // checked when it was collected
  o.row[at] = row_offset16(c, page, off, r.g);
  o.bias[at] = __uint_as_float(static_cast<uint32_t>(key >> 32));
}

// Smallest shift that maps [0, range] into 2048 bins.
__device__ __forceinline__ int bin_shift(uint32_t range) {
  const int top = 32 - __clz(static_cast<int>(range | 1u));   // bits in use
  return top > 11 ? top - 11 : 0;
}

// Exact selection by one CTA: a few histogram passes over the row narrow the
// dt bits of the w-th key to one value, then two passes write the keys above
// it and the lowest-indexed ones equal to it.  Each warp owns a contiguous part
// of the row, so the list is in a fixed order.
static __device__ __noinline__ void select_exact(const PagedCache& c, const PagedLists& o, const Row& r, int w,
                                                 SpSmem& sm) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int seg = ((r.nq + kSpWarps - 1) / kSpWarps + 31) / 32 * 32;
  const int x0 = min(r.nq, warp * seg), x1 = min(r.nq, x0 + seg);
  const size_t base = (static_cast<size_t>(r.b) * c.Hkv + r.g) * o.cap;
  auto each = [&](auto&& f) {   // f(quad, bits, seen): the whole warp calls it together
    for (int q0 = x0; q0 < x1; q0 += 32) {
      const int x = q0 + lane;
      uint32_t v[4] = {0u, 0u, 0u, 0u};
      const uint32_t seen = x < x1 ? load_quad(c, r, x, quad_page_or_none(c, r, x), v) : 0u;
      f(x, v, seen);
    }
  };
  if (tid < 4) sm.stat[tid] = tid == 1 ? 0xFFFFFFFFu : 0u;   // [count, min, max]
  __syncthreads();
  {
    uint32_t n = 0, lo = 0xFFFFFFFFu, hi = 0u;
    each([&](int, const uint32_t(&v)[4], uint32_t seen) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (seen >> e & 1u) {
          ++n;
          lo = min(lo, v[e]);
          hi = max(hi, v[e]);
        }
    });
    n = __reduce_add_sync(0xFFFFFFFFu, n);
    lo = __reduce_min_sync(0xFFFFFFFFu, lo);
    hi = __reduce_max_sync(0xFFFFFFFFu, hi);
    if (lane == 0) {
      atomicAdd(&sm.stat[0], n);
      atomicMin(&sm.stat[1], lo);
      atomicMax(&sm.stat[2], hi);
    }
  }
  __syncthreads();
  const uint32_t total = sm.stat[0];
  uint32_t lo = sm.stat[1], hi = sm.stat[2];
  uint32_t k = static_cast<uint32_t>(w);   // keys to keep of those in [lo, hi]
  if (total > static_cast<uint32_t>(w)) {
    while (lo < hi) {
      const int s = bin_shift(hi - lo);
      for (int i = tid; i < kBins; i += kSpThreads) sm.hist[i] = 0;
      __syncthreads();
      each([&](int, const uint32_t(&v)[4], uint32_t seen) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if ((seen >> e & 1u) && v[e] >= lo && v[e] <= hi) atomicAdd(&sm.hist[(v[e] - lo) >> s], 1u);
      });
      __syncthreads();
      uint32_t kin, cnt;
      const uint32_t bin = find_bin_from_top(sm.hist, kBins, k, sm.red, sm.vars, &kin, &cnt);
      k = kin;
      const uint32_t l2 = lo + (bin << s);
      hi = min(hi, l2 + ((1u << s) - 1u));
      lo = l2;
    }
  } else {
    // pages outside the pool left no more than w keys: all of them are kept
    k = total;
    lo = 0u;
  }
  // the keys above lo, then the k lowest-indexed ones equal to it
  uint32_t gt = 0, eq = 0;
  each([&](int, const uint32_t(&v)[4], uint32_t seen) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      gt += (seen >> e & 1u) && v[e] > lo;
      eq += (seen >> e & 1u) && v[e] == lo;
    }
  });
  gt = __reduce_add_sync(0xFFFFFFFFu, gt);
  eq = __reduce_add_sync(0xFFFFFFFFu, eq);
  if (lane == 0) {
    sm.red[warp] = gt;
    sm.red[16 + warp] = eq;
  }
  __syncthreads();
  uint32_t gpos = 0, epos = 0, gall = 0;
  for (int i = 0; i < kSpWarps; ++i) {
    if (i < warp) {
      gpos += sm.red[i];
      epos += sm.red[16 + i];
    }
    gall += sm.red[i];
  }
  const uint32_t lt = lanemask_lt();
  each([&](int x, const uint32_t(&v)[4], uint32_t seen) {
    const int j0 = x < r.nq ? quad_position(r, x) : 0;
    uint32_t n = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) n += (seen >> e & 1u) && v[e] == lo;
    // this lane's first equal key's rank: prefix of n (0..4) over the lanes
    const uint32_t b0 = __ballot_sync(0xFFFFFFFFu, n & 1u), b1 = __ballot_sync(0xFFFFFFFFu, n & 2u),
                   b2 = __ballot_sync(0xFFFFFFFFu, n & 4u);
    uint32_t er = epos + __popc(b0 & lt) + 2u * __popc(b1 & lt) + 4u * __popc(b2 & lt);
    epos += __popc(b0) + 2u * __popc(b1) + 4u * __popc(b2);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool above = (seen >> e & 1u) && v[e] > lo;
      const uint32_t vote = __ballot_sync(0xFFFFFFFFu, above);
      if (above) write_entry(c, o, base + gpos + __popc(vote & lt), r, composite_key(v[e], j0 + e));
      gpos += __popc(vote);
      if ((seen >> e & 1u) && v[e] == lo) {
        if (er < k) write_entry(c, o, base + gall + er, r, composite_key(v[e], j0 + e));
        ++er;
      }
    }
  });
  // entries that pages outside the pool left empty
  for (int e = static_cast<int>(min(total, static_cast<uint32_t>(w))) + tid; e < w; e += kSpThreads) {
    o.row[base + e] = kNoRow;
    o.bias[base + e] = 0.0f;
  }
}

__global__ void __launch_bounds__(kSpThreads, kSpMinBlocks)
    select_paged_kernel(const __grid_constant__ PagedCache c, const __grid_constant__ PagedLists o) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  SpSmem& sm = *reinterpret_cast<SpSmem*>(smem_raw);
  cg::cluster_group cluster = cg::this_cluster();
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int csize = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int bg = blockIdx.x / csize;
  const int b = bg / c.Hkv, g = bg % c.Hkv;
  const int w = c.w;
  const SeqView view = seq_view(c, b);
  if (view.n <= w) return;   // the attention takes such a row as it is (the whole cluster returns)
  const Row r = make_row(c, view, b, g);
  const size_t base = static_cast<size_t>(bg) * o.cap;

  // ---- the sample and its threshold (every CTA of the cluster finds the same)
  uint32_t* sample = reinterpret_cast<uint32_t*>(sm.keys);
  const int squads = min(kSpSampleQuads, r.nq);
  if (tid < 8) sm.stat[tid] = tid == 1 ? 0xFFFFFFFFu : 0u;   // [sampled, min, max, ...]
  __syncthreads();
  {
    constexpr int kPer = kSpSampleQuads / kSpThreads;
    int page[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int s = i * kSpThreads + tid;
      page[i] = s < squads ? quad_page_or_none(c, r, static_cast<int>(static_cast<long long>(s) * r.nq / squads)) : 0;
    }
    uint32_t n = 0, lo = 0xFFFFFFFFu, hi = 0u;
    uint32_t v[kPer][4], seen[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int s = i * kSpThreads + tid;
      seen[i] = s < squads ? load_quad(c, r, static_cast<int>(static_cast<long long>(s) * r.nq / squads), page[i], v[i])
                           : 0u;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int s = i * kSpThreads + tid;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool ok = seen[i] >> e & 1u;
        if (s < squads) sample[4 * s + e] = ok ? v[i][e] : 0u;
        if (ok) {
          ++n;
          lo = min(lo, v[i][e]);
          hi = max(hi, v[i][e]);
        }
      }
    }
    n = __reduce_add_sync(0xFFFFFFFFu, n);
    lo = __reduce_min_sync(0xFFFFFFFFu, lo);
    hi = __reduce_max_sync(0xFFFFFFFFu, hi);
    if (lane == 0) {
      atomicAdd(&sm.stat[0], n);
      atomicMin(&sm.stat[1], lo);
      atomicMax(&sm.stat[2], hi);
    }
  }
  __syncthreads();
  const uint32_t ns = sm.stat[0], smax = sm.stat[2];
  uint32_t thr = sm.stat[1];
  // the sample's rank that the w-th key of the row lies above but for one row in many thousands
  const float expect = static_cast<float>(w) * static_cast<float>(ns) / static_cast<float>(view.n);
  uint32_t k = static_cast<uint32_t>(expect + 4.0f * sqrtf(expect) + 5.0f);
  if (k < ns) {
    uint32_t lo = thr, hi = smax;
    while (lo < hi) {
      const int s = bin_shift(hi - lo);
      for (int i = tid; i < kBins; i += kSpThreads) sm.hist[i] = 0;
      __syncthreads();
      for (int i = tid; i < 4 * squads; i += kSpThreads) {
        const uint32_t x = sample[i];   // unseen places hold 0: below lo, or the lowest value there is
        if (x >= lo && x <= hi) atomicAdd(&sm.hist[(x - lo) >> s], 1u);
      }
      __syncthreads();
      uint32_t kin, cnt;
      const uint32_t bin = find_bin_from_top(sm.hist, kBins, k, sm.red, sm.vars, &kin, &cnt);
      k = kin;
      const uint32_t l2 = lo + (bin << s);
      hi = min(hi, l2 + ((1u << s) - 1u));
      lo = l2;
      if (cnt <= 16u) break;   // its lower edge takes a few more keys than the exact value would
    }
    thr = lo;
  }
  __syncthreads();   // the sample is read before keys are collected over it

  // ---- collect: 128-key chunks dealt to the cluster's warps in turn
  uint32_t n_mine = 0;
  uint64_t* mine = sm.keys[warp];
  {
    const int nchunk = (r.nq + 31) / 32, step = csize * kSpWarps;
    const uint32_t lt = lanemask_lt();
    int page[kSpChunks];
    const int first = rank * kSpWarps + warp;
#pragma unroll
    for (int u = 0; u < kSpChunks; ++u) page[u] = quad_page_or_none(c, r, (first + u * step) * 32 + lane);
    for (int c0 = first; c0 < nchunk; c0 += kSpChunks * step) {
      uint32_t v[kSpChunks][4], seen[kSpChunks];
#pragma unroll
      for (int u = 0; u < kSpChunks; ++u) {
        const int x = (c0 + u * step) * 32 + lane;
        seen[u] = x < r.nq ? load_quad(c, r, x, page[u], v[u]) : 0u;
      }
#pragma unroll
      for (int u = 0; u < kSpChunks; ++u)
        page[u] = quad_page_or_none(c, r, (c0 + (kSpChunks + u) * step) * 32 + lane);
#pragma unroll
      for (int u = 0; u < kSpChunks; ++u) {
        const int x = (c0 + u * step) * 32 + lane;
        const int j0 = x < r.nq ? quad_position(r, x) : 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool take = (seen[u] >> e & 1u) && v[u][e] >= thr;
          const uint32_t vote = __ballot_sync(0xFFFFFFFFu, take);
          const uint32_t pos = n_mine + __popc(vote & lt);
          if (take && pos < static_cast<uint32_t>(kSpRegion)) mine[pos] = composite_key(v[u][e], j0 + e);
          n_mine += __popc(vote);
        }
      }
    }
  }
  // ---- the w-th key's bin, over the cluster
  const int shift = bin_shift(smax > thr ? smax - thr : 0u);
  auto bin_of = [&](uint64_t key) {
    return min(static_cast<uint32_t>(kBins - 1), (static_cast<uint32_t>(key >> 32) - thr) >> shift);
  };
  for (int i = tid; i < kBins; i += kSpThreads) sm.hist[i] = 0;
  if (tid < 8) sm.stat[tid] = 0u;   // [0] overflow, [1] sure keys of this CTA, first CTA: [2] bin, [3] needed in it, [4] edge keys, [5] exact
  __syncthreads();
  if (lane == 0) {
    sm.count[warp] = n_mine;
    if (n_mine > static_cast<uint32_t>(kSpRegion)) sm.stat[0] = 1u;
  }
  for (uint32_t i = lane; i < min(n_mine, static_cast<uint32_t>(kSpRegion)); i += 32)
    atomicAdd(&sm.hist[bin_of(mine[i])], 1u);
  cluster.sync();
  SpSmem* lead = cluster.map_shared_rank(&sm, 0);
  if (rank == 0) {
    uint32_t bad = sm.stat[0];
    for (int q = 1; q < csize; ++q) {
      SpSmem* other = cluster.map_shared_rank(&sm, q);
      bad |= other->stat[0];
      for (int i = tid; i < kBins; i += kSpThreads) sm.hist[i] += other->hist[i];
    }
    uint32_t mysum = 0;
    for (int i = tid; i < kBins; i += kSpThreads) mysum += sm.hist[i];
    uint32_t total;
    block_exclusive_scan(mysum, sm.red, &total);
    bad |= total < static_cast<uint32_t>(w);
    if (!bad) {
      uint32_t kin, cnt;
      const uint32_t bin = find_bin_from_top(sm.hist, kBins, static_cast<uint32_t>(w), sm.red, sm.vars, &kin, &cnt);
      bad = cnt > static_cast<uint32_t>(kSpEdge);
      if (tid == 0) {
        sm.stat[2] = bin;
        sm.stat[3] = kin;
      }
    }
    if (tid == 0) sm.stat[5] = bad;
  }
  cluster.sync();
  const uint32_t bad = lead->stat[5], wbin = lead->stat[2], need = lead->stat[3];
  uint32_t sure = 0;
  if (!bad) {
    // keys inside the bin go to the first CTA (they are ranked by value, so
    // their order there does not matter); keys above it are counted
    for (uint32_t i = lane; i < n_mine; i += 32) {
      const uint64_t key = mine[i];
      const uint32_t bin = bin_of(key);
      sure += bin > wbin;
      if (bin == wbin) lead->edge[atomicAdd(&lead->stat[4], 1u)] = key;
    }
    sure = __reduce_add_sync(0xFFFFFFFFu, sure);
    if (lane == 0) {
      sm.count[warp] = sure;
      atomicAdd(&sm.stat[1], sure);
    }
  }
  cluster.sync();
  if (!bad) {
    uint32_t pos = 0;
    for (int q = 0; q < rank; ++q) pos += cluster.map_shared_rank(&sm, q)->stat[1];
    for (int i = 0; i < warp; ++i) pos += sm.count[i];
    const uint32_t lt = lanemask_lt();
    for (uint32_t i0 = 0; i0 < n_mine; i0 += 32) {
      const uint32_t i = i0 + lane;
      const uint64_t key = i < n_mine ? mine[i] : 0ull;
      const bool keep = i < n_mine && bin_of(key) > wbin;
      const uint32_t vote = __ballot_sync(0xFFFFFFFFu, keep);
      if (keep) write_entry(c, o, base + pos + __popc(vote & lt), r, key);
      pos += __popc(vote);
    }
    if (rank == 0) {
      // the bin's `need` best keys, each at its rank
      const uint32_t ne = sm.stat[4];
      for (uint32_t i = tid; i < ne; i += kSpThreads) {
        const uint64_t key = sm.edge[i];
        uint32_t above = 0;
        for (uint32_t q = 0; q < ne; ++q) above += sm.edge[q] > key;
        if (above < need) write_entry(c, o, base + (w - need) + above, r, key);
      }
    }
  }
  cluster.sync();   // no CTA leaves while another reads its shared memory
  if (bad && rank == 0) select_exact(c, o, r, w, sm);
}

}  // namespace

cudaError_t launch_select_paged(const PagedCache& c, const PagedLists& lists, cudaStream_t s) {
  constexpr int smem = static_cast<int>(sizeof(SpSmem));
  cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(select_paged_kernel), smem);
  if (e != cudaSuccess) return e;
  const int nsm = sm_count();
  if (nsm <= 0) return cudaErrorInvalidDevice;
  const int rows = c.B * c.Hkv;
  // CTAs per row: while they fit on the SMs at once and each has 4096 keys of the
  // longest row the table can hold
  const long long keys = static_cast<long long>(c.max_pages) * c.page_size;
  int csize = 1;
  while (csize < 8 && 2LL * csize * rows <= static_cast<long long>(kSpMinBlocks) * nsm && keys >= 4096LL * 2 * csize)
    csize *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows) * csize);
  cfg.blockDim = dim3(kSpThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = csize;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, select_paged_kernel, c, lists);
}

}  // namespace dma
