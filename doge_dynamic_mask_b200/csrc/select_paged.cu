// Selection of the decode step over a paged cache: the kept keys of rows longer than the kept window.
//
// Method: page "Transformers 中的 Doge 小语言模型完全指南", section
// "动态掩码注意力（DMA）：从缓存 value states 生成稀疏掩码", step 3
// (prepare_dynamic_mask: of the keys a query sees, the keep_window_size best by
// dt; ties go to the lower index).  dt of every cached token lies in its page.
//
// Design.  One CTA, or a cluster of them, per (sequence, kv head).  The row is
// read once: a sample (2048 keys, of long rows 4096, in runs of eight spread over
// the row) gives a threshold that the w-th best key is above with four standard
// deviations to spare, and every thread appends the keys at or above it that it
// meets (about 1.6 w in all at 64k keys) to a list of its own in shared memory,
// by predicated instructions without votes or branches; the few keys that find
// their list full spill to a list of the CTA.  A histogram of the collected keys
// over the cluster finds the w-th key's bin; keys above the bin are kept, and the
// few inside are ranked one against another by (dt, index).  When one value takes
// many places of the sample around the threshold (a model at its start has dt = 1
// everywhere) only the keys above it are collected, and the lowest-indexed ones
// of that value fill the list.  Rows the sample misjudges (too few keys, too many
// in one bin) are selected exactly by the cluster's first CTA in a few more
// passes.  The order of the list is fixed by the row alone, so the attention adds
// its terms in the same order every time.
//
// What bounds it: the latency and the integer instructions of its steps rather
// than the one read of dt.  512 rows of 32k to 64k keys, w = 2048: about 58 us for
// 100 MB (16 us at the copy rate); in cycles of a CTA of 512 threads, two CTAs an
// SM: sample 6k, threshold 3k, collection 24k (near the copy rate while it lasts),
// bins 4k, edge 4k, writing 5k.  Lists per warp built with votes at 256 threads, four
// CTAs an SM, took 77k cycles a CTA: the same time.  Starting the collection's
// loads before the sample only made the sample wait for them.  One row of 500k keys
// on a cluster: 17 us; counting into the first CTA's histogram by remote atomics,
// instead of adding the CTAs' histograms there, took 2 us more.
#include <cooperative_groups.h>

#include <algorithm>
#include <cmath>

#include "paged.cuh"
#include "select_common.cuh"

namespace dma {
namespace {

namespace cg = cooperative_groups;

constexpr int kSpSample = 512;           // sampled octs (runs of eight positions), at most
constexpr int kSpSampleLong = 131072;    // rows up to this length take half of them (512 rows of 32k to 64k keys at w = 2048
                                         // and 4000, attention included: 162 and 260 us; all of them 166 and 264; a quarter 161 and 276)
constexpr int kSpEdge = 512;             // keys inside the w-th key's bin
constexpr int kSpMaxCluster = 8;         // CTAs of a row
constexpr int kSpSpill = 128;            // keys of a CTA that found their thread's list full
// many rows: 512 threads, two CTAs per SM; rows split over a cluster: 1024
// threads, one CTA per SM
template <int THREADS>
struct SpCfg {
  static constexpr int kMinBlocks = THREADS == 512 ? 2 : 1;
  static constexpr int kUnroll = 2;   // octs in flight per thread
  static constexpr int kSlack = 4;    // list rows past the room: keys appended between two checks
};

struct SpShared {
  __align__(16) uint32_t hist[kBins];
  uint64_t edge[kSpEdge];                // (first CTA) keys inside the w-th key's bin
  uint64_t spill[kSpSpill];              // keys that found their thread's list full
  uint32_t warp[3][32];                  // per-warp values
  uint32_t bin[3];                       // top_bin's answer
  uint32_t keys, sure, spills;           // this CTA's collected keys, those above the bin, those in `spill`
  uint32_t edges, exact;                 // (first CTA) keys in `edge`; the row needs the exact selection
  uint32_t ties;                         // this CTA's keys of the tied value
};
// dynamic shared memory: SpShared, then the collected keys' dt bits and
// positions, [room + kSlack][2][THREADS] (first the sample's values)

// Appends (bits, pos) at shared address `at` and moves it on, when bits reach
// the threshold: four predicated instructions, no branch.
template <int THREADS>
__device__ __forceinline__ void append_if(uint32_t& at, uint32_t bits, uint32_t pos, uint32_t thr) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ge.u32 p, %1, %3;\n\t@p st.shared.u32 [%0], %1;\n\t@p st.shared.u32 [%0+%4], %2;\n\t"
      "@p add.u32 %0, %0, %5;\n\t}"
      : "+r"(at)
      : "r"(bits), "r"(pos), "r"(thr), "n"(4 * THREADS), "n"(8 * THREADS)
      : "memory");
}

// A row's visible keys as octs of eight positions: octs [0, noa) cover the
// sinks, the rest the positions from `start` on.
struct Row {
  const int32_t* table;
  int g, sinks, start, len, noa, no, ob;
};

__device__ __forceinline__ Row make_row(const PagedCache& c, const SeqView& v, int b, int g) {
  Row r;
  r.table = c.table + static_cast<size_t>(b) * c.max_pages;
  r.g = g;
  r.len = v.len;
  r.sinks = v.shift > 0 ? c.sinks : 0;
  r.start = v.shift > 0 ? c.sinks + v.shift : 0;
  r.noa = (r.sinks + 7) >> 3;
  r.ob = r.start >> 3;
  r.no = r.noa + ((r.len + 7) >> 3) - r.ob;
  return r;
}

__device__ __forceinline__ int oct_position(const Row& r, int x) { return 8 * (x < r.noa ? x : x - r.noa + r.ob); }

// which of an oct's positions from j0 on are visible (bit e)
__device__ __forceinline__ uint32_t oct_mask(const Row& r, int x, int j0) {
  if (x > r.noa && x + 1 < r.no) return 255u;   // inside the second range
  const int lo = x < r.noa ? 0 : r.start, hi = x < r.noa ? r.sinks : r.len;
  const uint32_t below = (1u << min(8, max(0, lo - j0))) - 1u;
  return ((1u << min(8, max(0, hi - j0))) - 1u) & ~below;
}

// The table entry of an oct's first position (0 from oct `end` on).
__device__ __forceinline__ int oct_page(const PagedCache& c, const Row& r, int x, int end) {
  if (x >= end) return 0;
  int off;
  return __ldg(r.table + page_slot(c, oct_position(r, x), off));
}

// dt bits of an oct; returns which of its positions are seen (bit e).  VEC: the
// page size is a multiple of eight, so an oct lies in one page and two 16-byte
// loads bring it.
template <bool VEC>
__device__ __forceinline__ uint32_t load_oct(const PagedCache& c, const Row& r, int x, int page, uint32_t (&v)[8],
                                             int end) {
  if (x >= end) return 0u;
  const int j0 = oct_position(r, x);
  uint32_t seen = oct_mask(r, x, j0);
  int off;
  int slot = page_slot(c, j0, off);
  if constexpr (VEC) {
    page = checked_page(c, page);
    if (page < 0) return 0u;
    const uint4* src = reinterpret_cast<const uint4*>(c.dt_pages + dt_offset(c, page, off, r.g));
    const uint4 a = __ldg(src), b = __ldg(src + 1);
    v[0] = a.x;
    v[1] = a.y;
    v[2] = a.z;
    v[3] = a.w;
    v[4] = b.x;
    v[5] = b.y;
    v[6] = b.z;
    v[7] = b.w;
  } else {
    // the entries of all eight first, then their dt: one latency each
    int pages[8], offs[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      pages[e] = e == 0 ? page : pages[e > 0 ? e - 1 : 0];
      if (off == c.page_size) {
        off = 0;
        ++slot;
        if (seen >> e) pages[e] = __ldg(r.table + slot);
      }
      offs[e] = off++;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if ((seen >> e & 1u) && checked_page(c, pages[e]) < 0) seen &= ~(1u << e);
      v[e] = seen >> e & 1u ? __float_as_uint(__ldg(c.dt_pages + dt_offset(c, pages[e], offs[e], r.g))) : 0u;
    }
  }
  return seen;
}

// A step of the collection: 32 octs from q0 on, eight keys of them per lane.  VEC:
// an oct a lane; else lane l has every 32nd key from the l-th on, so that a load
// of the warp reads neighbouring keys (64 sequences of 32k to 64k keys in pages of
// five, the step with its attention: 480 us with an oct a lane, 274 us so; in pages
// of 100, 208 and 225 us).
template <bool VEC>
__device__ __forceinline__ int step_position(const Row& r, int q0, int e) {
  const int lane = threadIdx.x & 31;
  return VEC ? oct_position(r, q0 + lane) + e : oct_position(r, q0 + 4 * e + (lane >> 3)) + (lane & 7);
}

// dt bits of this lane's keys of a step, 0 for those that are not seen.  page: the
// table entry of its oct (VEC).
template <bool VEC>
__device__ __forceinline__ uint32_t load_step(const PagedCache& c, const Row& r, int q0, int page, uint32_t (&v)[8],
                                              int end) {
  const int lane = threadIdx.x & 31;
  uint32_t seen = 0u;
  if constexpr (VEC) {
    seen = load_oct<true>(c, r, q0 + lane, page, v, end);
  } else {
    int pages[8], offs[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int x = q0 + 4 * e + (lane >> 3), j = oct_position(r, x) + (lane & 7);
      const bool there = x < end && (x < r.noa ? j < r.sinks : j >= r.start && j < r.len);
      seen |= there ? 1u << e : 0u;
      const int slot = page_slot(c, there ? j : 0, offs[e]);
      pages[e] = there ? __ldg(r.table + slot) : 0;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if ((seen >> e & 1u) && checked_page(c, pages[e]) < 0) seen &= ~(1u << e);
      v[e] = seen >> e & 1u ? __float_as_uint(__ldg(c.dt_pages + dt_offset(c, pages[e], offs[e], r.g))) : 0u;
    }
  }
  return seen;
}

// A row's kept list.
struct Kept {
  int32_t* pos;
  float* bias;
  __device__ __forceinline__ void put(uint32_t at, int j, uint32_t bits) const {
    pos[at] = j;
    bias[at] = __uint_as_float(bits);
  }
  __device__ __forceinline__ void put(uint32_t at, uint64_t key) const {
    put(at, static_cast<int>(composite_index(key)), static_cast<uint32_t>(key >> 32));
  }
};

// Smallest shift that maps [0, range] into 2048 bins.
__device__ __forceinline__ int bin_shift(uint32_t range) {
  const int top = 32 - __clz(static_cast<int>(range | 1u));   // bits in use
  return top > 11 ? top - 11 : 0;
}

// The highest value of the bin that begins at lo, or hi where that is lower (without
// the sum's overflow: bits near 2^32, which no dt >= 0 has, must not widen the range
// or leave it empty).
__device__ __forceinline__ uint32_t bin_top(uint32_t lo, int shift, uint32_t hi) {
  return hi - lo < (1u << shift) ? hi : lo + ((1u << shift) - 1u);
}

// Sum of the warps' values before this warp, from one value per warp.
__device__ __forceinline__ uint32_t warps_before(const uint32_t* per_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  return __reduce_add_sync(0xFFFFFFFFu, lane < warp ? per_warp[lane] : 0u);
}

// The histogram bin (from the top) that holds the k-th key, how many of its
// keys belong to the k, and how many it has; the histogram is cleared.  Every
// thread calls it after a barrier behind the histogram's last addition and
// gets the answer; `k` keys are there.  others: histograms of the cluster's
// other CTAs to add.
template <int THREADS, class F>
__device__ __forceinline__ void top_bin(SpShared& sm, uint32_t k, F&& others, uint32_t& bin, uint32_t& need,
                                        uint32_t& count) {
  constexpr int PER = kBins / THREADS;   // bins per thread, the highest at thread 0
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int base = kBins - (tid + 1) * PER;
  uint32_t h[PER], local = 0;
#pragma unroll
  for (int i = 0; i < PER; i += 2) {
    uint2* mine = reinterpret_cast<uint2*>(sm.hist + base + i);
    const uint2 x = *mine, y = others(base + i);
    *mine = make_uint2(0u, 0u);
    h[i] = x.x + y.x;
    h[i + 1] = x.y + y.y;
    local += h[i] + h[i + 1];
  }
  uint32_t above = local;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, above, d);
    if (lane >= d) above += y;
  }
  if (lane == 31) sm.warp[0][warp] = above;
  __syncthreads();
  above += warps_before(sm.warp[0]) - local;
  if (above < k && above + local >= k) {
#pragma unroll
    for (int i = PER - 1; i >= 0; --i) {
      if (above < k && above + h[i] >= k) {
        sm.bin[0] = static_cast<uint32_t>(base + i);
        sm.bin[1] = k - above;
        sm.bin[2] = h[i];
      }
      above += h[i];
    }
  }
  __syncthreads();
  bin = sm.bin[0];
  need = sm.bin[1];
  count = sm.bin[2];
}

// The rank in the sample whose key the w-th key of the row lies above but for
// one row in a hundred thousand, when `expect` of the w best are sampled.
template <class T>
__host__ __device__ __forceinline__ T sample_rank(T expect) {
  return expect + T(4.3) * sqrt(expect) + T(5);
}

struct NoOthers {
  __device__ __forceinline__ uint2 operator()(int) const { return make_uint2(0u, 0u); }
};

// (count, minimum, maximum) over the block of each thread's own
template <int THREADS>
__device__ __forceinline__ void block_range(SpShared& sm, uint32_t& n, uint32_t& lo, uint32_t& hi) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  n = __reduce_add_sync(0xFFFFFFFFu, n);
  lo = __reduce_min_sync(0xFFFFFFFFu, lo);
  hi = __reduce_max_sync(0xFFFFFFFFu, hi);
  if (lane == 0) {
    sm.warp[0][warp] = n;
    sm.warp[1][warp] = lo;
    sm.warp[2][warp] = hi;
  }
  __syncthreads();
  const bool in = lane < THREADS / 32;
  n = __reduce_add_sync(0xFFFFFFFFu, in ? sm.warp[0][lane] : 0u);
  lo = __reduce_min_sync(0xFFFFFFFFu, in ? sm.warp[1][lane] : 0xFFFFFFFFu);
  hi = __reduce_max_sync(0xFFFFFFFFu, in ? sm.warp[2][lane] : 0u);
}

// Exact selection by one CTA: a few histogram passes over the row narrow the
// dt bits of the w-th key to one value, then two passes write the keys above
// it and the lowest-indexed ones equal to it.  Each warp owns a contiguous part
// of the row, so the list is in a fixed order.
template <int THREADS, bool VEC>
static __device__ __noinline__ void select_exact(const PagedCache& c, const Kept& out, const Row& r, int w, SpShared& sm) {
  constexpr int kWarps = THREADS / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int seg = ((r.no + kWarps - 1) / kWarps + 31) / 32 * 32;
  const int x0 = min(r.no, warp * seg), x1 = min(r.no, x0 + seg);
  auto each = [&](auto&& f) {   // f(oct, bits, seen): the whole warp calls it together
    for (int q0 = x0; q0 < x1; q0 += 32) {
      const int x = q0 + lane;
      uint32_t v[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
      const uint32_t seen = x < x1 ? load_oct<VEC>(c, r, x, oct_page(c, r, x, x1), v, x1) : 0u;
      f(x, v, seen);
    }
  };
  uint32_t total = 0, lo = 0xFFFFFFFFu, hi = 0u;
  each([&](int, const uint32_t(&v)[8], uint32_t seen) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (seen >> e & 1u) {
        ++total;
        lo = min(lo, v[e]);
        hi = max(hi, v[e]);
      }
  });
  for (int i = tid; i < kBins; i += THREADS) sm.hist[i] = 0;
  __syncthreads();   // what the caller left in shared memory has been read
  block_range<THREADS>(sm, total, lo, hi);
  uint32_t k = static_cast<uint32_t>(w);   // keys to keep of those in [lo, hi]
  if (total > static_cast<uint32_t>(w)) {
    while (lo < hi) {
      const int s = bin_shift(hi - lo);
      __syncthreads();
      each([&](int, const uint32_t(&v)[8], uint32_t seen) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if ((seen >> e & 1u) && v[e] >= lo && v[e] <= hi) atomicAdd(&sm.hist[(v[e] - lo) >> s], 1u);
      });
      __syncthreads();
      uint32_t bin, cnt;
      top_bin<THREADS>(sm, k, NoOthers{}, bin, k, cnt);
      const uint32_t l2 = lo + (bin << s);
      hi = bin_top(l2, s, hi);
      lo = l2;
    }
  } else {
    // pages outside the pool left no more than w keys: all of them are kept
    k = total;
    lo = 0u;
  }
  // the keys above lo, then the k lowest-indexed ones equal to it
  uint32_t gt = 0, eq = 0;
  each([&](int, const uint32_t(&v)[8], uint32_t seen) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      gt += (seen >> e & 1u) && v[e] > lo;
      eq += (seen >> e & 1u) && v[e] == lo;
    }
  });
  gt = __reduce_add_sync(0xFFFFFFFFu, gt);
  eq = __reduce_add_sync(0xFFFFFFFFu, eq);
  __syncthreads();
  if (lane == 0) {
    sm.warp[0][warp] = gt;
    sm.warp[1][warp] = eq;
  }
  __syncthreads();
  uint32_t gpos = warps_before(sm.warp[0]), epos = warps_before(sm.warp[1]);
  const uint32_t gall = __reduce_add_sync(0xFFFFFFFFu, lane < kWarps ? sm.warp[0][lane] : 0u);
  const uint32_t lt = lanemask_lt();
  each([&](int x, const uint32_t(&v)[8], uint32_t seen) {
    const int j0 = x < r.no ? oct_position(r, x) : 0;
    uint32_t n = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) n += (seen >> e & 1u) && v[e] == lo;
    // this lane's first equal key's rank: prefix of n (0..8) over the lanes
    const uint32_t b0 = __ballot_sync(0xFFFFFFFFu, n & 1u), b1 = __ballot_sync(0xFFFFFFFFu, n & 2u),
                   b2 = __ballot_sync(0xFFFFFFFFu, n & 4u), b3 = __ballot_sync(0xFFFFFFFFu, n & 8u);
    uint32_t er = epos + __popc(b0 & lt) + 2u * __popc(b1 & lt) + 4u * __popc(b2 & lt) + 8u * __popc(b3 & lt);
    epos += __popc(b0) + 2u * __popc(b1) + 4u * __popc(b2) + 8u * __popc(b3);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const bool above = (seen >> e & 1u) && v[e] > lo;
      const uint32_t vote = __ballot_sync(0xFFFFFFFFu, above);
      if (above) out.put(gpos + __popc(vote & lt), j0 + e, v[e]);
      gpos += __popc(vote);
      if ((seen >> e & 1u) && v[e] == lo) {
        if (er < k) out.put(gall + er, j0 + e, v[e]);
        ++er;
      }
    }
  });
  // entries that pages outside the pool left empty
  for (int e = static_cast<int>(min(total, static_cast<uint32_t>(w))) + tid; e < w; e += THREADS) out.put(e, -1, 0u);
}

// CLUSTER: a row's octs are dealt to the CTAs of a cluster (else it has one CTA).
template <int THREADS, bool VEC, bool CLUSTER>
__global__ void __launch_bounds__(THREADS, SpCfg<THREADS>::kMinBlocks)
    select_paged_kernel(const __grid_constant__ PagedCache c, const __grid_constant__ PagedLists o, int room) {
  using Cfg = SpCfg<THREADS>;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  SpShared& sm = *reinterpret_cast<SpShared*>(smem_raw);
  uint32_t* list = reinterpret_cast<uint32_t*>(smem_raw + sizeof(SpShared));
  cg::cluster_group cluster = cg::this_cluster();
  auto sync_all = [&]() {
    if (CLUSTER)
      cluster.sync();
    else
      __syncthreads();
  };
  const int csize = CLUSTER ? static_cast<int>(cluster.num_blocks()) : 1;
  const int rank = CLUSTER ? static_cast<int>(cluster.block_rank()) : 0;
  auto of_rank = [&](int q) { return CLUSTER ? cluster.map_shared_rank(&sm, q) : &sm; };
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bg = blockIdx.x / csize;
  const int w = c.w;
  const SeqView view = seq_view(c, bg / c.Hkv);
  if (view.n <= w) return;   // the attention takes such a row as it is (the whole cluster returns)
  const Row r = make_row(c, view, bg / c.Hkv, bg % c.Hkv);
  const Kept out{o.pos + static_cast<size_t>(bg) * o.cap, o.bias + static_cast<size_t>(bg) * o.cap};

  // ---- the sample and its threshold (every CTA of the cluster finds the same)
  uint32_t* sample = list;
  const int socts = min(view.n > kSpSampleLong ? kSpSample : kSpSample / 2, r.no);
  for (int i = tid; i < kBins; i += THREADS) sm.hist[i] = 0;
  if (tid == 0) sm.keys = sm.sure = sm.spills = sm.edges = sm.exact = sm.ties = 0u;
  uint32_t ns = 0, thr = 0xFFFFFFFFu, smax = 0u;
  static_assert(THREADS >= kSpSample, "a sampled oct per thread, and the sample fits eight list rows");
  if (tid < socts) {
    const int x = static_cast<int>(static_cast<uint32_t>(tid * r.no) / static_cast<uint32_t>(socts));   // below 2^26
    uint32_t v[8];
    const uint32_t seen = load_oct<VEC>(c, r, x, oct_page(c, r, x, r.no), v, r.no);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const bool ok = seen >> e & 1u;
      sample[e * kSpSample + tid] = ok ? v[e] : 0u;
      if (ok) {
        ++ns;
        thr = min(thr, v[e]);
        smax = max(smax, v[e]);
      }
    }
  }
  block_range<THREADS>(sm, ns, thr, smax);
  uint32_t k = static_cast<uint32_t>(
      sample_rank(static_cast<float>(w) * static_cast<float>(ns) / static_cast<float>(view.n)));
  bool tied = thr == smax;   // the threshold is one value with many keys of the sample
  if (k < ns) {
    uint32_t lo = thr, hi = smax;
    while (lo < hi) {
      const int s = bin_shift(hi - lo);
      if (tid < socts) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t x = sample[e * kSpSample + tid];   // unseen places hold 0: below lo, or the lowest value there is
          if (x >= lo && x <= hi) atomicAdd(&sm.hist[(x - lo) >> s], 1u);
        }
      }
      __syncthreads();
      uint32_t bin, cnt;
      top_bin<THREADS>(sm, k, NoOthers{}, bin, k, cnt);
      const uint32_t l2 = lo + (bin << s);
      hi = bin_top(l2, s, hi);
      lo = l2;
      if (cnt <= 16u) break;   // its lower edge takes a few more keys than the exact value would
      tied = lo == hi;
    }
    thr = lo;
  }
  const uint32_t tie = thr;
  // (0: positions that are not seen read as 0, below every threshold; nothing lies above
  // 2^32 - 1, whose row comes out right by collecting the tied keys themselves)
  tied = (tied || thr == 0u) && thr != 0xFFFFFFFFu;
  if (tied) ++thr;
  __syncthreads();   // the sample has been read: keys are written over it

  // ---- collect, an oct per thread and step
  const int shift = bin_shift(smax > thr ? smax - thr : 0u);
  auto bin_of = [&](uint32_t bits) { return min(static_cast<uint32_t>(kBins - 1), (bits - thr) >> shift); };
  constexpr uint32_t kStep = 8u * THREADS;   // bytes between a thread's keys
  const uint32_t first = smem_u32(list + tid);
  const uint32_t full = first + static_cast<uint32_t>(room) * kStep;
  uint32_t at = first;   // place of this thread's next key
  uint32_t n_tied = 0;
  // each warp of the cluster takes a contiguous part of the row, 32 octs at a
  // time, so that the list ends up roughly in the order of the positions
  const int part = (r.no + csize * THREADS - 1) / (csize * THREADS) * 32;
  const int xw = min(r.no, (rank * (THREADS / 32) + warp) * part), xe = min(r.no, xw + part);
  {
    int page[Cfg::kUnroll];
    uint32_t v[Cfg::kUnroll][8], seen[Cfg::kUnroll];
#pragma unroll
    for (int u = 0; u < Cfg::kUnroll; ++u) page[u] = VEC ? oct_page(c, r, xw + lane + 32 * u, xe) : 0;
#pragma unroll
    for (int u = 0; u < Cfg::kUnroll; ++u) {
      seen[u] = load_step<VEC>(c, r, xw + 32 * u, page[u], v[u], xe);
      if (VEC) page[u] = oct_page(c, r, xw + lane + 32 * (Cfg::kUnroll + u), xe);
    }
    for (int q0 = xw; q0 < xe; q0 += 32 * Cfg::kUnroll) {
#pragma unroll
      for (int u = 0; u < Cfg::kUnroll; ++u) {
        if (VEC && seen[u] != 255u) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[u][e] = seen[u] >> e & 1u ? v[u][e] : 0u;
        }
        if (tied) {
#pragma unroll
          for (int e = 0; e < 8; ++e) n_tied += (seen[u] >> e & 1u) && v[u][e] == tie;
        }
        const int qu = q0 + 32 * u, j0 = step_position<VEC>(r, qu, 0);
#pragma unroll
        for (int e0 = 0; e0 < 8; e0 += Cfg::kSlack) {
#pragma unroll
          for (int e = e0; e < e0 + Cfg::kSlack; ++e)
            append_if<THREADS>(at, v[u][e], VEC ? j0 + e : step_position<VEC>(r, qu, e), thr);
          for (; at > full; at -= kStep) {   // the keys in the slack rows move to the CTA's spill
            const uint32_t last = (at - first) / kStep - 1u;
            const uint32_t bits = list[2 * last * THREADS + tid], pos = list[(2 * last + 1) * THREADS + tid];
            const uint32_t i = atomicAdd(&sm.spills, 1u);
            if (i < static_cast<uint32_t>(kSpSpill)) sm.spill[i] = composite_key(bits, pos);
            atomicAdd(&sm.keys, 1u);
            atomicAdd(&sm.hist[bin_of(bits)], 1u);
          }
        }
        // this place's next keys travel while the others are looked through
        seen[u] = load_step<VEC>(c, r, qu + 32 * Cfg::kUnroll, page[u], v[u], xe);
        if (VEC) page[u] = oct_page(c, r, qu + lane + 64 * Cfg::kUnroll, xe);
      }
    }
  }
  const int n = static_cast<int>((at - first) / kStep);   // this thread's keys
  auto key_pos = [&](int i) { return static_cast<int>(list[(2 * i + 1) * THREADS + tid]); };
  // f(i, bits, bin) for each of them, four read at a time (the slack rows follow the last)
  auto each_key = [&](auto&& f) {
    static_assert(Cfg::kSlack >= 3, "reads past a full list");
    for (int i0 = 0; i0 < n; i0 += 4) {
      uint32_t bits[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) bits[i] = list[2 * (i0 + i) * THREADS + tid];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i0 + i < n) f(i0 + i, bits[i], static_cast<int>(bin_of(bits[i])));
    }
  };
  {
    const uint32_t all = __reduce_add_sync(0xFFFFFFFFu, static_cast<uint32_t>(n));
    n_tied = __reduce_add_sync(0xFFFFFFFFu, n_tied);
    if (lane == 0) {
      atomicAdd(&sm.keys, all);
      atomicAdd(&sm.ties, n_tied);
      sm.warp[2][warp] = n_tied;
    }
    each_key([&](int, uint32_t, int bin) { atomicAdd(&sm.hist[bin], 1u); });
  }

  // ---- the w-th key's bin, over the cluster
  sync_all();
  uint32_t bad, total, ties, ties_before;   // ..before: in the CTAs before this one
  {
    const SpShared* other = of_rank(min(lane, csize - 1));   // a CTA a lane
    const bool in = lane < csize;
    const uint32_t spills = other->spills, keys = other->keys, tied_keys = other->ties;
    bad = __any_sync(0xFFFFFFFFu, spills > static_cast<uint32_t>(kSpSpill));
    total = __reduce_add_sync(0xFFFFFFFFu, in ? keys : 0u);
    ties = __reduce_add_sync(0xFFFFFFFFu, in ? tied_keys : 0u);
    ties_before = __reduce_add_sync(0xFFFFFFFFu, lane < rank ? tied_keys : 0u);
  }
  // keys of the tied value that the list still has room for
  const uint32_t fill = total < static_cast<uint32_t>(w) ? static_cast<uint32_t>(w) - total : 0u;
  bad |= fill > ties;
  SpShared* lead = of_rank(0);
  if (!bad && fill == 0u && rank == 0) {
    uint32_t wbin, need, cnt;
    top_bin<THREADS>(
        sm, static_cast<uint32_t>(w),
        [&](int i) {
          uint2 s = make_uint2(0u, 0u);
          if (CLUSTER) {
            uint2 y[kSpMaxCluster];   // all on their way at once
#pragma unroll
            for (int q = 1; q < kSpMaxCluster; ++q)
              y[q] = q < csize ? *reinterpret_cast<const uint2*>(of_rank(q)->hist + i) : make_uint2(0u, 0u);
#pragma unroll
            for (int q = 1; q < kSpMaxCluster; ++q) {
              s.x += y[q].x;
              s.y += y[q].y;
            }
          }
          return s;
        },
        wbin, need, cnt);
    if (tid == 0 && cnt > static_cast<uint32_t>(kSpEdge)) sm.exact = 1u;
  }
  sync_all();
  const int wbin = fill > 0u ? -1 : static_cast<int>(lead->bin[0]);   // below all bins: every collected key is kept
  const uint32_t need = fill > 0u ? 0u : lead->bin[1];
  bad |= lead->exact;
  uint32_t before = 0;   // the warp's sure keys before this thread's
  if (!bad) {
    // keys inside the bin go to the first CTA (they are ranked by value, so
    // their order there does not matter); keys above it are counted
    each_key([&](int i, uint32_t bits, int bin) {
      before += bin > wbin;
      if (bin == wbin) lead->edge[atomicAdd(&lead->edges, 1u)] = composite_key(bits, key_pos(i));
    });
    if (tid < sm.spills) {
      const uint64_t key = sm.spill[tid];
      const int bin = static_cast<int>(bin_of(static_cast<uint32_t>(key >> 32)));
      if (bin > wbin) atomicAdd(&sm.sure, 1u);
      if (bin == wbin) lead->edge[atomicAdd(&lead->edges, 1u)] = key;
    }
    const uint32_t own = before;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, before, d);
      if (lane >= d) before += y;
    }
    if (lane == 31) {
      sm.warp[1][warp] = before;
      atomicAdd(&sm.sure, before);
    }
    before -= own;
  }
  sync_all();
  if (!bad) {
    const uint32_t sure = of_rank(min(lane, csize - 1))->sure;
    const uint32_t start = __reduce_add_sync(0xFFFFFFFFu, lane < rank ? sure : 0u);
    uint32_t pos = start + warps_before(sm.warp[1]) + before;
    each_key([&](int i, uint32_t bits, int bin) {
      if (bin > wbin) out.put(pos++, key_pos(i), bits);
    });
    // then the spilled ones, in the order of their positions
    const uint32_t spills = sm.spills;
    const uint64_t key = tid < spills ? sm.spill[tid] : 0ull;
    auto is_sure = [&](uint64_t k) { return static_cast<int>(bin_of(static_cast<uint32_t>(k >> 32))) > wbin; };
    if (spills > 0) {
      pos = start + __reduce_add_sync(0xFFFFFFFFu, lane < THREADS / 32 ? sm.warp[1][lane] : 0u);
      if (tid < spills && is_sure(key)) {
        for (uint32_t i = 0; i < spills; ++i)
          pos += is_sure(sm.spill[i]) && composite_index(sm.spill[i]) < composite_index(key);
        out.put(pos, key);
      }
    }
    // the lowest-indexed keys of the tied value: a warp whose part has some of them
    // reads it again
    uint32_t trank = ties_before + warps_before(sm.warp[2]);
    for (int x0 = xw; x0 < xe && trank < fill; x0 += 32) {
      const int x = x0 + lane;
      uint32_t v[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
      const uint32_t seen = load_oct<VEC>(c, r, x, oct_page(c, r, x, xe), v, xe);
      uint32_t m = 0u;
#pragma unroll
      for (int e = 0; e < 8; ++e) m |= (seen >> e & 1u) && v[e] == tie ? 1u << e : 0u;
      uint32_t upto = __popc(m);
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, upto, d);
        if (lane >= d) upto += y;
      }
      uint32_t mine = trank + upto - __popc(m);
      for (; m && mine < fill; m &= m - 1u, ++mine)
        out.put(total + mine, oct_position(r, x) + __ffs(static_cast<int>(m)) - 1, tie);
      trank += __shfl_sync(0xFFFFFFFFu, upto, 31);
    }
    if (rank == 0) {
      // the bin's `need` best keys, each at its rank
      const uint32_t ne = sm.edges;
      for (uint32_t i = tid; i < ne; i += THREADS) {
        const uint64_t mine = sm.edge[i];
        uint32_t above = 0;
        for (uint32_t q = 0; q < ne; ++q) above += sm.edge[q] > mine;
        if (above < need) out.put(w - need + above, mine);
      }
    }
  }
  if (CLUSTER) cluster.sync();   // no CTA leaves while another reads its shared memory
  if (bad && rank == 0) select_exact<THREADS, VEC>(c, out, r, w, sm);
}

// List entries per thread in the longest row, over `threads` threads: the share of the
// keys expected above the threshold, and its standard deviation (of the threshold's
// rank in the sample, and of the share).
struct Share {
  double mean, deviation;
};

Share share_of(const PagedCache& c, int threads) {
  const double keys = static_cast<double>(c.longest);
  const double ratio = keys / (keys > kSpSampleLong ? 8.0 * kSpSample : 4.0 * kSpSample);   // keys per sampled one
  const double rank = sample_rank(c.w / ratio);
  const double mean = rank * ratio / threads;
  return Share{mean, std::sqrt(mean + mean * mean / rank)};
}

// list entries per thread that let `per_sm` CTAs share an SM's shared memory
template <int THREADS>
int most_room(int per_sm) {
  return ((227 * 1024) / per_sm - 1024 - static_cast<int>(sizeof(SpShared))) / (8 * THREADS) - SpCfg<THREADS>::kSlack;
}

template <int THREADS, bool VEC, bool CLUSTER>
cudaError_t launch_sp(const PagedCache& c, const PagedLists& lists, int rows, int csize, cudaStream_t s) {
  // four standard deviations of room where shared memory has it (a few keys
  // spill where it has less; windows far beyond it are selected exactly)
  const Share share = share_of(c, THREADS * csize);
  const int room = std::max(8, static_cast<int>(std::min(share.mean + 4.0 * share.deviation + 2.0,
                                                         static_cast<double>(most_room<THREADS>(SpCfg<THREADS>::kMinBlocks)))));
  const int smem = static_cast<int>(sizeof(SpShared)) + 8 * (room + SpCfg<THREADS>::kSlack) * THREADS;
  const void* fn = reinterpret_cast<const void*>(select_paged_kernel<THREADS, VEC, CLUSTER>);
  const cudaError_t e = ensure_dyn_smem(fn, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows) * csize);
  cfg.blockDim = dim3(THREADS);
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
  cfg.numAttrs = CLUSTER ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, select_paged_kernel<THREADS, VEC, CLUSTER>, c, lists, room);
}

}  // namespace

cudaError_t launch_select_paged(const PagedCache& c, const PagedLists& lists, cudaStream_t s) {
  const int nsm = sm_count();
  if (nsm <= 0) return cudaErrorInvalidDevice;
  const int rows = c.B * c.Hkv;
  const bool vec = c.page_size % 8 == 0;
  // few rows: as many CTAs per row as the SMs hold at once, each with 4096 keys or
  // more of the longest row (one sequence of 500k keys, 8 heads, attention included:
  // 28.5 us on eight CTAs a row, 109 us on one; 4 sequences with a window of 8192 keys, 4
  // heads, in tables of 500k: 20 us on two CTAs a row, 33 us on the eight that the tables'
  // length would ask for)
  int csize = 1;
  while (csize < kSpMaxCluster && 2LL * csize * rows <= nsm && c.longest >= 4096 * 2 * csize) csize *= 2;
  if (csize > 1)
    return vec ? launch_sp<1024, true, true>(c, lists, rows, csize, s)
               : launch_sp<1024, false, true>(c, lists, rows, csize, s);
  // many rows: one CTA each, or as many as give the lists of a large window room
  // while two CTAs share an SM (512 rows of 32k to 64k keys at w = 4000, the step with
  // its attention: 306 us with one CTA an SM, 260 us so)
  for (; csize < kSpMaxCluster; csize *= 2) {
    const Share share = share_of(c, 512 * csize);
    if (share.mean + 2.0 * share.deviation <= most_room<512>(2)) break;
  }
  if (csize > 1)
    return vec ? launch_sp<512, true, true>(c, lists, rows, csize, s)
               : launch_sp<512, false, true>(c, lists, rows, csize, s);
  return vec ? launch_sp<512, true, false>(c, lists, rows, 1, s) : launch_sp<512, false, false>(c, lists, rows, 1, s);
}

}  // namespace dma
