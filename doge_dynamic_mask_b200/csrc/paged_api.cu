// C ABI of the paged cache (append, decode step) and of the prologue's
// backward: argument checks, workspace layout, launches.  See include/dma.h.
#include <algorithm>
#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/dma.h"
#include "dma_internal.h"

using namespace dma;

namespace {

template <class... P>
bool ready(const P*... p) {   // every pointer given and 16-byte aligned
  return ((p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) && ...);
}

bool rope_args_ok(float eps, float theta) { return eps >= 0.0f && eps <= 1.0f && theta > 1.0f && theta < 3.0e38f; }

// elements between tokens: whole 16-byte units, no overlap
bool stride_ok(long long stride, int heads, int d) { return stride >= static_cast<long long>(heads) * d && stride % 8 == 0; }

dma_status_t check_pages(int B, int max_pages, int num_pages, int page_size, long long page_stride, int Hkv, int d) {
  if (B < 1 || max_pages < 1 || num_pages < 1 || page_size < 1) return DMA_ERR_INVALID_ARG;
  const long long page = static_cast<long long>(page_size) * Hkv * d;
  if (page_stride < page || page_stride % 8 != 0) return DMA_ERR_INVALID_ARG;
  if (B > 65536 || static_cast<long long>(max_pages) * page_size > kMaxLen) return DMA_ERR_UNSUPPORTED;
  // rows are addressed in 16-byte units of 32 bits (64 GiB of K, and of V)
  if (page_stride / 8 > (1LL << 32) / num_pages - 1) return DMA_ERR_UNSUPPORTED;
  return DMA_OK;
}

// keys a query may see, at most
long long visible_cap(int max_pages, int page_size, int window, int sinks) {
  const long long cap = static_cast<long long>(max_pages) * page_size;
  return window > 0 ? std::min(cap, static_cast<long long>(window) + sinks) : cap;
}

// Paged decode workspace: header, the attention's scratch, and, when a query
// may see more than keep_window_size keys, the kept lists.
struct PagedWorkspace {
  size_t scratch, pos, bias, bytes;
  int cap;
};

PagedWorkspace paged_workspace(int B, int max_pages, int page_size, int Hq, int Hkv, int d, int w, int window, int sinks) {
  PagedWorkspace p{};
  p.scratch = kHeaderBytes;
  p.bytes = align_up(p.scratch + attn_paged_scratch_bytes(Hq, Hkv, d), 256);
  if (visible_cap(max_pages, page_size, window, sinks) > w) {
    p.cap = w;
    const size_t list = static_cast<size_t>(B) * Hkv * w * 4;
    p.pos = p.bytes;
    p.bias = align_up(p.pos + list, 256);
    p.bytes = align_up(p.bias + list, 256);
  }
  return p;
}

dma_status_t check_paged_decode(int B, int max_pages, int page_size, int Hq, int Hkv, int d, int w, int window,
                                int sinks) {
  if (B < 1 || max_pages < 1 || page_size < 1 || w < 1 || window < 0 || sinks < 0) return DMA_ERR_INVALID_ARG;
  const dma_status_t st = check_heads(Hq, Hkv, d);
  if (st != DMA_OK) return st;
  if (B > 65536 || static_cast<long long>(max_pages) * page_size > kMaxLen) return DMA_ERR_UNSUPPORTED;
  // the attention counts 16-key tiles of all rows in 31 bits
  const long long keys = std::min<long long>(visible_cap(max_pages, page_size, window, sinks), w);
  if ((keys + 15) / 16 * B * Hkv >= 1LL << 31) return DMA_ERR_UNSUPPORTED;
  return DMA_OK;
}

}  // namespace

extern "C" {

dma_status_t dma_append_paged(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                              int64_t v_stride, const float* q_norm_w, const float* k_norm_w, float eps,
                              float rope_theta, const float* W_dt, const float* A, const int32_t* cu_tokens,
                              const int32_t* positions, const int32_t* page_table, int T, int B, int max_pages,
                              int num_pages, int page_size, int64_t page_stride, int Hq, int Hkv, int d, void* q_out,
                              void* k_out, void* k_pages, void* v_pages, float* dt_pages, void* workspace,
                              size_t ws_bytes, dma_stream_t stream) {
  if (!ready(q, k, v, q_norm_w, k_norm_w, W_dt, A, cu_tokens, positions, page_table, q_out, k_pages, v_pages, dt_pages,
             workspace) ||
      (k_out && !ready(k_out)))
    return DMA_ERR_INVALID_ARG;
  if (!rope_args_ok(eps, rope_theta) || T < 1) return DMA_ERR_INVALID_ARG;
  dma_status_t st = check_heads(Hq, Hkv, d);
  if (st != DMA_OK) return st;
  if (!stride_ok(q_stride, Hq, d) || !stride_ok(k_stride, Hkv, d) || !stride_ok(v_stride, Hkv, d))
    return DMA_ERR_INVALID_ARG;
  if ((st = check_pages(B, max_pages, num_pages, page_size, page_stride, Hkv, d)) != DMA_OK) return st;
  if (static_cast<long long>(T) * Hq >= (1LL << 31)) return DMA_ERR_UNSUPPORTED;
  if (ws_bytes < kHeaderBytes) return DMA_ERR_WORKSPACE;
  if ((st = device_ok()) != DMA_OK) return st;
  const AppendPaged p{q,       k,         v,          q_stride,   k_stride,    v_stride, q_norm_w, k_norm_w,
                      W_dt,    A,         cu_tokens,  positions,  page_table,  q_out,    k_out,    k_pages,
                      v_pages, dt_pages,  page_stride, eps,       rope_theta,  T,        B,        max_pages,
                      num_pages, page_size, Hq,       Hkv,        d};
  const cudaError_t e = launch_append_paged(p, static_cast<uint32_t*>(workspace), reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DMA_OK : cuda_fail(e);
}

size_t dma_decode_paged_workspace_size(int B, int max_pages, int page_size, int Hq, int Hkv, int d,
                                       int keep_window_size, int window, int sinks) {
  if (check_paged_decode(B, max_pages, page_size, Hq, Hkv, d, keep_window_size, window, sinks) != DMA_OK) return 0;
  return paged_workspace(B, max_pages, page_size, Hq, Hkv, d, keep_window_size, window, sinks).bytes;
}

dma_status_t dma_decode_paged(const void* q, const void* k_pages, const void* v_pages, const float* dt_pages,
                              const int32_t* page_table, const int32_t* lengths, int B, int max_pages, int num_pages,
                              int page_size, int64_t page_stride, int Hq, int Hkv, int d, int keep_window_size,
                              int window, int sinks, float scale, void* out, void* workspace, size_t ws_bytes,
                              dma_stream_t stream) {
  if (!ready(q, k_pages, v_pages, dt_pages, page_table, lengths, out, workspace)) return DMA_ERR_INVALID_ARG;
  if (!(scale == scale) || scale > 3.0e38f || scale < -3.0e38f) return DMA_ERR_INVALID_ARG;
  dma_status_t st = check_paged_decode(B, max_pages, page_size, Hq, Hkv, d, keep_window_size, window, sinks);
  if (st != DMA_OK) return st;
  if ((st = check_pages(B, max_pages, num_pages, page_size, page_stride, Hkv, d)) != DMA_OK) return st;
  const PagedWorkspace wsl = paged_workspace(B, max_pages, page_size, Hq, Hkv, d, keep_window_size, window, sinks);
  if (ws_bytes < wsl.bytes) return DMA_ERR_WORKSPACE;
  if ((st = device_ok()) != DMA_OK) return st;
  char* ws = static_cast<char*>(workspace);
  PagedCache c;
  c.dt_pages = dt_pages;
  c.table = page_table;
  c.lengths = lengths;
  c.page_stride16 = page_stride / 8;
  c.B = B;
  c.max_pages = max_pages;
  c.num_pages = num_pages;
  c.page_size = page_size;
  c.page_shift = -1;
  c.page_inv = 1.0f / static_cast<float>(page_size);
  for (int i = 0; i <= 20; ++i)
    if (page_size == 1 << i) c.page_shift = i;
  c.Hkv = Hkv;
  c.d = d;
  c.w = keep_window_size;
  c.window = std::min(window, kMaxLen);   // a longer one reaches every key, like kMaxLen
  c.sinks = window > 0 ? std::min(sinks, kMaxLen) : 0;
  c.longest = static_cast<int>(visible_cap(max_pages, page_size, window, sinks));
  c.err = reinterpret_cast<uint32_t*>(ws);
  PagedLists lists{nullptr, nullptr, 0};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (wsl.cap > 0) {
    lists = PagedLists{reinterpret_cast<int32_t*>(ws + wsl.pos), reinterpret_cast<float*>(ws + wsl.bias), wsl.cap};
    if ((e = launch_select_paged(c, lists, s)) != cudaSuccess) return cuda_fail(e);
  }
  e = launch_attn_paged(c, lists, q, k_pages, v_pages, Hq, scale, ws + wsl.scratch, out, s);
  return e == cudaSuccess ? DMA_OK : cuda_fail(e);
}

size_t dma_prologue_backward_workspace_size(int B, int L, int Hq, int Hkv, int d) {
  if (B < 1 || L < 1 || check_heads(Hq, Hkv, d) != DMA_OK) return 0;
  if (static_cast<long long>(B) * L * Hq >= (1LL << 31)) return 0;
  return kHeaderBytes + prologue_backward_scratch_bytes(d);
}

dma_status_t dma_prologue_backward(const void* q, const void* k, int64_t q_stride, int64_t k_stride,
                                   const float* q_norm_w, const float* k_norm_w, float eps, float rope_theta,
                                   const int32_t* positions, const void* dq_out, const void* dk_out, int B, int L,
                                   int Hq, int Hkv, int d, void* dq, void* dk, int64_t dq_stride, int64_t dk_stride,
                                   float* dq_norm_w, float* dk_norm_w, void* workspace, size_t ws_bytes,
                                   dma_stream_t stream) {
  if (!ready(q, k, q_norm_w, k_norm_w, positions, dq_out, dk_out, dq, dk, dq_norm_w, dk_norm_w, workspace))
    return DMA_ERR_INVALID_ARG;
  if (!rope_args_ok(eps, rope_theta) || B < 1 || L < 1) return DMA_ERR_INVALID_ARG;
  dma_status_t st = check_heads(Hq, Hkv, d);
  if (st != DMA_OK) return st;
  if (!stride_ok(q_stride, Hq, d) || !stride_ok(k_stride, Hkv, d) || !stride_ok(dq_stride, Hq, d) ||
      !stride_ok(dk_stride, Hkv, d))
    return DMA_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * L * Hq >= (1LL << 31)) return DMA_ERR_UNSUPPORTED;
  if (ws_bytes < dma_prologue_backward_workspace_size(B, L, Hq, Hkv, d)) return DMA_ERR_WORKSPACE;
  if ((st = device_ok()) != DMA_OK) return st;
  uint32_t* header = static_cast<uint32_t*>(workspace);
  float* part = reinterpret_cast<float*>(static_cast<char*>(workspace) + kHeaderBytes);
  const PrologueBackward p{q,         k,         q_stride,  k_stride,  q_norm_w,   k_norm_w,
                           positions, dq_out,    dk_out,    dq,        dk,         dq_stride,
                           dk_stride, dq_norm_w, dk_norm_w, part,      header + kHdrPbWord,
                           eps,       rope_theta, B,        L,         Hq,         Hkv,       d};
  const cudaError_t e = launch_prologue_backward(p, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DMA_OK : cuda_fail(e);
}

}  // extern "C"
