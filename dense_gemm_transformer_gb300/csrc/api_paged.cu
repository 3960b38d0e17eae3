// api_paged.cu -- the C ABI of the operators on a paged cache (gemm.h):
// argument checks, scratch and launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>
#include <new>

#include "gemm.h"
#include "handle.h"
#include "kernels.h"

namespace {

constexpr int64_t kMaxInt = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxPages = int64_t(1) << 30;
constexpr int64_t kMaxTileParts = int64_t(1) << 24;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool known_type(int t) { return t == GEMM_TYPE_FP32 || t == GEMM_TYPE_BF16 || t == GEMM_TYPE_FP16; }
size_t type_bytes(int t) { return t == GEMM_TYPE_FP32 ? 4 : 2; }
gemm_status_t cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return GEMM_OK;
  cudaGetLastError();
  return GEMM_ERR_CUDA;
}

// The handle's device must be the current one: launches, attributes and
// allocations go to that.
gemm_status_t check_device(gemm_handle_t h) {
  int device;
  const cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return cuda_status(e);
  return device == h->device ? GEMM_OK : GEMM_ERR_INVALID_VALUE;
}

gemm_status_t check_rotary(const gemm_rotary_t& a) {
  if (!known_type(a.in_type) || !known_type(a.out_type)) return GEMM_ERR_INVALID_VALUE;
  if ((a.interleaved | a.inverse) & ~1) return GEMM_ERR_INVALID_VALUE;
  if (a.heads < 0 || a.kv_heads < 0 || a.head_dim < 2 || a.head_dim % 2 != 0 || a.rotary_dim < 0 ||
      a.rotary_dim > a.head_dim || a.rotary_dim % 2 != 0 || a.tokens < 0 || a.page_size < 0)
    return GEMM_ERR_INVALID_VALUE;
  if (a.heads > 65535 || a.kv_heads > 65535 || a.tokens > kMaxInt) return GEMM_ERR_INVALID_VALUE;
  if (a.head_dim > 512) return GEMM_ERR_NOT_SUPPORTED;  // a block's threads take whole heads
  if (!std::isfinite(a.amplitude)) return GEMM_ERR_INVALID_VALUE;
  if (a.rotary_dim > 0 && a.position_bytes != 4 && a.position_bytes != 8) return GEMM_ERR_INVALID_VALUE;
  const bool paged = a.page_size > 0;
  if (paged && (a.num_pages < 0 || a.num_pages > kMaxPages)) return GEMM_ERR_INVALID_VALUE;
  if (a.tokens == 0) return GEMM_OK;  // (a tensor without elements has no address)
  if (paged && (a.k == nullptr || a.v == nullptr)) return GEMM_ERR_INVALID_VALUE;
  if (!paged && a.v != nullptr) return GEMM_ERR_INVALID_VALUE;
  if (a.heads == 0 && (a.k == nullptr || a.kv_heads == 0)) return GEMM_OK;
  if (a.heads > 0 && (a.q == nullptr || a.q_out == nullptr)) return GEMM_ERR_INVALID_VALUE;
  if (a.k != nullptr && a.k_out == nullptr) return GEMM_ERR_INVALID_VALUE;
  if (paged && (a.v_out == nullptr || a.slots == nullptr)) return GEMM_ERR_INVALID_VALUE;
  if (a.rotary_dim > 0 && (a.positions == nullptr || a.freqs == nullptr)) return GEMM_ERR_INVALID_VALUE;
  const size_t in = type_bytes(a.in_type), out = type_bytes(a.out_type);
  if (!aligned(a.q, in) || !aligned(a.k, in) || !aligned(a.v, in) || !aligned(a.q_out, out) ||
      !aligned(a.k_out, out) || !aligned(a.v_out, out) || !aligned(a.freqs, 8) || !aligned(a.slots, 8) ||
      (a.rotary_dim > 0 && !aligned(a.positions, static_cast<size_t>(a.position_bytes))))
    return GEMM_ERR_MISALIGNED;
  return GEMM_OK;
}

gemm_status_t check_attention(const gemm_paged_attention_t& a) {
  if (a.type != GEMM_TYPE_BF16 && a.type != GEMM_TYPE_FP16) return GEMM_ERR_INVALID_VALUE;
  if (a.sequences < 0 || a.heads < 1 || a.kv_heads < 1 || a.heads % a.kv_heads != 0 || a.heads > 32768 ||
      a.head_dim < 1 || a.page_size < 1 || a.table_width < 0 || a.window < 0 || a.max_q < 0 || a.tokens < 0 ||
      a.num_pages < 0 || a.max_kv < 0)
    return GEMM_ERR_INVALID_VALUE;
  if (a.tokens > kMaxInt || a.num_pages > kMaxPages ||
      static_cast<int64_t>(a.table_width) * a.page_size > kMaxInt - 65536)
    return GEMM_ERR_INVALID_VALUE;
  if (!std::isfinite(a.scale) || !std::isfinite(a.softcap) || a.softcap < 0.f) return GEMM_ERR_INVALID_VALUE;
  if (a.cu_q == nullptr && a.tokens != a.sequences) return GEMM_ERR_INVALID_VALUE;
  if ((a.head_dim != 64 && a.head_dim != 128) || a.page_size % 16 != 0) return GEMM_ERR_NOT_SUPPORTED;
  if (a.tokens == 0 || a.sequences == 0) return GEMM_OK;
  if (a.max_q < 1 || a.q == nullptr || a.out == nullptr || a.kv_lens == nullptr) return GEMM_ERR_INVALID_VALUE;
  if (a.table_width > 0 && (a.table == nullptr || (a.num_pages > 0 && (a.k_pages == nullptr || a.v_pages == nullptr))))
    return GEMM_ERR_INVALID_VALUE;
  if (!aligned(a.q, 16) || !aligned(a.out, 16) || !aligned(a.k_pages, 16) || !aligned(a.v_pages, 16) ||
      !aligned(a.table, 4) || !aligned(a.kv_lens, 4) || !aligned(a.cu_q, 4) || !aligned(a.lse, 4))
    return GEMM_ERR_MISALIGNED;
  if ((a.q_token | a.q_head | a.out_token | a.out_head | a.k_page | a.k_slot | a.k_head | a.v_page | a.v_slot |
       a.v_head) % 8 != 0)
    return GEMM_ERR_MISALIGNED;
  if (a.out == a.q) return GEMM_ERR_INVALID_VALUE;  // rows with results that are not finite are computed again
  return GEMM_OK;
}

gemm_status_t check_cache(gemm_handle_t h, const gemm_cache_t* c, int64_t n, bool pools) {
  if (h == nullptr || c == nullptr || n < 0 || n > kMaxInt) return GEMM_ERR_INVALID_VALUE;
  if (c->sequences < 0 || c->table_width < 0 || c->page_size < 1 || c->num_pages < 0 || c->num_pages > kMaxPages ||
      c->pool_count < 0 || c->pool_count > 8 ||
      static_cast<int64_t>(c->table_width) * c->page_size > kMaxInt - 65536)
    return GEMM_ERR_INVALID_VALUE;
  if (!pools || c->pool_count == 0) return GEMM_OK;
  if (c->page_bytes < 0 || c->page_bytes > kMaxInt) return GEMM_ERR_INVALID_VALUE;
  if (c->page_bytes % 16 != 0) return GEMM_ERR_MISALIGNED;
  int64_t groups = 0;
  for (int i = 0; i < c->pool_count; ++i) {
    const int64_t n = c->pool_groups[i];
    if (n < 0 || n > 65535 || (c->pools[i] == nullptr && n > 0 && c->num_pages > 0)) return GEMM_ERR_INVALID_VALUE;
    if (!aligned(c->pools[i], 16) || c->pool_group_stride[i] % 16 != 0 || c->pool_page_stride[i] % 16 != 0)
      return GEMM_ERR_MISALIGNED;
    groups += n;
  }
  // a warp's pieces of all groups of one page are counted in 32 bits
  if (groups * (c->page_bytes / 4096 + 1) > kMaxInt) return GEMM_ERR_INVALID_VALUE;
  return GEMM_OK;
}

gemm_status_t check_state(const gemm_cache_t& c, bool lens) {
  if ((c.num_pages > 0 && c.refs == nullptr) || (c.sequences > 0 && c.table_width > 0 && c.table == nullptr) ||
      (lens && c.sequences > 0 && c.lens == nullptr))
    return GEMM_ERR_INVALID_VALUE;
  if (!aligned(c.table, 4) || !aligned(c.lens, 4) || !aligned(c.refs, 4)) return GEMM_ERR_MISALIGNED;
  return GEMM_OK;
}

// A new device block of `bytes` zeros.
gemm_status_t zeroed_block(void** block, size_t bytes) {
  // a stream of its own for the zeros: the caller's may not wait for the
  // default one, or may be recording a graph, which the zeros are no part of
  cudaStream_t stream;
  void* p = nullptr;
  if (cudaMalloc(&p, bytes) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_ALLOC;
  }
  cudaError_t e = cudaStreamCreateWithFlags(&stream, cudaStreamNonBlocking);
  if (e == cudaSuccess) {
    e = cudaMemsetAsync(p, 0, bytes, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    cudaStreamDestroy(stream);
  }
  if (e != cudaSuccess) {
    cudaFree(p);
    return cuda_status(e);
  }
  *block = p;
  return GEMM_OK;
}

// The smallest block that holds `bytes` of the handle's scratch for `stream`
// (block i has 2^i MiB); `blocks`: which of it.
gemm_status_t scratch_of(gemm_handle_t h, void* (dgt::StreamScratch::*blocks)[dgt::kScratchBlocks], void* stream,
                         size_t bytes, void** out) {
  int i = 0;
  while ((size_t(1) << (20 + i)) < bytes) ++i;
  if (i >= dgt::kScratchBlocks) return GEMM_ERR_ALLOC;
  unsigned long long id = reinterpret_cast<uintptr_t>(stream);
  cudaStreamCaptureStatus state;
  cudaError_t e = cudaStreamIsCapturing(static_cast<cudaStream_t>(stream), &state);
  const bool captured = e == cudaSuccess && state != cudaStreamCaptureStatusNone;
  if (e == cudaSuccess && !captured) e = cudaStreamGetId(static_cast<cudaStream_t>(stream), &id);
  if (e != cudaSuccess) return cuda_status(e);
  std::lock_guard<std::mutex> lock(h->paged_lock);
  dgt::StreamScratch* s = h->paged_scratch;
  while (s != nullptr && (s->stream != id || s->captured != captured)) s = s->next;
  if (s == nullptr) {
    s = new (std::nothrow) dgt::StreamScratch{};
    if (s == nullptr) return GEMM_ERR_ALLOC;
    s->stream = id;
    s->captured = captured;
    s->next = h->paged_scratch;
    h->paged_scratch = s;
  }
  void** block = &(s->*blocks)[i];
  gemm_status_t st = GEMM_OK;
  if (*block == nullptr) {
    // (while a stream is being captured, only a thread in this mode may allocate)
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    cudaThreadExchangeStreamCaptureMode(&mode);
    st = zeroed_block(block, size_t(1) << (20 + i));
    cudaThreadExchangeStreamCaptureMode(&mode);
  }
  *out = *block;
  return st;
}

}  // namespace

extern "C" {

gemm_status_t gemm_rotary(gemm_handle_t h, const gemm_rotary_t* a, void* stream) {
  if (h == nullptr || a == nullptr) return GEMM_ERR_INVALID_VALUE;
  gemm_status_t st = check_rotary(*a);
  if (st != GEMM_OK) return st;
  if (a->tokens == 0 || (a->heads == 0 && (a->k == nullptr || a->kv_heads == 0))) return GEMM_OK;
  st = check_device(h);
  if (st != GEMM_OK) return st;
  return cuda_status(dgt::launch_rotary(*a, h->sms, h->d_status, static_cast<cudaStream_t>(stream)));
}

gemm_status_t gemm_paged_attention(gemm_handle_t h, const gemm_paged_attention_t* given, void* stream) {
  if (h == nullptr || given == nullptr) return GEMM_ERR_INVALID_VALUE;
  gemm_status_t st = check_attention(*given);
  if (st != GEMM_OK) return st;
  if (given->tokens == 0 || given->sequences == 0) return GEMM_OK;
  st = check_device(h);
  if (st != GEMM_OK) return st;
  gemm_paged_attention_t bounded = *given;
  bounded.max_q = static_cast<int32_t>(std::min<int64_t>(bounded.max_q, bounded.tokens));
  const gemm_paged_attention_t* a = &bounded;
  // the 16-row kernel's blocks, (sequence, key head, 16 rows), in a 1-D grid
  const int64_t group = a->heads / a->kv_heads, rows = a->max_q * group;
  const int64_t row_tiles = ((group <= dgt::kPagedMostGroup ? std::min<int64_t>(rows, dgt::kPagedFewRows) : rows) + 15) / 16;
  if (static_cast<int64_t>(a->sequences) * a->kv_heads > kMaxInt / row_tiles) return GEMM_ERR_INVALID_VALUE;
  const dgt::PagedPlan plan = dgt::paged_attention_plan(*a, h->sms);
  if (plan.tile_parts > kMaxTileParts) return GEMM_ERR_INVALID_VALUE;
  void* ws;
  st = scratch_of(h, &dgt::StreamScratch::attn, stream, dgt::paged_scratch_bytes(plan, a->head_dim), &ws);
  if (st != GEMM_OK) return st;
  dgt::last_main_launch().valid = false;
  st = cuda_status(dgt::launch_paged_attention(*a, plan, ws, h->sms, static_cast<uint64_t>(h->opt_wait_us) * 1000u,
                                               h->d_status, static_cast<cudaStream_t>(stream)));
  if (st != GEMM_OK) return st;
  gemm_plan_t p{};
  p.family = GEMM_FAMILY_PAGED_ATTENTION;
  p.tile_m = plan.tile_rows;
  p.tile_n = plan.tile_keys;
  p.tile_k = a->head_dim;
  p.split_k = plan.splits;
  p.stages = plan.stages;
  p.grid = plan.grid;
  p.kernels = plan.kernels;
  std::lock_guard<std::mutex> lock(h->paged_lock);
  h->plan = p;
  h->null_shape = dgt::last_main_launch();
  return GEMM_OK;
}

gemm_status_t gemm_cache_grow(gemm_handle_t h, const gemm_cache_t* c, int64_t n, const int32_t* seqs,
                              const int32_t* counts, int64_t tokens, int64_t* positions, int64_t* slots,
                              int32_t* info, void* stream) {
  gemm_status_t st = check_cache(h, c, n, true);
  if (st == GEMM_OK) st = check_state(*c, true);
  if (st != GEMM_OK) return st;
  if (info == nullptr || tokens < 0 || tokens > kMaxInt || (n > 0 && (seqs == nullptr || counts == nullptr)))
    return GEMM_ERR_INVALID_VALUE;
  if (!aligned(seqs, 4) || !aligned(counts, 4) || !aligned(info, 4) || !aligned(positions, 8) || !aligned(slots, 8))
    return GEMM_ERR_MISALIGNED;
  st = check_device(h);
  if (st != GEMM_OK) return st;
  void* ws;
  st = scratch_of(h, &dgt::StreamScratch::cache, stream, dgt::cache_scratch_bytes(c->num_pages, n), &ws);
  if (st != GEMM_OK) return st;
  return cuda_status(dgt::launch_cache_grow(*c, n, seqs, counts, tokens, positions, slots, info, ws, h->sms,
                                            h->d_status, static_cast<cudaStream_t>(stream)));
}

gemm_status_t gemm_cache_shrink(gemm_handle_t h, const gemm_cache_t* c, int64_t n, const int32_t* seqs,
                                const int32_t* counts, void* stream) {
  gemm_status_t st = check_cache(h, c, n, false);
  if (st == GEMM_OK) st = check_state(*c, true);
  if (st != GEMM_OK) return st;
  if (n == 0) return GEMM_OK;
  if (seqs == nullptr) return GEMM_ERR_INVALID_VALUE;
  if (!aligned(seqs, 4) || !aligned(counts, 4)) return GEMM_ERR_MISALIGNED;
  st = check_device(h);
  if (st != GEMM_OK) return st;
  return cuda_status(dgt::launch_cache_shrink(*c, n, seqs, counts, h->d_status, static_cast<cudaStream_t>(stream)));
}

gemm_status_t gemm_cache_fork(gemm_handle_t h, const gemm_cache_t* c, int64_t n, const int32_t* parents,
                              const int32_t* children, int32_t* copied, int32_t* info, void* stream) {
  gemm_status_t st = check_cache(h, c, n, true);
  if (st == GEMM_OK) st = check_state(*c, true);
  if (st != GEMM_OK) return st;
  if (info == nullptr || (n > 0 && (parents == nullptr || children == nullptr || copied == nullptr)))
    return GEMM_ERR_INVALID_VALUE;
  if (!aligned(parents, 4) || !aligned(children, 4) || !aligned(copied, 4) || !aligned(info, 4))
    return GEMM_ERR_MISALIGNED;
  st = check_device(h);
  if (st != GEMM_OK) return st;
  void* ws;
  st = scratch_of(h, &dgt::StreamScratch::cache, stream, dgt::cache_scratch_bytes(c->num_pages, n), &ws);
  if (st != GEMM_OK) return st;
  return cuda_status(dgt::launch_cache_fork(*c, n, parents, children, copied, info, ws, h->sms, h->d_status,
                                            static_cast<cudaStream_t>(stream)));
}

gemm_status_t gemm_cache_compact(gemm_handle_t h, const gemm_cache_t* c, int32_t* info, void* stream) {
  gemm_status_t st = check_cache(h, c, 0, true);
  if (st == GEMM_OK) st = check_state(*c, false);
  if (st != GEMM_OK) return st;
  if (info == nullptr) return GEMM_ERR_INVALID_VALUE;
  if (!aligned(info, 4)) return GEMM_ERR_MISALIGNED;
  st = check_device(h);
  if (st != GEMM_OK) return st;
  void* ws;
  st = scratch_of(h, &dgt::StreamScratch::cache, stream, dgt::cache_scratch_bytes(c->num_pages, 0), &ws);
  if (st != GEMM_OK) return st;
  return cuda_status(
      dgt::launch_cache_compact(*c, info, ws, h->sms, h->d_status, static_cast<cudaStream_t>(stream)));
}

gemm_status_t gemm_cache_copy(gemm_handle_t h, const gemm_cache_t* c, int64_t n, const int32_t* src,
                              const int32_t* dst, void* stream) {
  gemm_status_t st = check_cache(h, c, n, true);
  if (st != GEMM_OK) return st;
  if (n == 0) return GEMM_OK;
  if (src == nullptr || dst == nullptr) return GEMM_ERR_INVALID_VALUE;
  if (!aligned(src, 4) || !aligned(dst, 4)) return GEMM_ERR_MISALIGNED;
  st = check_device(h);
  if (st != GEMM_OK) return st;
  return cuda_status(
      dgt::launch_cache_copy(*c, n, src, dst, h->sms, h->d_status, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
