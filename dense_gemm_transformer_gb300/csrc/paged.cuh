// paged.cuh -- what the two kernels of the attention over a paged cache share:
// their parameters, the sequences' bounds, the scores.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>
#include <type_traits>

#include "kernels.h"
#include "ptx.cuh"

namespace dgt {

struct PagedParams {
  gemm_paged_attention_t a;
  int group;       // query heads a key head
  uint32_t group_inv;  // ceil(2^32 / group): x / group = umulhi(x, group_inv) for x, group < 2^16
  // scale log2(e); with a softcap c: scale / c, and c log2(e); with one of at
  // most kCapShared (cap_shared) also 2 log2(e) scale / c
  float scale_log2, cap_in, cap_out, cap_in2;
  int cap_shared;
  int* status;
  // The kernel of 16 rows a block takes the sequences with at most
  // `few_rows` rows a key head; the tile kernel the others (tiled != 0).
  int tiled, few_rows;
  // 16-row kernel
  int row_tiles;   // blocks of 16 rows a (sequence, key head)
  int splits;      // most parts of a range
  int tiles_per;   // key tiles a part
  int row_stages;  // tiles in a warp's ring of the 16-row kernel
  int units;       // (sequence, key head, row tile, part)
  float* part;     // partial results: 16 x D sums, then 16 maxima, 16 sums
  int* arrived;    // parts of a range that are written
  int* queue;      // beside the tile kernel: units taken, blocks that have found none left; its items
  // tile kernel
  int tile_tokens;   // tokens a 128-row tile: 128 / group
  int tile_splits;   // parts of an item's keys
  int tile_parts;    // room for parts of items
  int box;           // keys a copy: the largest power of two that divides page_size, at most 128
  float* tile_part;  // per part 256 x D sums, 256 maxima, 256 sums (tile_splits > 1)
  float s_scale;     // what makes a score of s: the scale's magnitude, c, or 2 c with cap_shared
  int flip;          // a negative scale without a cap
  uint8_t* redo;     // per part and softmax warp: a result is not finite
  uint64_t wait_ns;
  int out_v8;        // rows of out are 32-byte aligned
};

__device__ __forceinline__ int by_group(const PagedParams& p, int x) {
  return p.group == 1 ? x : static_cast<int>(__umulhi(static_cast<uint32_t>(x), p.group_inv));
}

// A sequence of the call: its first new token, how many, and its keys,
// brought into range (reported, then n or len 0 or the most there can be).
struct PagedSeq {
  int64_t first;
  int n, len;
};
__device__ __forceinline__ PagedSeq paged_seq(const PagedParams& p, int seq, bool report) {
  const gemm_paged_attention_t& a = p.a;
  PagedSeq s{seq, 1, a.kv_lens[seq]};
  if (a.cu_q != nullptr) {
    s.first = a.cu_q[seq];
    const int64_t n = static_cast<int64_t>(a.cu_q[seq + 1]) - s.first;
    const bool bad = s.first < 0 || n < 0 || s.first + n > a.tokens;
    if ((bad || n > a.max_q) && report) atomicExch(p.status, kDevBadIndex);
    s.n = bad ? 0 : static_cast<int>(n);
  }
  const int64_t most = static_cast<int64_t>(a.table_width) * a.page_size;
  if (s.len < 0 || s.len > most) {
    if (report) atomicExch(p.status, kDevBadIndex);
    s.len = s.len < 0 ? 0 : static_cast<int>(most);
  }
  return s;
}

__device__ __forceinline__ float as_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float as_f(__half x) { return __half2float(x); }
// Two values as one register of 16-bit elements, `lo` in the low half.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if constexpr (std::is_same_v<T, __nv_bfloat16>)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <typename T>
__device__ __forceinline__ void unpack2(uint32_t r, float& lo, float& hi) {
  T x[2];
  memcpy(x, &r, 4);
  lo = as_f(x[0]);
  hi = as_f(x[1]);
}

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The largest cap for which the kernels take tanh(x) as 1 - 2 / (e^{2x} + 1).
// That cancels for small x and is off by some 2^-23, which the cap makes 2^-23
// c of a score (a CPU emulation in fp32: 8e-6 with c = 50, 1e-3 with 10^4).  Up
// to here that is 2^-17, of the order of the products' own error for scores
// near the cap, and 64 times less than what the rounding of the weights to 16
// bits costs.
constexpr float kCapShared = 64.f;
// A larger cap is none: a score would have to pass 2^88 for it to make a
// difference in fp32 (c tanh(s / c) is s (1 - (s / c)^2 / 3 + ...)).
constexpr float kCapNone = 0x1p100f;

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

// scale s in units of log2, through the cap where there is one.  (tanhf for
// every cap took 66.5 us for 63.5 for one token in 64 sequences of 100 to 8300
// keys, 12 heads of 128 over 2.)
__device__ __forceinline__ float score_of(float s, const PagedParams& p) {
  if (p.cap_out == 0.f) return s * p.scale_log2;
  if (!p.cap_shared) return p.cap_out * tanhf(s * p.cap_in);
  return p.cap_out * (1.f - __fdividef(2.f, exp2_approx(s * p.cap_in2) + 1.f));
}

// An item of the tile kernel: two 128-row tiles of a (sequence, key head) and
// one part of their keys.  Items are numbered by sequence, and in a sequence
// the last tokens first (they see the most keys).
struct PagedItem {
  PagedSeq s;
  int seq, head, pair, split;
  int part;     // number of the item (not valid: how many there are)
  bool valid;
};
// The item `idx`, found by the whole warp; not valid beyond the last one.
__device__ __forceinline__ PagedItem paged_item(const PagedParams& p, int idx, bool report) {
  const int lane = threadIdx.x & 31;
  PagedItem it;
  it.valid = false;
  it.part = idx;
  int base = 0;
  for (int s0 = 0; s0 < p.a.sequences; s0 += 32) {
    const int seq = s0 + lane;
    PagedSeq s{0, 0, 0};
    if (seq < p.a.sequences) s = paged_seq(p, seq, report);
    const bool many = static_cast<int64_t>(s.n) * p.group > p.few_rows;
    const int pairs = many ? (s.n + 2 * p.tile_tokens - 1) / (2 * p.tile_tokens) : 0;
    const int per_pair = p.a.kv_heads * p.tile_splits;
    int incl = pairs * per_pair;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    const unsigned at = __ballot_sync(0xffffffffu, idx < base + incl);
    if (at != 0) {
      const int src = __ffs(at) - 1;
      it.seq = s0 + src;
      it.s.first = __shfl_sync(0xffffffffu, s.first, src);
      it.s.n = __shfl_sync(0xffffffffu, s.n, src);
      it.s.len = __shfl_sync(0xffffffffu, s.len, src);
      const int n_pairs = __shfl_sync(0xffffffffu, pairs, src);
      const int local = idx - base - (__shfl_sync(0xffffffffu, incl, src) - n_pairs * per_pair);
      it.pair = n_pairs - 1 - local / per_pair;
      const int rest = local % per_pair;
      it.head = rest / p.tile_splits;
      it.split = rest % p.tile_splits;
      it.valid = true;
      return it;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  it.part = base;
  return it;
}

cudaError_t launch_paged_tiles(const PagedParams& p, int grid, cudaStream_t stream);

}  // namespace dgt
