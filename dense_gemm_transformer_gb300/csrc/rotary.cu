// rotary.cu -- rotary positions of queries and keys, dense or with the keys
// and values written into the pages of a cache.
//
// Pair i of a head, (a, b), turns by the angle w = position * f_i:
//
//     a' = s (a cos w - b sin w),   b' = s (b cos w + a sin w)
//
// and by -w for the gradient (the transposed rotation).  The angle is taken
// modulo a turn before it becomes a float: f_i / 2 pi as a 64-bit fraction
// of a turn (one multiplication in double precision a frequency, rounded to
// 2^-53 of itself), times the position in integer arithmetic, which wraps at
// whole turns by itself and adds no error of its own at any position.  The
// fp32 product position * f_i would be off by position * f_i * 2^-24: a tenth
// of a turn near position 10^6.
//
// The kernel reads and writes each element once and is bound by that
// traffic.  A block has a few tokens: its threads compute their sines and
// cosines once (about 40 instructions a pair: per head they would cost as
// much time as the traffic) into shared memory, and then turn VEC pairs of a
// head at a time, few registers a thread and so many threads an SM with their
// loads in flight: 8192 tokens x 72 heads of 128 in bf16 took 90 us with the
// sines in registers and two blocks an SM, 55 us so.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"

namespace dgt {
namespace {

constexpr int kRotThreads = 256;
constexpr int kRotTokens = 64;   // most tokens of a block

struct RotaryParams {
  gemm_rotary_t a;
  int groups;          // units of a head: head_dim / (2 VEC)
  int rows;            // heads of q, k and v together
  int rows_per_block, tokens_per_block;
  int* status;
};

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f(float x) { return x; }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f(float x) { return __float2half_rn(x); }

// N consecutive elements in accesses of at most 16 bytes.
template <typename T, int N>
struct alignas(sizeof(T) * N < 16 ? sizeof(T) * N : 16) Vec {
  T x[N];
};

template <typename TI, typename TO, int VEC>
__global__ void __launch_bounds__(kRotThreads, 5) rotary_kernel(const __grid_constant__ RotaryParams p) {
  extern __shared__ float2 cs[];  // amplitude (cos, sin) of the block's tokens and pairs
  __shared__ int64_t k_at[kRotTokens], v_at[kRotTokens];  // where a token's key and value go, -1: nowhere
  grid_dep_wait();
  grid_dep_launch();
  const gemm_rotary_t& a = p.a;
  const int half = a.rotary_dim / 2;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.tokens_per_block;
  const int tokens = static_cast<int>(min(static_cast<int64_t>(p.tokens_per_block), a.tokens - t0));
  const int r0 = blockIdx.y * p.rows_per_block, rows = min(p.rows_per_block, p.rows - r0);
  using In = Vec<TI, VEC>;
  using Out = Vec<TO, VEC>;
  // A thread has VEC pairs, from p0 on, of every step-th (token, head) of the
  // block: elements ea.. and eb.. of the head, VEC each.  Paired halves for
  // turned pairs that are not interleaved; otherwise 2 VEC consecutive
  // elements.
  const int step = kRotThreads / p.groups, lane_row = threadIdx.x / p.groups;
  const int p0 = (threadIdx.x - lane_row * p.groups) * VEC;
  const bool turned = p0 < half, halves = turned && !a.interleaved;
  const int ea = halves ? p0 : 2 * p0, eb = halves ? p0 + half : 2 * p0 + VEC;
  const int step_t = step / rows, step_r = step - step_t * rows;
  struct Place {
    int t, r;  // token of the block, head of the block's
  };
  auto next = [&](Place& x) {
    x.t += step_t;
    x.r += step_r;
    if (x.r >= rows) {
      x.r -= rows;
      ++x.t;
    }
  };
  Place at{lane_row / rows, 0};
  at.r = lane_row - at.t * rows;
  if (lane_row >= step) at.t = tokens;  // threads beyond the last whole head
  In xa, xb;
  auto load = [&](const Place& x) {
    if (x.t >= tokens) return;
    const int64_t t = t0 + x.t;
    const int r = r0 + x.r;
    const TI* src = r < a.heads                ? static_cast<const TI*>(a.q) + t * a.q_token + r * a.q_head
                    : r < a.heads + a.kv_heads ? static_cast<const TI*>(a.k) + t * a.k_token + (r - a.heads) * a.k_head
                                               : static_cast<const TI*>(a.v) + t * a.v_token +
                                                     (r - a.heads - a.kv_heads) * a.v_head;
    xa = *reinterpret_cast<const In*>(src + ea);
    xb = *reinterpret_cast<const In*>(src + eb);
  };
  load(at);  // in flight while the angles are computed
  uint64_t* turns = reinterpret_cast<uint64_t*>(cs + p.tokens_per_block * half);  // f_i / 2 pi in units of 2^-64 turn
  for (int i = threadIdx.x; i < half; i += kRotThreads) {
    double f = a.freqs[i] * 0.15915494309189533577;  // 1 / (2 pi)
    f -= floor(f);
    turns[i] = __double2ull_rz(f * 18446744073709551616.0);  // an f of 1 saturates to the nearest fraction
  }
  __syncthreads();
  for (int i = threadIdx.x; i < tokens * half; i += kRotThreads) {
    const int t = i / half;
    const int64_t pos = a.position_bytes == 8 ? static_cast<const int64_t*>(a.positions)[t0 + t]
                                              : static_cast<const int32_t*>(a.positions)[t0 + t];
    const int64_t w = static_cast<int64_t>(static_cast<uint64_t>(pos) * turns[i - t * half]);  // in [-1/2, 1/2) turn
    float sn, cn;
    sincospif(static_cast<float>(w) * 0x1p-63f, &sn, &cn);
    cs[i] = make_float2(cn * a.amplitude, (a.inverse ? -sn : sn) * a.amplitude);
  }
  for (int t = threadIdx.x; t < tokens; t += kRotThreads) {
    int64_t k_to = (t0 + t) * a.k_out_token, v_to = 0;
    if (a.page_size > 0) {
      const int64_t slot = a.slots[t0 + t];
      k_to = v_to = -1;
      if (slot >= a.num_pages * a.page_size) {
        atomicExch(p.status, kDevBadIndex);
      } else if (slot >= 0) {
        const int64_t page = slot / a.page_size, at = slot - page * a.page_size;
        k_to = page * a.k_out_page + at * a.k_out_token;
        v_to = page * a.v_out_page + at * a.v_out_token;
      }
    }
    k_at[t] = k_to;
    v_at[t] = v_to;
  }
  __syncthreads();
  for (bool first = true; at.t < tokens; first = false, next(at)) {
    if (!first) load(at);
    const int r = r0 + at.r;
    TO* dst;
    if (r < a.heads) {
      dst = static_cast<TO*>(a.q_out) + (t0 + at.t) * a.q_out_token + r * a.q_out_head;
    } else {
      const bool key = r < a.heads + a.kv_heads;
      const int64_t to = key ? k_at[at.t] : v_at[at.t];
      if (to < 0 && a.page_size > 0) continue;
      dst = key ? static_cast<TO*>(a.k_out) + to + (r - a.heads) * a.k_out_head
                : static_cast<TO*>(a.v_out) + to + (r - a.heads - a.kv_heads) * a.v_out_head;
    }
    Out ya, yb;
    const float2* w = cs + at.t * half + p0;
    if (!turned || r >= a.heads + a.kv_heads) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        ya.x[j] = from_f<TO>(to_f(xa.x[j]));
        yb.x[j] = from_f<TO>(to_f(xb.x[j]));
      }
    } else if (VEC == 1 || halves) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float e = to_f(xa.x[j]), o = to_f(xb.x[j]);
        ya.x[j] = from_f<TO>(e * w[j].x - o * w[j].y);
        yb.x[j] = from_f<TO>(o * w[j].x + e * w[j].y);
      }
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        // pair j: elements 2 j and 2 j + 1 of the 2 VEC
        const float e = to_f(2 * j < VEC ? xa.x[(2 * j) % VEC] : xb.x[(2 * j) % VEC]);
        const float o = to_f(2 * j + 1 < VEC ? xa.x[(2 * j + 1) % VEC] : xb.x[(2 * j + 1) % VEC]);
        (2 * j < VEC ? ya : yb).x[(2 * j) % VEC] = from_f<TO>(e * w[j].x - o * w[j].y);
        (2 * j + 1 < VEC ? ya : yb).x[(2 * j + 1) % VEC] = from_f<TO>(o * w[j].x + e * w[j].y);
      }
    }
    *reinterpret_cast<Out*>(dst + ea) = ya;
    *reinterpret_cast<Out*>(dst + eb) = yb;
  }
}

template <typename TI, typename TO, int VEC>
cudaError_t launch(const gemm_rotary_t& a, int sms, int* status, cudaStream_t stream) {
  RotaryParams p;
  p.a = a;
  p.groups = a.head_dim / (2 * VEC);
  p.rows = a.heads + (a.k != nullptr ? a.kv_heads : 0) + (a.v != nullptr ? a.kv_heads : 0);
  p.status = status;
  // A block's tokens: about eight units a thread over all heads, and sines
  // that fit 32 KB.  With few tokens the heads are shared out over blocks,
  // down to one unit a thread (latency counts, and the sines are computed in
  // parallel), until there are four blocks an SM: eight measured 2 us less on
  // 8192 tokens of 72 heads of 128, 2 us more on 16384 of 18 heads of 64.
  constexpr int kUnits = 8;
  const int64_t token_units = static_cast<int64_t>(p.rows) * p.groups;
  const int half = a.rotary_dim / 2;
  int64_t tokens = std::max<int64_t>(1, std::min<int64_t>(kRotTokens, kUnits * kRotThreads / token_units));
  if (half > 0) tokens = std::max<int64_t>(1, std::min<int64_t>(tokens, 4096 / half));
  const int64_t want = 4 * static_cast<int64_t>(sms);
  while (tokens > 1 && (a.tokens + tokens - 1) / tokens < want) tokens /= 2;
  const int64_t blocks = (a.tokens + tokens - 1) / tokens;
  const int64_t least = std::max<int64_t>(1, kRotThreads / p.groups);  // heads that give every thread a unit
  int64_t per = std::max<int64_t>(1, std::min<int64_t>(p.rows, kUnits * kRotThreads / p.groups));
  while (per > least && blocks * ((p.rows + per - 1) / per) < want) per = (per + 1) / 2;
  p.tokens_per_block = static_cast<int>(tokens);
  p.rows_per_block = static_cast<int>(per);
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((p.rows + per - 1) / per));
  return launch_pdl(rotary_kernel<TI, TO, VEC>, grid, dim3(kRotThreads),
                    tokens * half * sizeof(float2) + half * sizeof(uint64_t), stream, p);
}

template <typename TI, typename TO>
cudaError_t launch_types(const gemm_rotary_t& a, int sms, int* status, cudaStream_t stream) {
  // Eight pairs a thread of 16-bit inputs (16 bytes a load), four of 32-bit
  // ones, where every base and stride is a whole number of as many elements;
  // else four, or one.
  const int64_t in = a.q_token | a.q_head | a.k_token | a.k_head | a.v_token | a.v_head;
  const int64_t out = a.q_out_token | a.q_out_head | a.k_out_page | a.k_out_token | a.k_out_head | a.v_out_page |
                      a.v_out_token | a.v_out_head;
  const uintptr_t ip = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k) |
                       reinterpret_cast<uintptr_t>(a.v);
  const uintptr_t op = reinterpret_cast<uintptr_t>(a.q_out) | reinterpret_cast<uintptr_t>(a.k_out) |
                       reinterpret_cast<uintptr_t>(a.v_out);
  auto whole = [&](int vec) {
    return (in | out) % vec == 0 && ip % std::min<size_t>(vec * sizeof(TI), 16) == 0 &&
           op % std::min<size_t>(vec * sizeof(TO), 16) == 0 && a.head_dim % (2 * vec) == 0 &&
           a.rotary_dim % (2 * vec) == 0;
  };
  if constexpr (sizeof(TI) == 2)
    if (whole(8)) return launch<TI, TO, 8>(a, sms, status, stream);
  if (whole(4)) return launch<TI, TO, 4>(a, sms, status, stream);
  return launch<TI, TO, 1>(a, sms, status, stream);
}

}  // namespace

cudaError_t launch_rotary(const gemm_rotary_t& a, int sms, int* status, cudaStream_t stream) {
  using bf16 = __nv_bfloat16;
  if (a.in_type == GEMM_TYPE_FP32) {
    if (a.out_type == GEMM_TYPE_FP32) return launch_types<float, float>(a, sms, status, stream);
    if (a.out_type == GEMM_TYPE_BF16) return launch_types<float, bf16>(a, sms, status, stream);
    return launch_types<float, __half>(a, sms, status, stream);
  }
  if (a.in_type == GEMM_TYPE_BF16) {
    if (a.out_type == GEMM_TYPE_FP32) return launch_types<bf16, float>(a, sms, status, stream);
    if (a.out_type == GEMM_TYPE_BF16) return launch_types<bf16, bf16>(a, sms, status, stream);
    return launch_types<bf16, __half>(a, sms, status, stream);
  }
  if (a.out_type == GEMM_TYPE_FP32) return launch_types<__half, float>(a, sms, status, stream);
  if (a.out_type == GEMM_TYPE_BF16) return launch_types<__half, bf16>(a, sms, status, stream);
  return launch_types<__half, __half>(a, sms, status, stream);
}

}  // namespace dgt
