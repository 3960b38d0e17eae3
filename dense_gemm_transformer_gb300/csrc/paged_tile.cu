// paged_tile.cu -- attention of chunks of new tokens over a paged cache, on
// tcgen05 (the definition is in paged_attention.cu).
//
// An item is two tiles of 128 rows of a (sequence, key head) -- a row is a
// (token, head of the group) pair, 128 / group tokens a tile -- and its
// blocks of 128 keys: a block is 2 x 128 x 128 x D products for the scores
// and as many for the values, from 512 D bytes of cache that both tiles
// share, so it is bound by the tensor cores; the softmax of one tile runs
// while the tensor cores work on the other.  One block (CTA) an SM takes
// items in turn:
//
//   warp 0      loads: the queries of an item, and its keys and values block by
//               block into a ring of stages each, as 128-byte swizzled rows.
//               A page is not contiguous with the next one, so a copy is of
//               `box` keys (the largest power of two that divides the page
//               size, at most 128), whose pages the lanes have looked up.
//   warps 1, 2  one lane each issues S = Q K^T of tile 0 and 1, 64 keys at a
//               time into the tile's two S buffers in TMEM;
//   warps 3, 12 and O += P V, with P read from TMEM in place of the S it was
//               made from.  Four lanes because each loses as many cycles in
//               waits and commits as its instructions take: one lane for all
//               of it kept the tensor cores busy 55 % of a block, one a tile
//               65 % (both then waited at the same times).  Warp 3 also owns
//               the 512 columns of TMEM: per tile the S buffers and O.
//   warps 4-7   the softmax of tile 0, and 8-11 of tile 1: warp w has the 32
//               rows of TMEM lane quarter w % 4, one row a thread.  The
//               running maximum is raised, and O rescaled in TMEM, only where
//               a block's maximum exceeds it by more than kSlack (in log2):
//               until then the weights stay below 2^kSlack, which neither
//               their 16-bit form nor the fp32 sums lose accuracy by.
//
// A prompt of 8192 tokens, 64 heads of 128, takes 830 us (1.32 PFLOP/s, at the
// card's power limit).
//
// Slots past the sequence's last token may hold anything: their scores are
// masked by selection, and their values are overwritten with zeros in shared
// memory before the product.  A value that some rows see and others do not
// is in the product with weight 0 for the latter, where an infinity or NaN
// would still come through: an item whose sums are not finite is flagged, and
// the 16-row kernel, which runs beside this one and ends after it, computes
// its rows again without that.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <climits>
#include <cstdint>

#include "kernels.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace dgt {
namespace {

constexpr int kTileThreads = 416;
constexpr int kKeysBlock = 128;
constexpr int kHalfBytes = 128 * 128;  // 128 rows of 64 elements
constexpr float kSlack = 8.f;          // log2 of the largest weight under a maximum that was not raised

template <int D>
struct TileCfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kKStages = D == 128 ? 2 : 4, kVStages = D == 128 ? 3 : 4;  // K runs a block ahead of V
  static constexpr int kStages = kKStages + kVStages;
  static constexpr int kQBytes = 128 * D * 2;
  static constexpr int kStageBytes = 128 * D * 2;
  static constexpr int kBars = 2 * kStages + 23;
  static constexpr int kSmem = 2 * kQBytes + kStages * kStageBytes + 1024 + 8 * kBars + 16;
};

// fp16 weights are scaled by 2^7, so that small ones keep their accuracy:
// 2^(kSlack + 7) is still in range, and the factor cancels in O / l.
template <typename T>
__device__ __forceinline__ constexpr float weight_bias() { return std::is_same_v<T, __half> ? 7.f : 0.f; }

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t c0, int32_t c1,
                                            int32_t c2, int32_t c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], "
      "[%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// The whole warp waits; false for every lane when any lane gave up.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort, int* status, int code,
                                          uint64_t limit) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, status, code, limit));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ void st_global_v8(void* dst, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

__device__ __forceinline__ void tmem_ld_64(uint32_t addr, uint32_t (&s)[64]) {
  uint32_t a[32], b[32];
  tmem_ld_32x32b_x32(addr, a);
  tmem_ld_32x32b_x32(addr + 32, b);
  tmem_wait_ld();
#pragma unroll
  for (int t = 0; t < 32; ++t) {
    s[t] = a[t];
    s[32 + t] = b[t];
  }
}

__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The score of a key, in units of log2, is a s with a > 0.  Plain: s is the
// product (negated where the scale is negative, which is rare), a the scale.
// Capped by c, x = scale s / c: up to kCapShared s becomes tanh(x) / 2 = 1/2 -
// 1 / (e^{2 x} + 1), and a is 2 c; beyond, where that loses too much, tanh(x),
// and a is c.  What a row does not see becomes -inf, and so does its score.
// Few variants on purpose: a block's first pass through each is read from L2,
// a microsecond that a short item does not get back.
//
// Four scores share one reciprocal, that of their product (1 / u = r v for
// r = 1 / (u v)): reciprocals run at half the rate of exponentials here, and
// one each made a chunk of 512 tokens, 64 heads, against 8192 keys 190 us, one
// for two 173, one for four 166 (172 with the mask before them, which this
// needs).  The exponents stop at 30, where 1/2 - 1 / (2^30 + 1) is 1/2 in fp32,
// so that the product stays finite.  A NaN that a row sees makes all of its
// outputs NaN with or without that.
__device__ __forceinline__ void cap_scores(uint32_t (&s)[64], float cap_in) {
  const uint64_t cc = f2_pack(cap_in, cap_in), one = f2_pack(-1.f, -1.f), half = f2_pack(0.5f, 0.5f);
#pragma unroll
  for (int t = 0; t < 64; t += 4) {
    uint64_t e[2];  // -(e^{2 x} + 1) of two scores each
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float x0, x1;
      f2_unpack(f2_mul(f2_pack(__uint_as_float(s[t + 2 * u]), __uint_as_float(s[t + 2 * u + 1])), cc), x0, x1);
      e[u] = f2_fma(f2_pack(exp2_approx(min_nan(x0, 30.f)), exp2_approx(min_nan(x1, 30.f))), one, one);
    }
    float x, y, r;
    f2_unpack(f2_mul(e[0], e[1]), x, y);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * y));
    const uint64_t inv = f2_mul(f2_pack(r, r), f2_pack(y, x));
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      f2_unpack(f2_fma(inv, e[u ^ 1], half), x, y);
      s[t + 2 * u] = __float_as_uint(x);
      s[t + 2 * u + 1] = __float_as_uint(y);
    }
  }
}

// tanh(x), for caps that the form above is not exact enough for.
__device__ __forceinline__ void cap_scores_far(uint32_t (&s)[64], float cap_in) {
#pragma unroll
  for (int t = 0; t < 64; ++t) s[t] = __float_as_uint(tanhf(__uint_as_float(s[t]) * cap_in));
}

__device__ __forceinline__ float largest(const uint32_t (&s)[64]) {
  float top[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) top[q] = __uint_as_float(s[q]);
#pragma unroll
  for (int t = 4; t < 64; t += 2)
    top[(t >> 1) & 3] = max3(top[(t >> 1) & 3], __uint_as_float(s[t]), __uint_as_float(s[t + 1]));
  return max3(fmaxf(top[0], top[1]), top[2], top[3]);
}

// The weights 2^(a s + b) as pairs of 16-bit numbers (key 2 u in the low half
// of word u) to TMEM at `addr`, 32 at a time; returns their fp32 sum.  The
// rounding to 16 bits costs about as much accuracy as that of the output (the
// result is off by 0.0022 of its norm in bf16, where the output's rounding alone
// is 0.0017); a second number a weight, as the 16-row kernel has, would double
// the products that bound this one.
template <typename T>
__device__ __forceinline__ float half_weights(const uint32_t (&s)[64], uint32_t addr, float a, float b) {
  const uint64_t aa = f2_pack(a, a), bb = f2_pack(b, b);
  uint64_t sum[2] = {0ull, 0ull};  // pairs of +0.f
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w[16];
#pragma unroll
    for (int u = 0; u < 16; ++u) {
      const int t = 32 * h + 2 * u;
      float x0, x1;
      f2_unpack(f2_fma(f2_pack(__uint_as_float(s[t]), __uint_as_float(s[t + 1])), aa, bb), x0, x1);
      const float p0 = exp2_approx(x0), p1 = exp2_approx(x1);
      sum[u & 1] = f2_add(sum[u & 1], f2_pack(p0, p1));
      w[u] = pack2<T>(p0, p1);
    }
    tmem_st_32x32b_x16(addr + 16 * h, w);
  }
  float x, y, z, v;
  f2_unpack(sum[0], x, y);
  f2_unpack(sum[1], z, v);
  return (x + y) + (z + v);
}

// The keys an item's rows see, in blocks: those of its part.
struct Blocks {
  int lo, hi;      // keys that some row sees
  int first, end;  // blocks of 128 keys
};
__device__ __forceinline__ Blocks blocks_of(const PagedParams& p, const PagedItem& it) {
  Blocks b;
  const int t0 = it.pair * 2 * p.tile_tokens;
  const int t1 = min(t0 + 2 * p.tile_tokens, it.s.n);
  const int before = it.s.len - it.s.n;  // keys before the first new token
  b.hi = max(0, before + t1);
  b.lo = p.a.window > 0 ? max(0, max(0, before + t0 + 1) - p.a.window) : 0;
  const int k0 = b.lo / kKeysBlock, k1 = b.hi > b.lo ? (b.hi + kKeysBlock - 1) / kKeysBlock : k0;
  const int per = (k1 - k0 + p.tile_splits - 1) / p.tile_splits;
  b.first = min(k1, k0 + it.split * per);
  b.end = min(k1, b.first + per);
  return b;
}

// FAR: the cap is above kCapShared.  (A variant of its own: with tanhf beside
// the other forms an uncapped chunk of 512 tokens, 64 heads, against 8192 keys
// took 119.6 us for 115.3.)
template <typename T, int D, bool FAR>
__global__ void __launch_bounds__(kTileThreads, 1)
    paged_tile_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PagedParams p) {
  using C = TileCfg<D>;
  constexpr uint32_t kFmt = std::is_same_v<T, __nv_bfloat16> ? 1u : 0u;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t q_s = smem_u32(smem), kv_s = q_s + 2 * C::kQBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + 2 * C::kQBytes + C::kStages * C::kStageBytes);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const uint32_t bar0 = smem_u32(bars);
  // stages of K, then of V
  auto full = [&](uint32_t s) { return bar0 + 8 * s; };
  auto empty = [&](uint32_t s) { return bar0 + 8 * (C::kStages + s); };
  const uint32_t bar1 = bar0 + 16 * C::kStages;
  const uint32_t q_full = bar1, q_empty = bar1 + 8, tail = bar1 + 16;
  // per tile and buffer: S written, P written, its product complete; per
  // tile: the item's O written, and read
  auto s_full = [&](int i, int x) { return bar1 + 24 + 16 * i + 8 * x; };
  auto p_full = [&](int i, int x) { return bar1 + 56 + 16 * i + 8 * x; };
  auto pv_done = [&](int i, int x) { return bar1 + 88 + 16 * i + 8 * x; };
  auto o_full = [&](int i) { return bar1 + 120 + 8 * i; };
  auto o_empty = [&](int i) { return bar1 + 136 + 8 * i; };
  auto drain = [&](int i) { return bar1 + 152 + 8 * i; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 2);  // both tiles' products have read it
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 2);
    mbar_init(tail, 1);
    for (int i = 0; i < 2; ++i) {
      for (int x = 0; x < 2; ++x) {
        mbar_init(s_full(i, x), 1);
        mbar_init(p_full(i, x), 4);
        mbar_init(pv_done(i, x), 1);
      }
      mbar_init(o_full(i), 1);
      mbar_init(o_empty(i), 4);
      mbar_init(drain(i), 1);
      mbar_init(drain(2 + i), 1);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  // rows of the query tiles that no token fills are zeros throughout
  for (int i = threadIdx.x; i < 2 * C::kQBytes / 16; i += kTileThreads)
    reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 3) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dep_wait();
  grid_dep_launch();
  const gemm_paged_attention_t& a = p.a;
  const int grid = static_cast<int>(gridDim.x);
  // Item k of this block: rounds of the grid alternate the blocks' order, so
  // that the one with the longest item of a round gets the shortest of the
  // next.
  auto item_at = [&](int k) {
    const int idx = k * grid + ((k & 1) ? grid - 1 - static_cast<int>(blockIdx.x) : static_cast<int>(blockIdx.x));
    return paged_item(p, idx, warp == 0 && idx < grid);
  };
  const int tile_rows = p.tile_tokens * p.group;

  if (warp == 0) {
    // -------------------------------------------------------------- loads
    const int boxes = kKeysBlock / p.box;
    uint32_t n = 0, items = 0, tails = 0;  // blocks, items, blocks with zeros so far
    uint32_t filled[2] = {0, 0};           // stages of K and V filled
    int computed = 0;                      // items of the call, none after a wait that ran out
    bool ok = true;
    for (int k = 0; ok; ++k) {
      const PagedItem it = item_at(k);
      if (!it.valid) {
        computed = min(it.part, p.tile_parts);
        break;
      }
      if (it.part >= p.tile_parts) {  // only where the sequences' offsets are out of order
        if (lane == 0) atomicExch(p.status, kDevBadIndex);
        computed = p.tile_parts;
        break;
      }
      const Blocks b = blocks_of(p, it);
      if (b.first >= b.end) continue;
      // The page and slot of the lane's box of block j; the page is checked
      // when it is used, a block later.
      const int32_t* table = a.table + it.seq * a.table_row;
      auto lookup = [&](int j, int& page, int& slot, bool& there) {
        const int key = j * kKeysBlock + lane * p.box;
        there = j < b.end && lane < boxes && key < b.hi && key + p.box > b.lo;
        slot = 0;
        page = -1;
        if (there) {
          const int col = key / a.page_size;
          slot = key - col * a.page_size;
          page = table[col];
        }
      };
      int page, slot, next_page, next_slot;
      bool there, next_there;
      lookup(b.first, page, slot, there);
      const int token0 = it.pair * 2 * p.tile_tokens;
      const int tiles = token0 + p.tile_tokens < it.s.n ? 2 : 1;
      if (!warp_wait(q_empty, (items & 1u) ^ 1u, abort_flag, p.status, kDevTimeoutEmpty, p.wait_ns)) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(q_full, tiles * C::kHalves * tile_rows * 128);
        for (int t = 0; t < tiles; ++t)
          for (int h = 0; h < C::kHalves; ++h)
            tma_load_4d(q_s + t * C::kQBytes + h * kHalfBytes, &tmQ, q_full, 64 * h, 0, it.head,
                        static_cast<int>(it.s.first) + token0 + t * p.tile_tokens);
      }
      __syncwarp();
      ++items;
      for (int j = b.first; j < b.end; ++j, ++n) {
        lookup(j + 1, next_page, next_slot, next_there);
        if (there && (page < 0 || page >= a.num_pages)) {
          atomicExch(p.status, kDevBadIndex);
          page = -1;  // a copy from a page that is not there gives zeros
        }
        // Values past the last token become zeros before the products see the
        // stage: those copies land on a barrier of this warp's own.
        const int past = j + 1 == b.end ? (j + 1) * kKeysBlock - b.hi : 0;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          constexpr int kN[2] = {C::kKStages, C::kVStages};
          const uint32_t st = n % kN[kv] + (kv ? C::kKStages : 0), use = n / kN[kv];
          if (!warp_wait(empty(st), (use & 1u) ^ 1u, abort_flag, p.status, kDevTimeoutEmpty, p.wait_ns)) {
            ok = false;
            break;
          }
          const uint32_t bar = kv && past > 0 ? tail : full(st);
          if (lane == 0) mbar_arrive_expect_tx(bar, C::kStageBytes);
          __syncwarp();
          if (lane < boxes) {
            const uint32_t dst = kv_s + st * C::kStageBytes + lane * p.box * 128;
#pragma unroll
            for (int h = 0; h < C::kHalves; ++h)
              tma_load_4d(dst + h * kHalfBytes, kv ? &tmV : &tmK, bar, 64 * h, slot, it.head, page);
          }
          filled[kv] = n + 1;
        }
        if (!ok) break;
        if (past > 0) {
          if (!warp_wait(tail, tails & 1u, abort_flag, p.status, kDevTimeoutFull, p.wait_ns)) {
            ok = false;
            break;
          }
          ++tails;
          // the rest of their last copy: the ones behind it are zeros
          const uint32_t st = n % C::kVStages + C::kKStages;
          const int r0 = kKeysBlock - past, r1 = (r0 + p.box - 1) / p.box * p.box;
          uint8_t* v = smem + 2 * C::kQBytes + st * C::kStageBytes;
          for (int x = lane; x < (r1 - r0) * 8 * C::kHalves; x += 32) {
            const int half = x / ((r1 - r0) * 8), rest = x % ((r1 - r0) * 8);
            *reinterpret_cast<uint4*>(v + half * kHalfBytes + r0 * 128 + rest * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(full(st));
        }
        page = next_page;
        slot = next_slot;
        there = next_there;
      }
    }
    // how many there are to join, for the kernel that ends after this one
    if (lane == 0 && blockIdx.x == 0) p.queue[2] = computed;
    // every copy lands before the block exits: the last use of each stage
    if (lane == 0) {
      if (items > 0) drain_wait(q_full, (items - 1) & 1u, p.status, p.wait_ns);
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const uint32_t stages = kv ? C::kVStages : C::kKStages;
        for (uint32_t i = 1; i <= stages && i <= filled[kv]; ++i) {
          const uint32_t u = filled[kv] - i;
          drain_wait(full(u % stages + (kv ? C::kKStages : 0)), (u / stages) & 1u, p.status, p.wait_ns);
        }
      }
    }
  } else if (warp < 4 || warp == 12) {
    // ------------------------------------------------- matrix instructions
    constexpr uint32_t kIdescS = make_idesc(kFmt, false, false, 128, 64);
    constexpr uint32_t kIdescO = make_idesc(kFmt, false, true, 128, D);
    const bool values = warp == 3 || warp == 12;  // this warp's products
    const int tile = warp == 2 || warp == 12;
    const uint32_t s_tmem = tmem + 128 * tile, o_tmem = tmem + 256 + D * tile;
    const uint64_t qd = smem_desc_sw128(q_s + tile * C::kQBytes, 16, 1024);
    const uint32_t stage0 = values ? C::kKStages : 0, stages = values ? C::kVStages : C::kKStages;
    uint32_t st = 0, st_phase = 0;  // the ring's next stage, and its phase
    uint32_t items = 0, outs = 0, blocks = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      const PagedItem it = item_at(k);
      if (!it.valid || it.part >= p.tile_parts) break;
      const Blocks b = blocks_of(p, it);
      if (b.first >= b.end) continue;
      // a tile without rows: its warps only give the stages back
      const bool present = (it.pair * 2 + tile) * p.tile_tokens < it.s.n;
      if (lane == 0) {
        auto wait = [&](uint32_t bar, uint32_t parity, int code) {
          return mbar_wait(bar, parity, abort_flag, p.status, code, p.wait_ns);
        };
        ok = values ? !present || wait(o_empty(tile), (outs & 1u) ^ 1u, kDevTimeoutAccEmpty)
                    : wait(q_full, items & 1u, kDevTimeoutFull);
        for (int j = b.first; j < b.end && ok; ++j) {
          ok = wait(full(stage0 + st), st_phase, kDevTimeoutFull);
          if (!ok) break;
          const uint32_t at = kv_s + (stage0 + st) * C::kStageBytes;
          if (present && values) {
            const uint64_t vd = smem_desc_sw128(at, kHalfBytes, 1024);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              ok = ok && wait(p_full(tile, x), blocks & 1u, kDevTimeoutFull);
              if (!ok) break;
              tc_fence_after();
#pragma unroll
              for (int s = 0; s < 4; ++s)
                mma_bf16_tmem_a(o_tmem, s_tmem + 64 * x + 8 * s, vd + 128 * (4 * x + s), kIdescO,
                                (j > b.first || x + s > 0) ? 1u : 0u);
              mma_commit(pv_done(tile, x));
            }
            ++blocks;
          } else if (present) {
            const uint64_t kd = smem_desc_sw128(at, 16, 1024);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              // the buffer's last P read
              ok = ok && wait(pv_done(tile, x), (blocks & 1u) ^ 1u, kDevTimeoutAccEmpty);
              if (!ok) break;
              tc_fence_after();
#pragma unroll
              for (int h = 0; h < C::kHalves; ++h)
#pragma unroll
                for (int s = 0; s < 4; ++s)
                  mma_bf16(s_tmem + 64 * x, qd + h * (kHalfBytes / 16) + 2 * s,
                           kd + 64 * 128 / 16 * x + h * (kHalfBytes / 16) + 2 * s, kIdescS, h + s > 0 ? 1u : 0u);
              mma_commit(s_full(tile, x));
            }
            ++blocks;
          }
          if (!ok) break;
          mma_commit(empty(stage0 + st));
          if (++st == stages) {
            st = 0;
            st_phase ^= 1u;
          }
        }
        if (ok) {
          if (!values) mma_commit(q_empty);
          if (values && present) {
            mma_commit(o_full(tile));
            ++outs;
          }
        }
        ++items;
      }
      ok = __all_sync(0xffffffffu, ok);
    }
    if (lane == 0) {
      mma_commit(drain(2 * values + tile));
      drain_wait(drain(2 * values + tile), 0, p.status, p.wait_ns);
    }
  } else {
    // ------------------------------------------------------------- softmax
    const int tile = (warp - 4) / 4, quarter = warp & 3;
    const int r = quarter * 32 + lane;  // this thread's row
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t s_addr = tmem + lanes + 128 * tile, o_addr = tmem + lanes + 256 + D * tile;
    uint32_t blocks = 0, outs = 0;  // S and O of this tile so far
    for (int k = 0;; ++k) {
      const PagedItem it = item_at(k);
      if (!it.valid || it.part >= p.tile_parts) break;
      const Blocks b = blocks_of(p, it);
      const int token = (it.pair * 2 + tile) * p.tile_tokens + by_group(p, r);
      const bool valid = r < tile_rows && token < it.s.n;
      const bool any = b.first < b.end;
      const bool present = (it.pair * 2 + tile) * p.tile_tokens < it.s.n;  // the tile has rows
      const int hi = valid ? max(0, it.s.len - it.s.n + token + 1) : 0;
      float m = neg_inf(), l = 0.f;
      bool ok = true;
      // every row of the warp with a token sees the keys up to here (what the
      // other rows make of them is not stored)
      const int all_hi = __reduce_min_sync(0xffffffffu, valid ? hi : INT_MAX);
      for (int j = b.first; j < b.end && present; ++j, ++blocks) {
        // the block in halves of 64 keys, a buffer each
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          if (!warp_wait(s_full(tile, half), blocks & 1u, abort_flag, p.status, kDevTimeoutAccFull, p.wait_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const int key0 = j * kKeysBlock + 64 * half;
          const bool whole = key0 + 64 <= all_hi && (a.window == 0 || __all_sync(0xffffffffu, hi - a.window <= key0));
          uint32_t s[64];
          tmem_ld_64(s_addr + 64 * half, s);
          if (p.flip) {
#pragma unroll
            for (int t = 0; t < 64; ++t) s[t] ^= 0x80000000u;
          }
          // Capped scores are masked before, too, with zeros: what an unseen
          // slot holds would reach the scores that share its reciprocal (and
          // so would an infinity, which a scale of 0 makes a NaN).
#pragma unroll 1
          for (bool capped = p.cap_out == 0.f;; capped = true) {
            if (!whole) {
              // this row sees the keys [hi - window, hi)
              const int from = a.window > 0 ? hi - a.window - key0 : 0, to = hi - key0;
              const uint32_t unseen = capped ? 0xff800000u : 0u;
#pragma unroll
              for (int t = 0; t < 64; ++t) s[t] = t >= from && t < to ? s[t] : unseen;
            }
            if (capped) break;
            if constexpr (FAR)
              cap_scores_far(s, p.cap_in);
            else
              cap_scores(s, p.cap_in2);
          }
          const float best = largest(s) * p.s_scale;
          const bool raise = __any_sync(0xffffffffu, best > m + kSlack);
          if (raise) {
            const float m_new = fmaxf(m, best);
            const float alpha = m == neg_inf() ? 0.f : exp2_approx(m - m_new);
            m = m_new;
            l *= alpha;
            if (half == 1 || j > b.first) {
              // The products so far: this buffer's last one came before its S;
              // the other buffer's may still run.
              if (!warp_wait(pv_done(tile, half ^ 1), (half ? blocks : blocks - 1) & 1u, abort_flag, p.status,
                             kDevTimeoutAccFull, p.wait_ns)) {
                ok = false;
                break;
              }
              tc_fence_after();
#pragma unroll 1
              for (int h = 0; h < D; h += 16) {  // (16 columns: the scores are still in registers)
                uint32_t o[16];
                tmem_ld_32x32b_x16(o_addr + h, o);
                tmem_wait_ld();
#pragma unroll
                for (int t = 0; t < 16; ++t) o[t] = __float_as_uint(__uint_as_float(o[t]) * alpha);
                tmem_st_32x32b_x16(o_addr + h, o);
              }
            }
          }
          const float shift = m == neg_inf() ? 0.f : m - weight_bias<T>();
          l += half_weights<T>(s, s_addr + 64 * half, p.s_scale, -shift);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full(tile, half));
        }
        if (!ok) break;
      }
      if (!ok) break;
      // O / l, or the part's sums
      float acc = 0.f;  // NaN when a sum is not finite
      const int64_t row = it.s.first + token;
      const int head = it.head * p.group + r - by_group(p, r) * p.group;
      T* out = static_cast<T*>(a.out) + row * a.out_token + head * a.out_head;
      const size_t floats = 256 * (D + 2);
      float* part = p.tile_part + static_cast<size_t>(it.part) * floats;
      const bool parts = p.tile_splits > 1;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      if (any && present) {
        if (!warp_wait(o_full(tile), outs & 1u, abort_flag, p.status, kDevTimeoutAccFull, p.wait_ns)) break;
        tc_fence_after();
        ++outs;
      }
#pragma unroll
      for (int h = 0; h < D; h += 32) {
        uint32_t o[32];
        if (any && present) {
          tmem_ld_32x32b_x32(o_addr + h, o);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int t = 0; t < 32; ++t) o[t] = 0u;
        }
        if (!valid) continue;
#pragma unroll
        for (int t = 0; t < 32; ++t) acc = fmaf(__uint_as_float(o[t]), 0.f, acc);
        if (parts) {
#pragma unroll
          for (int t = 0; t < 32; t += 4)
            *reinterpret_cast<uint4*>(part + (128 * tile + r) * D + h + t) = make_uint4(o[t], o[t + 1], o[t + 2], o[t + 3]);
        } else {
          uint32_t w[16];
#pragma unroll
          for (int t = 0; t < 16; ++t)
            w[t] = l == 0.f ? 0u : pack2<T>(__uint_as_float(o[2 * t]) * inv, __uint_as_float(o[2 * t + 1]) * inv);
          if (p.out_v8) {
#pragma unroll
            for (int t = 0; t < 16; t += 8) {
              const uint32_t x[8] = {w[t], w[t + 1], w[t + 2], w[t + 3], w[t + 4], w[t + 5], w[t + 6], w[t + 7]};
              st_global_v8(out + h + 2 * t, x);
            }
          } else {
#pragma unroll
            for (int t = 0; t < 16; t += 4)
              *reinterpret_cast<uint4*>(out + h + 2 * t) = make_uint4(w[t], w[t + 1], w[t + 2], w[t + 3]);
          }
        }
      }
      if (any && present) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(o_empty(tile));
      }
      if (valid) {
        const float top = m == neg_inf() ? m : m - weight_bias<T>();
        if (parts) {
          part[256 * D + 128 * tile + r] = top;
          part[256 * (D + 1) + 128 * tile + r] = l;
        } else if (a.lse != nullptr) {
          a.lse[row * a.heads + head] = l == 0.f ? neg_inf() : (top + log2f(l)) * 0.6931471805599453f;
        }
      }
      // 0 where everything is finite, and where a row sees no key
      const bool again = __any_sync(0xffffffffu, valid && (!(acc == 0.f) || !(l * 0.f == 0.f)));
      if (lane == 0) p.redo[static_cast<size_t>(it.part) * 8 + (warp - 4)] = again ? 1 : 0;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 3) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

using Encode = PFN_cuTensorMapEncodeTiled_v12000;

CUresult encode4(Encode encode, CUtensorMap* m, bool bf16, const void* ptr, const int64_t (&dim)[4],
                 const int64_t (&stride)[3], const uint32_t (&box)[4]) {
  cuuint64_t dims[4], strides[3];
  cuuint32_t boxes[4], ones[4] = {1, 1, 1, 1};
  int64_t dense = dim[0] * 2;
  for (int i = 0; i < 4; ++i) {
    dims[i] = static_cast<cuuint64_t>(dim[i] > 0 ? dim[i] : 1);
    boxes[i] = box[i];
  }
  for (int i = 0; i < 3; ++i) {
    // a dimension of one has no stride of its own
    strides[i] = static_cast<cuuint64_t>(dim[i + 1] > 1 ? stride[i] * 2 : dense);
    dense = static_cast<int64_t>(strides[i]) * dim[i + 1];
    if (dense % 16 != 0) dense = dim[0] * 2;
  }
  return encode(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                const_cast<void*>(ptr), dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

template <typename T, int D, bool FAR>
cudaError_t launch_tiles(const PagedParams& p, int grid, cudaStream_t stream) {
  cudaError_t e = tc_init_driver();
  if (e != cudaSuccess) return e;
  const Encode encode = tc_encoder();
  if (encode == nullptr) return cudaErrorNotSupported;
  const gemm_paged_attention_t& a = p.a;
  constexpr bool bf16 = std::is_same_v<T, __nv_bfloat16>;
  CUtensorMap tq, tk, tv;
  // no pages: the maps need an address, and nothing is read through them
  const void* kp = a.num_pages > 0 ? a.k_pages : a.q;
  const void* vp = a.num_pages > 0 ? a.v_pages : a.q;
  // queries: (element, head of the group, key head, token); pages: (element,
  // slot, key head, page)
  if (encode4(encode, &tq, bf16, a.q, {D, p.group, a.kv_heads, a.tokens}, {a.q_head, a.q_head * p.group, a.q_token},
              {64, static_cast<uint32_t>(p.group), 1, static_cast<uint32_t>(p.tile_tokens)}) != CUDA_SUCCESS ||
      encode4(encode, &tk, bf16, kp, {D, a.page_size, a.kv_heads, a.num_pages}, {a.k_slot, a.k_head, a.k_page},
              {64, static_cast<uint32_t>(p.box), 1, 1}) != CUDA_SUCCESS ||
      encode4(encode, &tv, bf16, vp, {D, a.page_size, a.kv_heads, a.num_pages}, {a.v_slot, a.v_head, a.v_page},
              {64, static_cast<uint32_t>(p.box), 1, 1}) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> attr_done{0};
  e = once_per_device(attr_done, [] {
    return cudaFuncSetAttribute(paged_tile_kernel<T, D, FAR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                TileCfg<D>::kSmem);
  });
  if (e != cudaSuccess) return e;
  last_main_launch() =
      LaunchShape{dim3(static_cast<unsigned>(grid)), dim3(kTileThreads), TileCfg<D>::kSmem, 1, true};
  return launch_pdl(paged_tile_kernel<T, D, FAR>, dim3(static_cast<unsigned>(grid)), dim3(kTileThreads),
                    TileCfg<D>::kSmem, stream, tq, tk, tv, p);
}

template <typename T, int D>
cudaError_t launch_tiles_as(const PagedParams& p, int grid, cudaStream_t stream) {
  return p.cap_out > 0.f && !p.cap_shared ? launch_tiles<T, D, true>(p, grid, stream)
                                          : launch_tiles<T, D, false>(p, grid, stream);
}

}  // namespace

cudaError_t launch_paged_tiles(const PagedParams& p, int grid, cudaStream_t stream) {
  if (p.a.type == GEMM_TYPE_BF16)
    return p.a.head_dim == 64 ? launch_tiles_as<__nv_bfloat16, 64>(p, grid, stream)
                              : launch_tiles_as<__nv_bfloat16, 128>(p, grid, stream);
  return p.a.head_dim == 64 ? launch_tiles_as<__half, 64>(p, grid, stream) : launch_tiles_as<__half, 128>(p, grid, stream);
}

}  // namespace dgt
