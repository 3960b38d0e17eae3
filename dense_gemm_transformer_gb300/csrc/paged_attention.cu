// paged_attention.cu -- attention of new tokens over a paged cache.
//
// For the row of query head h and new token i of a sequence with n new
// tokens and N keys, p = N - n + i, over the keys p - window < j <= p:
//
//     s_j = scale q . k_j   (softcap c > 0: c tanh(s_j / c)),
//     out = sum_j e^{s_j - m} v_j / l,   l = sum_j e^{s_j - m},   lse = m + log l
//
// in one pass over the keys with the running maximum m and sum l of the
// softmax.  The heads of a group read the same keys, so the rows of a (sequence,
// key head) are (token, head of the group) pairs, and a block takes 16 of
// them: m16n8k16 matrix instructions, whose rate is several times what the
// traffic needs when every key is read for 16 rows only.
//
// What bounds it is the read of the keys and values, once.  So that each SM
// has enough of it in flight, every warp streams its own tiles of 16 keys
// (tile w, w + 4, ... of the block's range) through a private ring of
// tiles filled by 16-byte asynchronous copies: the warps share
// nothing until they have run out of keys, and there is no block-wide
// barrier in the loop.  The range of a sequence is split over blocks when
// there are too few (sequence, head) pairs to fill the SMs; the block that
// finishes last joins the parts, in the parts' order, so the result does not
// depend on which one that is.  One token in each of 64 sequences of 1 to 8192
// keys, 12 heads of 128 over 2: 63 us, 4.7 TB/s; against 1001 keys of one
// sequence 8.5 us, a chain of latencies.
//
// A tile that some row of the block sees only in part goes without the
// matrix instruction for the values: there, 0 x v would let an infinity or
// NaN of a token a row must not see into that row.  Slots that no row sees
// (past the sequence, before the window) are copied as zeros.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "kernels.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace dgt {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = kPagedPartRows;  // rows a block (M of the matrix instruction)
constexpr int kKeys = 16;              // keys a warp's tile
// Tiles in a warp's ring: two, or more where that many bytes fit for all of a
// call's blocks at once (paged_attention_plan).
constexpr int kStages = 2, kDeepStages = 4;
constexpr int ring_bytes(int dim, int stages) { return kWarps * stages * 2 * kKeys * dim * 2; }
// The joins keep the maxima (then weights) and sums of a range's parts there.
static_assert(kPagedMostSplits * kRows * 2 * static_cast<int>(sizeof(float)) <= ring_bytes(64, kStages));

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, bool valid) {
  const int bytes = valid ? 16 : 0;  // the rest of the 16 bytes is filled with zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

template <typename T>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same_v<T, __nv_bfloat16>)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The largest weight is 2^kBias, here and in the sums, and the factor cancels
// in the output.  In fp16 numbers below 2^-14 have fewer bits: with 1 for the
// largest, a quarter of a million keys with weights of 2^-18 each that a warp
// meets beside a few of 1 had their part off by 2^-7 of itself.
template <typename T>
constexpr float kBias = std::is_same_v<T, __half> ? 14.f : 0.f;

struct RowsShared {
  float m[kWarps][kRows], l[kWarps][kRows];
  float f[kWarps][kRows];  // factors of the warps' sums
  float inv[kRows];        // of a joined range: 1 / l
  int last, unit;
  unsigned redo[kWarps];   // of the items that are looked at: which to compute again
};

// The sums of a warp that are not numbers though the scores are (lsum: the
// rows' sums of weights): a value that a row sees is infinite or not a number.
// Of a weight's two 16-bit numbers one may be 0 or negative, and the sum of
// their products with an infinity NaN; which infinity it should be is found
// from the values, a tile at a time for all rows.  Not inlined: its registers
// are the kernel's otherwise, and those decide how many blocks an SM has.
template <typename T, int D>
__device__ __noinline__ void infinite_sums(const PagedParams& p, float* sums, const float* lsum, const int32_t* table,
                                           const T* vbase, int rows, int head0, int seen0, int tile, int tiles) {
  constexpr int kCols = D / 32;  // a lane's columns, consecutive ones
  struct alignas(2 * kCols) Cols {
    T x[kCols];
  };
  const gemm_paged_attention_t& a = p.a;
  const int lane = threadIdx.x & 31;
  // row `lane` sees the keys [from, to)
  const int to = lane < rows ? max(0, seen0 + by_group(p, head0 + lane)) : 0;
  const int from = a.window > 0 ? max(0, to - a.window) : 0;
  unsigned plus[kCols] = {}, minus[kCols] = {}, nan[kCols] = {};  // bit r: row r sees such a value
#pragma unroll 1
  for (int it = 0; it < tiles; ++it) {
    const int key0 = (tile + it * kWarps) * kKeys, col = key0 / a.page_size;
    const int page = table[col];
    if (page < 0 || page >= a.num_pages) continue;
    const T* v = vbase + page * a.v_page + (key0 - col * a.page_size) * a.v_slot + kCols * lane;
    Cols y[kKeys];
#pragma unroll
    for (int k = 0; k < kKeys; ++k) y[k] = *reinterpret_cast<const Cols*>(v + k * a.v_slot);
#pragma unroll
    for (int k = 0; k < kKeys; ++k) {
      const unsigned seen = __ballot_sync(0xffffffffu, key0 + k >= from && key0 + k < to);
#pragma unroll
      for (int x = 0; x < kCols; ++x) {
        const float f = as_f(y[k].x[x]);
        plus[x] |= f == -neg_inf() ? seen : 0u;
        minus[x] |= f == neg_inf() ? seen : 0u;
        nan[x] |= isnan(f) ? seen : 0u;
      }
    }
  }
#pragma unroll 1
  for (int r = 0; r < rows; ++r) {
    if (isnan(lsum[r])) continue;  // scores that are not numbers leave no other result
#pragma unroll
    for (int x = 0; x < kCols; ++x) {
      float* at = sums + r * D + ((kCols * lane + x) ^ (8 * (r & 3)));
      const bool up = plus[x] >> r & 1, down = minus[x] >> r & 1;
      if (isnan(*at) && up != down && !(nan[x] >> r & 1)) *at = up ? -neg_inf() : neg_inf();
    }
  }
}

// The rows row0 .. row0 + rows - 1 of a (sequence, key head), all of their
// keys or (of `splits` parts) part `split`.  `range` numbers the rows among
// the call's ranges of parts.  ahead_page: the table's entry ahead_col, read
// beside the sequence's length (-1: none).
template <typename T, int D>
__device__ __forceinline__ void rows_unit(const PagedParams& p, uint8_t* smem, RowsShared& sh, const PagedSeq& s,
                                          int seq, int head, int row0, int rows, int split, int splits, int range,
                                          int ahead_col, int ahead_page) {
  constexpr int kChunks = D / 8;                 // 16-byte chunks a row
  constexpr int kTileBytes = kKeys * D * 2;      // one tile of keys (or values)
  const int last_stage = p.row_stages - 1;       // kStages - 1 or kDeepStages - 1
  const int warp_bytes = p.row_stages * 2 * kTileBytes;
  constexpr int kCopies = kKeys * kChunks / 32;  // copies a lane per tile of keys (or values)
  const gemm_paged_attention_t& a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // Row r of the block: new token token0 + (head0 + r) / group, head (head0 +
  // r) % group of the group.
  const int token0 = row0 / p.group, head0 = row0 - token0 * p.group;
  // Keys row r sees: [lo(r), hi(r)).
  const int seen0 = s.len - s.n + token0 + 1;
  auto hi_of = [&](int r) { return max(0, seen0 + by_group(p, head0 + r)); };
  auto lo_of = [&](int r) { return a.window > 0 ? max(0, hi_of(r) - a.window) : 0; };
  const int lo = lo_of(0), hi = hi_of(rows - 1);
  // keys every row sees; in a tile without others of [lo, hi), all rows see
  // the same
  const int common_lo = lo_of(rows - 1), common_hi = hi_of(0);
  const int tile0 = lo / kKeys, tiles = hi > lo ? (hi + kKeys - 1) / kKeys - tile0 : 0;
  const int parts = max(1, (tiles + p.tiles_per - 1) / p.tiles_per);
  const int my_parts = min(parts, splits);
  if (split >= my_parts) return;
  // the last part takes what the bound on the keys did not foresee
  const int begin = split * p.tiles_per;
  const int end = split == my_parts - 1 ? tiles : begin + p.tiles_per;
  const int mine = max(0, (end - begin - warp + kWarps - 1) / kWarps);  // tiles of this warp

  const T* kbase = static_cast<const T*>(a.k_pages) + head * a.k_head;
  const T* vbase = static_cast<const T*>(a.v_pages) + head * a.v_head;
  const int32_t* table = a.table + seq * a.table_row;
  const uint32_t ring = smem_u32(smem) + warp * warp_bytes;

  // Page and first slot of the warp's tile 32 b + lane, for the batch b of
  // tiles being issued.
  int my_page = -1, my_slot = 0;
  auto load_pages = [&](int it) {
    const int t = tile0 + begin + warp + (it + lane) * kWarps;
    my_page = -1;
    if (it + lane < mine) {
      const int key = t * kKeys, col = key / a.page_size;
      my_slot = key - col * a.page_size;
      my_page = it == 0 && ahead_col == col ? ahead_page : table[col];
      if (my_page < 0 || my_page >= a.num_pages) {
        atomicExch(p.status, kDevBadIndex);
        my_page = -1;
      }
    }
  };
  auto issue = [&](int it) {
    if ((it & 31) == 0) load_pages(it);
    const int page = __shfl_sync(0xffffffffu, my_page, it & 31), slot = __shfl_sync(0xffffffffu, my_slot, it & 31);
    if (it < mine) {
      const int key0 = (tile0 + begin + warp + it * kWarps) * kKeys;
      const uint32_t dst = ring + (it & last_stage) * (2 * kTileBytes);
      const T* kp = kbase + (page < 0 ? 0 : page * a.k_page + slot * a.k_slot);
      const T* vp = vbase + (page < 0 ? 0 : page * a.v_page + slot * a.v_slot);
#pragma unroll
      for (int c = 0; c < kCopies; ++c) {
        const int x = c * 32 + lane, row = x / kChunks, chunk = x % kChunks;
        const bool there = page >= 0 && key0 + row >= lo && key0 + row < hi;
        const uint32_t to = dst + row * (D * 2) + ((chunk ^ (row & 7)) << 4);
        cp_async_16(to, there ? kp + row * a.k_slot + chunk * 8 : kbase, there);
        cp_async_16(to + kTileBytes, there ? vp + row * a.v_slot + chunk * 8 : vbase, there);
      }
    }
    cp_async_commit();
  };

#pragma unroll 1
  for (int s = 0; s < last_stage; ++s) issue(s);

  // Q as the matrix instruction's A: rows g and g + 8 of the lane's quad.
  const int g = lane >> 2, quad = lane & 3;
  uint32_t qf[D / 16][4];
  int rlo[2], rhi[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int r = g + 8 * u;
    const bool valid = r < rows;
    rhi[u] = valid ? hi_of(r) : 0;
    rlo[u] = valid ? lo_of(r) : 0;
    const int up = by_group(p, head0 + r);
    const T* q = static_cast<const T*>(a.q) + (s.first + token0 + up) * a.q_token +
                 (head * p.group + head0 + r - up * p.group) * a.q_head + 2 * quad;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      qf[k][u] = valid ? *reinterpret_cast<const uint32_t*>(q + 16 * k) : 0u;
      qf[k][u + 2] = valid ? *reinterpret_cast<const uint32_t*>(q + 16 * k + 8) : 0u;
    }
  }

  float o[D / 8][4];
#pragma unroll
  for (int d = 0; d < D / 8; ++d)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[d][e] = 0.f;
  float m[2] = {neg_inf(), neg_inf()}, l[2] = {0.f, 0.f};

  const int mat = lane >> 3, mrow = lane & 7;  // the 8 x 8 matrix and row whose address this lane gives
  for (int it = 0; it < mine; ++it) {
    issue(it + last_stage);
    if (last_stage == kDeepStages - 1)
      cp_async_wait<kDeepStages - 1>();
    else
      cp_async_wait<kStages - 1>();
    __syncwarp();
    const uint32_t ks = ring + (it & last_stage) * (2 * kTileBytes), vs = ks + kTileBytes;
    const int key0 = (tile0 + begin + warp + it * kWarps) * kKeys;
    // S: two 8-key columns; lane holds keys key0 + 8 j + 2 quad, + 1 of rows g, g + 8
    float s[2][4] = {};
    {
      const int row = (mat >> 1) * 8 + mrow;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t b[4];
        ldmatrix_x4(ks + row * (D * 2) + (((2 * k + (mat & 1)) ^ mrow) << 4), b);
        mma_16816<T>(s[0], qf[k], b[0], b[1]);
        mma_16816<T>(s[1], qf[k], b[2], b[3]);
      }
    }
    float top[2] = {neg_inf(), neg_inf()};
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int u = e >> 1, key = key0 + 8 * j + 2 * quad + (e & 1);
        s[j][e] = key >= rlo[u] && key < rhi[u] ? score_of(s[j][e], p) : neg_inf();
        top[u] = fmaxf(top[u], s[j][e]);
      }
    bool raised = false;
    float alpha[2], shift[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      top[u] = fmaxf(top[u], __shfl_xor_sync(0xffffffffu, top[u], 1));
      top[u] = fmaxf(top[u], __shfl_xor_sync(0xffffffffu, top[u], 2));
      const float next = fmaxf(m[u], top[u]);
      raised |= next > m[u];
      const float from = next == neg_inf() ? 0.f : next;  // a row that has seen no key yet: its scores are all -inf
      alpha[u] = exp2_approx(m[u] - from);                // 0 for the first key seen
      shift[u] = from - kBias<T>;
      m[u] = next;
    }
    if (__any_sync(0xffffffffu, raised)) {
#pragma unroll
      for (int d = 0; d < D / 8; ++d) {
        o[d][0] *= alpha[0];
        o[d][1] *= alpha[0];
        o[d][2] *= alpha[1];
        o[d][3] *= alpha[1];
      }
      l[0] *= alpha[0];
      l[1] *= alpha[1];
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[j][e] = exp2_approx(s[j][e] - shift[e >> 1]);
        l[e >> 1] += s[j][e];
      }
    if (max(key0, lo) >= common_lo && min(key0 + kKeys, hi) <= common_hi) {
      // The weights as the A operand, as a sum of two 16-bit numbers: one
      // would cost as much accuracy as the output's own rounding, and the
      // second product is free here.  (2^14 is in range, and so is what the
      // rounding leaves.)
      uint32_t ph[4], pl[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float p0 = s[x >> 1][2 * (x & 1)], p1 = s[x >> 1][2 * (x & 1) + 1];
        ph[x] = pack2<T>(p0, p1);
        float h0, h1;
        unpack2<T>(ph[x], h0, h1);
        pl[x] = pack2<T>(p0 - h0, p1 - h1);
      }
      const int row = (mat & 1) * 8 + mrow;
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        uint32_t b[4];
        ldmatrix_x4_trans(vs + row * (D * 2) + (((2 * d + (mat >> 1)) ^ mrow) << 4), b);
        mma_16816<T>(o[2 * d], ph, b[0], b[1]);
        mma_16816<T>(o[2 * d], pl, b[0], b[1]);
        mma_16816<T>(o[2 * d + 1], ph, b[2], b[3]);
        mma_16816<T>(o[2 * d + 1], pl, b[2], b[3]);
      }
    } else {
      // Rows see different keys of this tile: key by key, a row adds only
      // what it sees.  Key 8 j + 2 q + e is held by the quads' lane q.
#pragma unroll 1
      for (int key = 0; key < kKeys; ++key) {
        const int src = (lane & ~3) | ((key & 7) >> 1);
        float w[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float even = (key & 8) ? s[1][2 * u] : s[0][2 * u], odd = (key & 8) ? s[1][2 * u + 1] : s[0][2 * u + 1];
          w[u] = __shfl_sync(0xffffffffu, (key & 1) ? odd : even, src);
        }
        const bool see0 = key0 + key >= rlo[0] && key0 + key < rhi[0];
        const bool see1 = key0 + key >= rlo[1] && key0 + key < rhi[1];
        const uint8_t* vrow = smem + (vs - smem_u32(smem)) + key * (D * 2) + quad * 4;
#pragma unroll
        for (int d = 0; d < D / 8; ++d) {
          float v0, v1;
          unpack2<T>(*reinterpret_cast<const uint32_t*>(vrow + ((d ^ (key & 7)) << 4)), v0, v1);
          if (see0) {
            o[d][0] = fmaf(w[0], v0, o[d][0]);
            o[d][1] = fmaf(w[0], v1, o[d][1]);
          }
          if (see1) {
            o[d][2] = fmaf(w[1], v0, o[d][2]);
            o[d][3] = fmaf(w[1], v1, o[d][3]);
          }
        }
      }
    }
    __syncwarp();  // the tile's slot is filled again
  }
  cp_async_wait<0>();
  bool nan = false;  // a sum of these rows
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    float sum = 0.f;
#pragma unroll
    for (int d = 0; d < D / 8; ++d) sum += o[d][2 * u] + o[d][2 * u + 1];
    nan |= g + 8 * u < rows && isnan(sum);
    l[u] += __shfl_xor_sync(0xffffffffu, l[u], 1);
    l[u] += __shfl_xor_sync(0xffffffffu, l[u], 2);
    if (quad == 0) {
      sh.m[warp][g + 8 * u] = m[u] - kBias<T>;
      sh.l[warp][g + 8 * u] = l[u];
    }
  }
  __syncwarp();  // every lane is done with the ring: it takes the warp's sums
  // Row r, column c at [r][c ^ 8 (r & 3)]: without the exclusive-or, rows
  // r and r + 1 of a quad's stores would meet in the same banks.
  float* mine_o = reinterpret_cast<float*>(smem + warp * warp_bytes);
#pragma unroll
  for (int d = 0; d < D / 8; ++d)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int r = g + 8 * u, c = (8 * d + 2 * quad) ^ (8 * (r & 3));
      *reinterpret_cast<float2*>(mine_o + r * D + c) = make_float2(o[d][2 * u], o[d][2 * u + 1]);
    }
  if (__any_sync(0xffffffffu, nan)) {
    __syncwarp();
    infinite_sums<T, D>(p, mine_o, sh.l[warp], table, vbase, rows, head0, seen0, tile0 + begin + warp, mine);
  }
  __syncthreads();

  // Joins the warps: a thread per row weighs their sums, then every thread
  // adds four columns at a time.
  constexpr int kPart = kRows * (D + 2);
  float* part = p.part + (static_cast<int64_t>(range) * splits + split) * kPart;
  auto out_at = [&](int r) {
    const int up = by_group(p, head0 + r);
    return static_cast<T*>(a.out) + (s.first + token0 + up) * a.out_token +
           (head * p.group + head0 + r - up * p.group) * a.out_head;
  };
  auto store_lse = [&](int r, float mm, float ll) {
    if (a.lse == nullptr) return;
    const int up = by_group(p, head0 + r);
    a.lse[(s.first + token0 + up) * a.heads + head * p.group + head0 + r - up * p.group] =
        ll == 0.f ? neg_inf() : (mm + log2f(ll)) * 0.6931471805599453f;
  };
  if (threadIdx.x < kRows) {
    const int r = threadIdx.x;
    float mm = neg_inf(), ll = 0.f, f[kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sh.m[w][r]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      f[w] = sh.m[w][r] == mm ? 1.f : exp2_approx(sh.m[w][r] - mm);
      ll = fmaf(f[w], sh.l[w][r], ll);
    }
    const float inv = my_parts > 1 ? 1.f : ll == 0.f ? 0.f : 1.f / ll;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sh.f[w][r] = f[w] * inv;
    if (r < rows) {
      if (my_parts == 1) {
        store_lse(r, mm, ll);
      } else {
        __stcg(part + kRows * D + r, mm);
        __stcg(part + kRows * D + kRows + r, ll);
      }
    }
  }
  __syncthreads();
  for (int x = threadIdx.x; x < rows * (D / 4); x += kThreads) {
    const int r = x / (D / 4), c = 4 * (x % (D / 4));
    float4 o4 = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = sh.f[w][r];
      const float4 v = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem + w * warp_bytes) + r * D +
                                                        (c ^ (8 * (r & 3))));
      o4.x = fmaf(f, v.x, o4.x);
      o4.y = fmaf(f, v.y, o4.y);
      o4.z = fmaf(f, v.z, o4.z);
      o4.w = fmaf(f, v.w, o4.w);
    }
    if (my_parts == 1)
      *reinterpret_cast<uint2*>(out_at(r) + c) = make_uint2(pack2<T>(o4.x, o4.y), pack2<T>(o4.z, o4.w));
    else
      __stcg(reinterpret_cast<float4*>(part + r * D + c), o4);
  }
  if (my_parts == 1) return;

  // The last block of the range joins its parts.
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    const bool last = atomicAdd(p.arrived + range, 1) == my_parts - 1;
    if (last) p.arrived[range] = 0;
    sh.last = last ? 1 : 0;
  }
  __syncthreads();
  if (!sh.last) return;
  __threadfence();
  part = p.part + static_cast<int64_t>(range) * splits * kPart;
  // the parts' maxima and sums, row by row, then their weights, in place of
  // the ring
  float* jm = reinterpret_cast<float*>(smem);
  float* jl = jm + my_parts * kRows;
  for (int i = threadIdx.x; i < my_parts * kRows; i += kThreads) {
    const float* at = part + (i / kRows) * kPart + kRows * D + i % kRows;
    jm[i] = __ldcg(at);
    jl[i] = __ldcg(at + kRows);
  }
  __syncthreads();
  {
    constexpr int kPer = kThreads / kRows;  // threads a row
    const int r = threadIdx.x / kPer, q0 = threadIdx.x % kPer;
    float mm = neg_inf(), ll = 0.f;
    for (int q = q0; q < my_parts; q += kPer) mm = fmaxf(mm, jm[q * kRows + r]);
#pragma unroll
    for (int d = 1; d < kPer; d <<= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, d));
    for (int q = q0; q < my_parts; q += kPer) {
      const float mq = jm[q * kRows + r], f = mq == mm ? 1.f : exp2_approx(mq - mm);
      ll = fmaf(f, jl[q * kRows + r], ll);
      jm[q * kRows + r] = f;
    }
#pragma unroll
    for (int d = 1; d < kPer; d <<= 1) ll += __shfl_xor_sync(0xffffffffu, ll, d);
    if (q0 == 0) {
      sh.inv[r] = ll == 0.f ? 0.f : 1.f / ll;
      if (r < rows) store_lse(r, mm, ll);
    }
  }
  __syncthreads();
  constexpr int kRowsAtOnce = kThreads / (D / 4);  // a thread has four columns of every kRowsAtOnce-th row
  const int c = 4 * (threadIdx.x % (D / 4)), r0 = threadIdx.x / (D / 4);
  float4 o4[kRows / kRowsAtOnce];
#pragma unroll
  for (int i = 0; i < kRows / kRowsAtOnce; ++i) o4[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int q = 0; q < my_parts; ++q) {
    const float* at = part + q * kPart + c;
#pragma unroll
    for (int i = 0; i < kRows / kRowsAtOnce; ++i) {
      const int r = r0 + i * kRowsAtOnce;
      if (r >= rows) continue;
      const float4 v = __ldcg(reinterpret_cast<const float4*>(at + r * D));
      const float f = jm[q * kRows + r];
      o4[i].x = fmaf(f, v.x, o4[i].x);
      o4[i].y = fmaf(f, v.y, o4[i].y);
      o4[i].z = fmaf(f, v.z, o4[i].z);
      o4[i].w = fmaf(f, v.w, o4[i].w);
    }
  }
#pragma unroll
  for (int i = 0; i < kRows / kRowsAtOnce; ++i) {
    const int r = r0 + i * kRowsAtOnce;
    if (r >= rows) continue;
    const float inv = sh.inv[r];
    *reinterpret_cast<uint2*>(out_at(r) + c) =
        make_uint2(pack2<T>(o4[i].x * inv, o4[i].y * inv), pack2<T>(o4[i].z * inv, o4[i].w * inv));
  }
}

__device__ __forceinline__ float* sh_part_l(uint8_t* smem, int parts) {
  return reinterpret_cast<float*>(smem) + parts * kRows;
}

// Joins the parts of the 16 rows from r0 on of an item: eight threads a row
// weigh the parts, then a thread adds four columns of every so manieth row.
// Rows that are to be done again (flags) are left to that.
template <typename T, int D>
__device__ void join_rows(const PagedParams& p, uint8_t* smem, RowsShared& sh, const PagedItem& it, int r0) {
  constexpr size_t kFloats = 256 * (D + 2);
  constexpr int kPer = kThreads / kRows, kRowsAtOnce = kThreads / (D / 4);
  const float* part = p.tile_part + static_cast<size_t>(it.part) * kFloats;
  float* weight = reinterpret_cast<float*>(smem);  // [part][row]
  const gemm_paged_attention_t& a = p.a;
  auto token_of = [&](int r) {  // of row r0 + r, or -1
    const int in_tile = (r0 + r) % 128, up = by_group(p, in_tile);
    const int token = (2 * it.pair + (r0 + r) / 128) * p.tile_tokens + up;
    return up < p.tile_tokens && token < it.s.n ? token : -1;
  };
  auto head_of = [&](int r) {
    const int in_tile = (r0 + r) % 128;
    return it.head * p.group + in_tile - by_group(p, in_tile) * p.group;
  };
  {
    const int r = threadIdx.x / kPer, q0 = threadIdx.x % kPer;
    float mm = neg_inf(), ll = 0.f;
    int again = 0;
    for (int q = q0; q < p.tile_splits; q += kPer) {
      const float* at = part + q * kFloats + 256 * D + r0 + r;
      again |= p.redo[(it.part + q) * 8 + r0 / 32];
      weight[q * kRows + r] = at[0];
      sh_part_l(smem, p.tile_splits)[q * kRows + r] = at[256];
      mm = fmaxf(mm, at[0]);
    }
#pragma unroll
    for (int d = 1; d < kPer; d <<= 1) {
      mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, d));
      again |= __shfl_xor_sync(0xffffffffu, again, d);
    }
    for (int q = q0; q < p.tile_splits; q += kPer) {
      const float mq = weight[q * kRows + r], lq = sh_part_l(smem, p.tile_splits)[q * kRows + r];
      const float f = lq == 0.f ? 0.f : mq == mm ? 1.f : exp2_approx(mq - mm);
      ll = fmaf(f, lq, ll);
      weight[q * kRows + r] = f;
    }
#pragma unroll
    for (int d = 1; d < kPer; d <<= 1) ll += __shfl_xor_sync(0xffffffffu, ll, d);
    if (q0 == 0) {
      const int token = again ? -1 : token_of(r);
      sh.inv[r] = token < 0 ? -1.f : ll == 0.f ? 0.f : 1.f / ll;  // -1: not stored
      if (token >= 0 && a.lse != nullptr)
        a.lse[(it.s.first + token) * a.heads + head_of(r)] =
            ll == 0.f ? neg_inf() : (mm + log2f(ll)) * 0.6931471805599453f;
    }
  }
  __syncthreads();
  const int c = 4 * (threadIdx.x % (D / 4)), row = threadIdx.x / (D / 4);
  float4 o4[kRows / kRowsAtOnce];
#pragma unroll
  for (int i = 0; i < kRows / kRowsAtOnce; ++i) o4[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int q = 0; q < p.tile_splits; ++q) {
#pragma unroll
    for (int i = 0; i < kRows / kRowsAtOnce; ++i) {
      const int r = row + i * kRowsAtOnce;
      const float4 v = *reinterpret_cast<const float4*>(part + q * kFloats + (r0 + r) * D + c);
      const float f = weight[q * kRows + r];
      o4[i].x = fmaf(f, v.x, o4[i].x);
      o4[i].y = fmaf(f, v.y, o4[i].y);
      o4[i].z = fmaf(f, v.z, o4[i].z);
      o4[i].w = fmaf(f, v.w, o4[i].w);
    }
  }
#pragma unroll
  for (int i = 0; i < kRows / kRowsAtOnce; ++i) {
    const int r = row + i * kRowsAtOnce;
    const float inv = sh.inv[r];
    if (inv < 0.f) continue;
    T* out = static_cast<T*>(a.out) + (it.s.first + token_of(r)) * a.out_token + head_of(r) * a.out_head + c;
    *reinterpret_cast<uint2*>(out) =
        make_uint2(pack2<T>(o4[i].x * inv, o4[i].y * inv), pack2<T>(o4[i].z * inv, o4[i].w * inv));
  }
}

// Unit u of the 16-row kernel: a part of 16 rows of a (sequence, key head).
template <typename T, int D, bool TILED>
__device__ __forceinline__ void take_unit(const PagedParams& p, uint8_t* smem, RowsShared& sh, int u) {
  const gemm_paged_attention_t& a = p.a;
  int id = u;
  const int split = id % p.splits;
  id /= p.splits;
  const int range = id;
  const int row_tile = id % p.row_tiles;
  id /= p.row_tiles;
  const int head = id % a.kv_heads, seq = id / a.kv_heads;
  // Without a window the lane's first page is known before the length is:
  // one round trip to memory less.
  int ahead_col = -1, ahead_page = 0;
  if (a.window == 0) {
    const int64_t tile = static_cast<int64_t>(split) * p.tiles_per + (threadIdx.x >> 5) + (threadIdx.x & 31) * kWarps;
    const int64_t col = tile * kKeys / a.page_size;
    if (col < a.table_width) {
      ahead_col = static_cast<int>(col);
      ahead_page = a.table[seq * a.table_row + col];
    }
  }
  const PagedSeq s = paged_seq(p, seq, split == 0 && row_tile == 0 && threadIdx.x == 0);
  const int64_t rows = static_cast<int64_t>(s.n) * p.group;
  const int row0 = row_tile * kRows;
  if (row0 < rows && (!TILED || rows <= p.few_rows))
    rows_unit<T, D>(p, smem, sh, s, seq, head, row0, static_cast<int>(min(rows - row0, static_cast<int64_t>(kRows))),
                    split, p.splits, range, ahead_col, ahead_page);
}

// (Three blocks an SM with heads of 128, as paged_attention_plan counts on: the
// compiler takes 230 registers by itself, and 4 sequences of 32000 keys 39 us
// for 33.)
template <typename T, int D, bool TILED>
__global__ void __launch_bounds__(kThreads, D == 128 && !TILED ? 3 : 0) paged_rows_kernel(const __grid_constant__ PagedParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ RowsShared sh;
  // Beside the tile kernel, this one starts when all of that one's blocks
  // have: everything before it is complete then, and the rows taken here do
  // not depend on it.  It waits for it below, before it joins its parts, and
  // so ends after it.
  if constexpr (!TILED) grid_dep_wait();
  grid_dep_launch();
  if constexpr (!TILED) {
    take_unit<T, D, TILED>(p, smem, sh, blockIdx.x);
  } else {
    // The blocks that find room beside the tile kernel's take the units one
    // by one; those that start when it has ended find few left.
    for (;;) {
      if (threadIdx.x == 0) sh.unit = atomicAdd(p.queue, 1);
      __syncthreads();
      const int u = sh.unit;
      if (u >= p.units) break;
      take_unit<T, D, TILED>(p, smem, sh, u);
      __syncthreads();  // the shared memory, and sh.unit
    }
    if (threadIdx.x == 0 && atomicAdd(p.queue + 1, 1) == static_cast<int>(gridDim.x) - 1) {
      p.queue[0] = 0;  // every block has found the queue empty
      p.queue[1] = 0;
    }
  }
  if constexpr (TILED) {
    grid_dep_wait();
    const int64_t parts = p.queue[2];
    if (p.tile_splits > 1) {
      constexpr int kUnits = 256 / kRows;
      const int units = static_cast<int>(parts / p.tile_splits) * kUnits;
      for (int u = blockIdx.x; u < units; u += gridDim.x) {
        const PagedItem it = paged_item(p, (u / kUnits) * p.tile_splits, false);
        __syncthreads();  // the shared memory of the rows before
        join_rows<T, D>(p, smem, sh, it, (u % kUnits) * kRows);
      }
    }
    // Items with results that are not finite: a value that a row must not see
    // may have got into it (0 times an infinity), so those rows are computed
    // again here, 16 at a time, where that cannot happen.  The units are dealt
    // out to the blocks one by one.
    const int64_t units = parts * 16, grid = gridDim.x;
    for (int64_t base = blockIdx.x; base < units; base += grid * kThreads) {
      const int64_t mine = base + threadIdx.x * grid;
      const unsigned flagged = __ballot_sync(0xffffffffu, mine < units && p.redo[mine / 2] != 0);
      if ((threadIdx.x & 31) == 0) sh.redo[threadIdx.x / 32] = flagged;
      if (!__syncthreads_or(flagged != 0)) continue;
      for (int t = 0; t < kThreads; ++t) {
        if ((sh.redo[t / 32] >> (t % 32) & 1) == 0) continue;
        const int64_t u = base + t * grid;
        const int w = static_cast<int>(u % 16) / 2, half = static_cast<int>(u % 2);
        const PagedItem it = paged_item(p, static_cast<int>(u / 16), false);
        if (!it.valid) break;
        // the same rows' other parts: the first one that is flagged has them done
        bool done = false;
        for (int q = 1; q <= it.split; ++q) done |= p.redo[(it.part - q) * static_cast<int64_t>(8) + w] != 0;
        const int tile_rows = p.tile_tokens * p.group;
        const int tile0 = (2 * it.pair + w / 4) * tile_rows;
        const int64_t end = min(static_cast<int64_t>(tile0) + tile_rows, static_cast<int64_t>(it.s.n) * p.group);
        const int row0 = tile0 + (w % 4) * 32 + half * kRows;
        if (done || row0 >= end) continue;
        __syncthreads();  // the shared memory of the rows before
        rows_unit<T, D>(p, smem, sh, it.s, it.seq, it.head, row0,
                        static_cast<int>(min(end - row0, static_cast<int64_t>(kRows))), 0, 1, 0, -1, 0);
      }
      __syncthreads();  // sh.redo is written again
    }
  }
}

template <typename T, int D, bool TILED>
cudaError_t launch_rows_as(const PagedParams& p, int grid, cudaStream_t stream) {
  constexpr int most = ring_bytes(D, kDeepStages);
  const size_t smem = ring_bytes(D, p.row_stages);
  static std::atomic<uint64_t> attr_done{0};
  cudaError_t e = once_per_device(attr_done, [] {
    return cudaFuncSetAttribute(paged_rows_kernel<T, D, TILED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                most);
  });
  if (e != cudaSuccess) return e;
  if (!TILED) last_main_launch() = LaunchShape{dim3(static_cast<unsigned>(grid)), dim3(kThreads), smem, 1, true};
  return launch_pdl(paged_rows_kernel<T, D, TILED>, dim3(static_cast<unsigned>(grid)), dim3(kThreads), smem, stream, p);
}

template <typename T, int D>
cudaError_t launch_rows(const PagedParams& p, int grid, cudaStream_t stream) {
  return p.tiled ? launch_rows_as<T, D, true>(p, grid, stream) : launch_rows_as<T, D, false>(p, grid, stream);
}

int64_t most_keys(const gemm_paged_attention_t& a) {
  const int64_t most = static_cast<int64_t>(a.table_width) * a.page_size;
  return a.max_kv > 0 ? std::min(a.max_kv, most) : most;
}

// Key tiles of 16 that the longest range of the 16-row kernel has.
int64_t row_key_tiles(const gemm_paged_attention_t& a) {
  int64_t keys = most_keys(a);
  if (a.window > 0) keys = std::min<int64_t>(keys, static_cast<int64_t>(a.window) + kRows - 1 + kKeys);
  return (keys + kKeys - 1) / kKeys;
}

}  // namespace

PagedPlan paged_attention_plan(const gemm_paged_attention_t& a, int sms) {
  PagedPlan plan{};
  const int64_t group = a.heads / a.kv_heads;
  const int64_t max_rows = a.max_q * group;
  plan.tiled = max_rows > kPagedFewRows && group <= kPagedMostGroup;
  const int64_t row_tiles = ((plan.tiled ? kPagedFewRows : max_rows) + kRows - 1) / kRows;
  const int64_t ranges = static_cast<int64_t>(a.sequences) * a.kv_heads * row_tiles;
  // Parts of a range.  A part more costs the join of a range about 0.1 us
  // and saves every warp of the others a share of its tiles, 1.2 us each: the
  // sum is least near sqrt(3.3 tiles) parts (one token against 1001, 4001,
  // 8001 and 32001 keys: 9.3, 11.5, 13.7 and 20.7 us there; 16.7, 14.9, 15.9
  // and 20.7 in a quarter to an eighth as many parts, 9.3, 13.5, 19.3 and 36.5
  // in parts of a tile a warp).  Up to there: all blocks on the SMs at once
  // (three an SM), or for long ranges eight an SM, because the sequences of a
  // call differ in length and the shorter ones leave parts empty, but then at
  // least 32 tiles in each and two rounds of blocks: with one and a bit, 4
  // sequences of 32000 keys took 44.7 us for 33.7, 8 of 16000 40.9 for 30.3.
  const int64_t tiles = row_key_tiles(a), per_range = std::max<int64_t>(ranges, 1);
  const int64_t wave = 3 * static_cast<int64_t>(sms);
  int64_t want = std::min<int64_t>(ranges * (tiles / 32), 8 * static_cast<int64_t>(sms));
  if (want < 2 * wave) want = wave;
  int64_t splits = std::max<int64_t>(1, want / per_range);
  splits = std::min(splits, static_cast<int64_t>(std::sqrt(3.3 * static_cast<double>(tiles))));
  splits = std::min(splits, kPagedMostSplits);
  splits = std::max<int64_t>(1, std::min<int64_t>(splits, kPagedParts / per_range));
  plan.row_splits = static_cast<int>(splits);
  plan.row_grid = static_cast<int>(ranges * splits);
  // Deeper rings while they leave every block its place on an SM: one token in
  // 64 sequences of 1 to 256 keys, 6 heads of 64, 8.2 us with two tiles and 7.4
  // with four; with more blocks than places two are ahead (200 sequences of 1
  // to 500 keys: 23.0 for 26.8).
  const int64_t deep = 227 * 1024 / ring_bytes(a.head_dim, kDeepStages) * static_cast<int64_t>(sms);
  plan.row_stages = !plan.tiled && plan.row_grid <= deep ? kDeepStages : kStages;
  plan.tile_rows = kRows;
  plan.tile_keys = kKeys;
  plan.stages = plan.row_stages;
  plan.splits = plan.row_splits;
  plan.grid = plan.row_grid;
  plan.kernels = 1;
  if (!plan.tiled) return plan;
  // Items of the tile kernel: an upper bound from the call's tokens (a sequence
  // adds at most one item that is not full, and has more than kPagedFewRows rows).
  const int64_t pair_tokens = 2 * (128 / group);
  const int64_t long_seqs = std::min<int64_t>(a.sequences, a.tokens * group / (kPagedFewRows + 1));
  const int64_t most = std::max<int64_t>(1, a.kv_heads * (a.tokens / pair_tokens + long_seqs));
  int64_t keys = most_keys(a);
  if (a.window > 0) keys = std::min<int64_t>(keys, a.window + pair_tokens - 1 + 128);
  const int64_t blocks = (keys + 127) / 128;
  // About as many as there are: sequences of max_q new tokens each.
  auto pairs = [&](int64_t n) { return (n + pair_tokens - 1) / pair_tokens; };
  const int64_t items = std::min(
      most, std::max<int64_t>(1, a.kv_heads * (a.tokens / a.max_q * pairs(a.max_q) + pairs(a.tokens % a.max_q))));
  // Their keys are split into parts of at least four blocks so that the rounds
  // of parts on the SMs are short.  A part costs about five blocks beside its
  // own: 7 chunks of 320 tokens, 12 heads, against 7600 keys, 168 items, took
  // 322 us whole and 248 in three parts; 3 of 400, 16 heads over 4, against
  // 2000 keys, 84 items, 69 us in two parts, 65 in three and 43 whole.
  const int64_t most_parts =
      std::max<int64_t>(1, std::min({blocks / 4, kPagedTileParts / most, kPagedMostSplits}));
  auto cost = [&](int64_t n) { return (items * n + sms - 1) / sms * ((blocks + n - 1) / n + 5); };
  int64_t parts = 1;
  for (int64_t rounds = 1; rounds <= 8; ++rounds) {
    const int64_t n = std::max<int64_t>(1, std::min(rounds * sms / items, most_parts));
    if (cost(n) < cost(parts)) parts = n;
  }
  plan.tile_splits = static_cast<int>(parts);
  plan.tile_parts = most * parts;
  plan.tile_grid = static_cast<int>(std::min<int64_t>(sms, plan.tile_parts));
  plan.row_grid = static_cast<int>(
      std::min<int64_t>(3 * sms, std::max<int64_t>(plan.row_grid, parts > 1 ? most * 16 : most)));
  plan.tile_rows = 128;
  plan.tile_keys = 128;
  plan.stages = a.head_dim == 128 ? 5 : 8;
  plan.splits = plan.tile_splits;
  plan.grid = plan.tile_grid;
  plan.kernels = 2;
  return plan;
}

size_t paged_scratch_bytes(const PagedPlan& plan, int head_dim) {
  size_t bytes = kPagedRowScratch;
  if (plan.tiled) {
    bytes += (static_cast<size_t>(plan.tile_parts) * 8 + 255) / 256 * 256;
    if (plan.tile_splits > 1) bytes += static_cast<size_t>(plan.tile_parts) * 256 * (head_dim + 2) * sizeof(float);
  }
  return bytes;
}

cudaError_t launch_paged_attention(const gemm_paged_attention_t& a, const PagedPlan& plan, void* scratch, int sms,
                                   uint64_t wait_ns, int* status, cudaStream_t stream) {
  PagedParams p{};
  p.a = a;
  p.group = a.heads / a.kv_heads;
  p.group_inv = static_cast<uint32_t>((0x100000000ull + p.group - 1) / p.group);
  p.tiled = plan.tiled;
  p.few_rows = kPagedFewRows;
  p.row_tiles = static_cast<int>(((plan.tiled ? kPagedFewRows : static_cast<int64_t>(a.max_q) * p.group) + kRows - 1) / kRows);
  p.splits = plan.row_splits;
  p.row_stages = plan.row_stages;
  const int64_t tiles = row_key_tiles(a);
  p.tiles_per = static_cast<int>(std::max<int64_t>(1, (tiles + p.splits - 1) / p.splits));
  // A warp has every fourth tile of a part.  Where that is one to four tiles
  // and every block has an SM, parts of whole rounds: fewer to join, the longest
  // warp no longer (one token against 1001 and 8001 keys 9.1 and 13.3 us
  // without, 8.6 and 12.0 so; with three blocks an SM 9.6 and 10.1).
  if (plan.row_grid <= sms && p.tiles_per > kWarps && p.tiles_per < 4 * kWarps)
    p.tiles_per = (p.tiles_per + kWarps - 1) / kWarps * kWarps;
  p.units = a.sequences * a.kv_heads * p.row_tiles * p.splits;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  const float cap = a.softcap <= kCapNone ? a.softcap : 0.f;
  p.cap_in = cap > 0.f ? a.scale / cap : 0.f;
  p.cap_out = cap * 1.4426950408889634f;
  p.cap_shared = cap > 0.f && cap <= kCapShared;
  p.cap_in2 = 2.885390081777927f * p.cap_in;
  char* at = static_cast<char*>(scratch);
  p.arrived = reinterpret_cast<int*>(at);
  p.queue = p.arrived + kPagedParts;
  p.part = reinterpret_cast<float*>(at + (kPagedParts + 64) * sizeof(int));
  p.status = status;
  if (plan.tiled) {
    p.tile_tokens = 128 / p.group;
    // (a scale of 0 as a tiny one, of which an infinity is still one)
    p.s_scale = p.cap_shared ? 2.f * p.cap_out
                : cap > 0.f  ? p.cap_out
                             : std::max(std::fabs(p.scale_log2), 1e-30f);
    p.flip = cap == 0.f && p.scale_log2 < 0.f;
    p.tile_splits = plan.tile_splits;
    p.tile_parts = static_cast<int>(plan.tile_parts);
    p.box = 16;
    while (p.box < 128 && a.page_size % (2 * p.box) == 0) p.box *= 2;
    p.redo = reinterpret_cast<uint8_t*>(at + kPagedRowScratch);
    p.tile_part = reinterpret_cast<float*>(at + kPagedRowScratch + (static_cast<size_t>(plan.tile_parts) * 8 + 255) / 256 * 256);
    p.wait_ns = wait_ns > 0 ? wait_ns : kWaitLimitNs;
    p.out_v8 = (reinterpret_cast<uintptr_t>(a.out) % 32 == 0 && (a.out_token | a.out_head) % 16 == 0) ? 1 : 0;
    const cudaError_t e = launch_paged_tiles(p, plan.tile_grid, stream);
    if (e != cudaSuccess) return e;
  }
  if (a.type == GEMM_TYPE_BF16)
    return a.head_dim == 64 ? launch_rows<__nv_bfloat16, 64>(p, plan.row_grid, stream)
                            : launch_rows<__nv_bfloat16, 128>(p, plan.row_grid, stream);
  return a.head_dim == 64 ? launch_rows<__half, 64>(p, plan.row_grid, stream)
                          : launch_rows<__half, 128>(p, plan.row_grid, stream);
}

}  // namespace dgt
