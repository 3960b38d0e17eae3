// pages.cu -- the sequences and pages of a cache, on the device: growing,
// shrinking, forking, compacting, copying.
//
// The whole numbers are exact and do not depend on the order in which the
// blocks run: pages are taken by rank, the lowest free page first, and the
// ranks come from prefix sums.  The calls that need ranks run one kernel
// whose blocks each list the free (and used) pages of a segment of `refs`;
// the block that finishes last has every segment's counts, and does the rest
// of the call alone, so that a decode step costs one launch.  Moving the
// pages' bytes (a fork's last pages, compaction, a page that a growing sequence
// shares) is a second kernel that reads how many there are on the device; it is
// bound by HBM, 2 x the bytes: 794 MB of reads and writes take 137 us with the
// ranks before them, 5.8 TB/s.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"

namespace dgt {
namespace {

constexpr int kIdxThreads = 1024;
constexpr int kIdxWarps = kIdxThreads / 32;
constexpr int kIdxBatch = 4;                         // refs a thread reads at a time
constexpr int kIdxChunk = kIdxThreads * kIdxBatch;   // pages a block lists at a time
constexpr int kIdxBlocks = 128;                      // most blocks (segments)
constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 8;                         // 16-byte vectors a lane keeps in flight

// Scratch: a header of counters, then lists of pages and per-call arrays.
struct IdxHeader {
  unsigned ticket;  // blocks done, zero between calls
  int moves;        // pairs in src / dst
  int live;         // pages in use (compact)
  int ok;           // the call changes anything (fork)
  int free_count[kIdxBlocks], live_count[kIdxBlocks];
};

struct Scratch {
  IdxHeader* head;
  int32_t* free_list;  // segment s's free pages, ascending, from s * seg on
  int32_t* live_list;  // and its pages in use
  int32_t *src, *dst;  // pairs of pages to copy
  int32_t* map;        // compact: new place of a page that moves, -1 for a free one
  int32_t *at, *before, *token;  // per sequence of the call: first rank, length, first token
};

constexpr size_t kHeaderBytes = (sizeof(IdxHeader) + 255) / 256 * 256;

__host__ __device__ inline int64_t round_256(int64_t x) { return (x + 63) / 64 * 64; }

Scratch scratch_at(void* base, int64_t pages, int64_t n) {
  Scratch s;
  s.head = static_cast<IdxHeader*>(base);
  int32_t* p = reinterpret_cast<int32_t*>(static_cast<char*>(base) + kHeaderBytes);
  const int64_t np = round_256(pages), nn = round_256(n + 1);
  s.free_list = p;
  s.live_list = p + np;
  s.map = p + 2 * np;
  s.src = p + 3 * np;
  s.dst = s.src + std::max(np, nn);
  s.at = s.dst + std::max(np, nn);
  s.before = s.at + nn;
  s.token = s.before + nn;
  return s;
}

struct PageState {
  int32_t *table, *lens, *refs;
  int64_t table_row;
  int sequences, width, page_size, pages, seg;  // seg: pages a block lists
  int* status;
};

PageState state_of(const gemm_cache_t& c, int* status) {
  PageState s;
  s.table = c.table;
  s.lens = c.lens;
  s.refs = c.refs;
  s.table_row = c.table_row;
  s.sequences = c.sequences;
  s.width = c.table_width;
  s.page_size = c.page_size;
  s.pages = static_cast<int>(c.num_pages);
  int blocks = static_cast<int>(std::min<int64_t>((c.num_pages + kIdxChunk - 1) / kIdxChunk, kIdxBlocks));
  blocks = std::max(blocks, 1);
  const int64_t per = (c.num_pages + blocks - 1) / blocks;
  s.seg = static_cast<int>(std::max<int64_t>((per + kIdxChunk - 1) / kIdxChunk, 1) * kIdxChunk);
  s.status = status;
  return s;
}
int idx_blocks(const PageState& s) { return std::max(1, (s.pages + s.seg - 1) / s.seg); }

// Inclusive sum over the block; `part` holds kIdxWarps values.  The total is
// in *total for every thread.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* part, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  __syncthreads();  // the previous use of `part`
  if (lane == 31) part[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int64_t w = part[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, w, d);
      if (lane >= d) w += o;
    }
    part[lane] = w;
  }
  __syncthreads();
  *total = part[kIdxWarps - 1];
  return v + (warp > 0 ? part[warp - 1] : 0);
}

struct IdxShared {
  int64_t part[kIdxWarps];
  int cnt[kIdxBatch][kIdxWarps];
  int free_at[kIdxBlocks + 1], live_at[kIdxBlocks + 1];  // ranks of the segments' first pages
  int last;
};

// Lists the free pages (and with `live` the used ones) of this block's
// segment, ascending, and with `live` gives the free ones no place in ws.map;
// returns true in the block that finishes last, with the
// segments' ranks in sh.free_at / live_at.
__device__ bool list_pages(const PageState& st, const Scratch& ws, IdxShared& sh, bool live) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * st.seg;
  const int64_t end = min(first + st.seg, static_cast<int64_t>(st.pages));
  int n_free = 0, n_live = 0;
  for (int64_t base = first; base < end; base += kIdxChunk) {
    int r[kIdxBatch];
#pragma unroll
    for (int u = 0; u < kIdxBatch; ++u) {
      const int64_t i = base + u * kIdxThreads + threadIdx.x;
      r[u] = i < end ? st.refs[i] : -1;
    }
    unsigned m[kIdxBatch];
#pragma unroll
    for (int u = 0; u < kIdxBatch; ++u) {
      m[u] = __ballot_sync(0xffffffffu, r[u] == 0);
      if (lane == 0) sh.cnt[u][warp] = __popc(m[u]);
    }
    __syncthreads();
    // exclusive sums over the (batch, warp) counts, in page order
    if (warp < kIdxBatch) {
      int v = sh.cnt[warp][lane];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += o;
      }
      sh.cnt[warp][lane] = v;  // inclusive within the batch
    }
    __syncthreads();
    int before = 0;
#pragma unroll
    for (int u = 0; u < kIdxBatch; ++u) {
      const int rank = before + (warp > 0 ? sh.cnt[u][warp - 1] : 0) + __popc(m[u] & ((1u << lane) - 1u));
      const int64_t i = base + u * kIdxThreads + threadIdx.x;
      if (r[u] == 0) {
        ws.free_list[first + n_free + rank] = static_cast<int32_t>(i);
        if (live) ws.map[i] = -1;
      }
      if (live && r[u] != 0 && i < end) ws.live_list[first + n_live + static_cast<int>(i - base) - rank] = static_cast<int32_t>(i);
      before += sh.cnt[u][kIdxWarps - 1];
    }
    n_free += before;
    n_live += static_cast<int>(min(static_cast<int64_t>(kIdxChunk), end - base)) - before;
    __syncthreads();  // sh.cnt is written again
  }
  if (threadIdx.x == 0) {
    ws.head->free_count[blockIdx.x] = n_free;
    ws.head->live_count[blockIdx.x] = n_live;
  }
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    const bool last = atomicAdd(&ws.head->ticket, 1u) == gridDim.x - 1;
    if (last) ws.head->ticket = 0;
    sh.last = last ? 1 : 0;
  }
  __syncthreads();
  if (!sh.last) return false;
  __threadfence();
  if (threadIdx.x == 0) {
    int f = 0, l = 0;
    for (unsigned s = 0; s < gridDim.x; ++s) {
      sh.free_at[s] = f;
      sh.live_at[s] = l;
      f += __ldcg(&ws.head->free_count[s]);
      l += __ldcg(&ws.head->live_count[s]);
    }
    sh.free_at[gridDim.x] = f;
    sh.live_at[gridDim.x] = l;
  }
  __syncthreads();
  return true;
}

// The page of rank r in the segments' lists (r below the total).
__device__ __forceinline__ int32_t page_of(const int32_t* list, const int* at, int seg, int r) {
  int lo = 0, hi = static_cast<int>(gridDim.x);
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (at[mid] <= r) lo = mid; else hi = mid;
  }
  return __ldcg(list + static_cast<int64_t>(lo) * seg + (r - at[lo]));
}

__device__ __forceinline__ int pages_for(int tokens, int page_size) {
  return tokens / page_size + (tokens % page_size != 0);
}

// A sequence's length, brought into what its table row can hold.
__device__ __forceinline__ int length_of(const PageState& st, int seq) {
  const int n = st.lens[seq];
  const int64_t most = static_cast<int64_t>(st.width) * st.page_size;
  if (n < 0 || n > most) {
    atomicExch(st.status, kDevBadIndex);
    return n < 0 ? 0 : static_cast<int>(most);
  }
  return n;
}

// The page of a table entry, or -1 (reported) when there is no such page.
__device__ __forceinline__ int checked_page(const PageState& st, int page) {
  if (page >= 0 && page < st.pages) return page;
  atomicExch(st.status, kDevBadIndex);
  return -1;
}

__device__ __forceinline__ bool checked_seq(const PageState& st, int seq) {
  if (seq >= 0 && seq < st.sequences) return true;
  atomicExch(st.status, kDevBadIndex);
  return false;
}

__global__ void __launch_bounds__(kIdxThreads)
    cache_grow_kernel(const PageState st, const Scratch ws, int n, const int32_t* seqs, const int32_t* counts,
                      int tokens, int64_t* positions, int64_t* slots, int32_t* info, int copies) {
  __shared__ IdxShared sh;
  __shared__ int moves;
  grid_dep_wait();
  grid_dep_launch();
  if (!list_pages(st, ws, sh, false)) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t need = 0, token = 0;  // totals so far
  int refused = 0;
  for (int base = 0; base < n; base += kIdxThreads) {
    const int i = base + threadIdx.x;
    int64_t take = 0;
    int add = 0, no = 0, before = 0;
    if (i < n) {
      const int seq = seqs[i];
      add = counts[i];
      if (add < 0) {
        atomicExch(st.status, kDevBadIndex);
        add = 0;
      }
      if (checked_seq(st, seq)) {
        before = length_of(st, seq);
        const int64_t after = static_cast<int64_t>(before) + add;
        if (after > static_cast<int64_t>(st.width) * st.page_size) no = 1;
        take = (after + st.page_size - 1) / st.page_size - pages_for(before, st.page_size);
        if (add > 0 && before % st.page_size != 0) {
          const int page = checked_page(st, st.table[seq * st.table_row + before / st.page_size]);
          if (page >= 0 && st.refs[page] > 1) {
            // Another sequence holds the page that the tokens would go to (a
            // shrink has cut into a page that a fork shares): a copy of it is
            // the first page taken.
            ++take;
            if (!copies) no = 1;
            before = ~before;
          }
        }
      } else {
        no = 1;
      }
    }
    int64_t sum;
    int64_t incl = block_scan(take, sh.part, &sum);
    if (i < n) {
      ws.at[i] = static_cast<int32_t>(need + incl - take);  // (read where all of them are there)
      ws.before[i] = before;
    }
    need += sum;
    incl = block_scan(add, sh.part, &sum);
    if (i < n) ws.token[i] = static_cast<int32_t>(min(token + incl - add, static_cast<int64_t>(INT32_MAX)));
    token += sum;
    refused += __syncthreads_count(no);
  }
  const int64_t missing = max(static_cast<int64_t>(0), need - sh.free_at[gridDim.x]);
  const bool ok = missing == 0 && refused == 0;
  if (threadIdx.x == 0) {
    info[0] = ok ? static_cast<int32_t>(need) : 0;
    info[1] = static_cast<int32_t>(min(missing, static_cast<int64_t>(INT32_MAX)));
    info[2] = refused;
    if (tokens != token) atomicExch(st.status, kDevBadIndex);
    moves = 0;
    if (!ok) ws.head->moves = 0;
  }
  __syncthreads();  // ws.at, before, token, moves
  if (positions != nullptr || slots != nullptr) {
    for (int t = threadIdx.x; t < tokens; t += kIdxThreads) {
      int64_t position = 0, slot = -1;
      if (t < token) {
        int lo = 0, hi = n;  // the last sequence whose first token is <= t (empty ones have the next one's)
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (ws.token[mid] <= t) lo = mid; else hi = mid;
        }
        const int own = ws.before[lo] < 0 ? 1 : 0;
        const int before = own ? ~ws.before[lo] : ws.before[lo];
        position = static_cast<int64_t>(before) + (t - ws.token[lo]);
        if (ok) {
          const int pos = static_cast<int>(position);
          const int j = pos / st.page_size, held = pages_for(before, st.page_size) - own;
          const int page = j < held ? checked_page(st, st.table[seqs[lo] * st.table_row + j])
                                    : page_of(ws.free_list, sh.free_at, st.seg, ws.at[lo] + j - held);
          if (page >= 0) slot = static_cast<int64_t>(page) * st.page_size + pos % st.page_size;
        }
      }
      if (positions != nullptr) positions[t] = position;
      if (slots != nullptr) slots[t] = slot;
    }
  }
  __syncthreads();  // the table has been read
  if (!ok) return;
  for (int i = warp; i < n; i += kIdxWarps) {
    const int own = ws.before[i] < 0 ? 1 : 0;
    const int seq = seqs[i], before = own ? ~ws.before[i] : ws.before[i];
    const int after = before + max(counts[i], 0);
    const int held = pages_for(before, st.page_size) - own, wanted = pages_for(after, st.page_size);
    for (int j = held + lane; j < wanted; j += 32) {
      const int page = page_of(ws.free_list, sh.free_at, st.seg, ws.at[i] + j - held);
      int32_t* entry = st.table + seq * st.table_row + j;
      if (own && j == held) {
        const int to = atomicAdd(&moves, 1);  // (the order of the pairs makes no difference)
        ws.src[to] = *entry;
        ws.dst[to] = page;
        atomicSub(st.refs + *entry, 1);
      }
      *entry = page;
      st.refs[page] = 1;
    }
    if (lane == 0) st.lens[seq] = after;
  }
  __syncthreads();
  if (threadIdx.x == 0) ws.head->moves = moves;
}

// One warp a sequence.
__global__ void __launch_bounds__(256)
    cache_shrink_kernel(const PageState st, int n, const int32_t* seqs, const int32_t* counts) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int i = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (i >= n) return;
  const int seq = seqs[i];
  if (seq < 0 || seq >= st.sequences) {
    if (lane == 0) atomicExch(st.status, kDevBadIndex);
    return;
  }
  const int before = length_of(st, seq);
  int drop = counts != nullptr ? counts[i] : before;
  if (drop < 0) {
    if (lane == 0) atomicExch(st.status, kDevBadIndex);
    drop = 0;
  }
  const int after = max(before - drop, 0);
  const int held = pages_for(before, st.page_size), keep = pages_for(after, st.page_size);
  __syncwarp();
  for (int j = keep + lane; j < held; j += 32) {
    int32_t* entry = st.table + seq * st.table_row + j;
    const int page = checked_page(st, *entry);
    if (page >= 0) atomicSub(st.refs + page, 1);
    *entry = -1;
  }
  if (lane == 0) st.lens[seq] = after;
}

__global__ void __launch_bounds__(kIdxThreads)
    cache_fork_kernel(const PageState st, const Scratch ws, int n, const int32_t* parents, const int32_t* children,
                      int32_t* copied, int32_t* info) {
  __shared__ IdxShared sh;
  grid_dep_wait();
  grid_dep_launch();
  if (!list_pages(st, ws, sh, false)) return;
  int need = 0, refused = 0;
  for (int base = 0; base < n; base += kIdxThreads) {
    const int i = base + threadIdx.x;
    int take = 0, no = 0, len = 0;
    if (i < n) {
      const int parent = parents[i], child = children[i];
      if (checked_seq(st, parent) && checked_seq(st, child)) {
        len = length_of(st, parent);
        take = len % st.page_size != 0;
        no = st.lens[child] != 0;
      } else {
        no = 1;
      }
    }
    int64_t sum;
    const int64_t incl = block_scan(take, sh.part, &sum);
    if (i < n) {
      ws.at[i] = take ? need + static_cast<int>(incl) - 1 : -1;
      ws.before[i] = len;
    }
    need += static_cast<int>(sum);
    refused += __syncthreads_count(no);
  }
  const int missing = max(0, need - sh.free_at[gridDim.x]);
  const bool ok = missing == 0 && refused == 0;
  if (threadIdx.x == 0) {
    info[0] = ok ? need : 0;
    info[1] = missing;
    info[2] = refused;
    ws.head->moves = ok ? need : 0;
    ws.head->ok = ok ? 1 : 0;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kIdxThreads) {
    int page = -1;
    if (ok) {
      const int r = ws.at[i], len = ws.before[i];
      if (r >= 0) {
        page = page_of(ws.free_list, sh.free_at, st.seg, r);
        ws.src[r] = checked_page(st, st.table[parents[i] * st.table_row + len / st.page_size]);
        ws.dst[r] = page;
      }
      st.lens[children[i]] = len;
    }
    copied[i] = page;
  }
}

__global__ void __launch_bounds__(kIdxThreads)
    cache_compact_kernel(const PageState st, const Scratch ws, int32_t* info) {
  __shared__ IdxShared sh;
  __shared__ int below;  // pages in use below `live`
  grid_dep_wait();
  grid_dep_launch();
  if (!list_pages(st, ws, sh, true)) return;
  const int live = sh.live_at[gridDim.x], free_pages = sh.free_at[gridDim.x];
  if (threadIdx.x == 0) {
    // The first page in use at or beyond `live` by bisection over the ranks.
    int lo = 0, hi = live;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (page_of(ws.live_list, sh.live_at, st.seg, mid) < live) lo = mid + 1; else hi = mid;
    }
    below = lo;
  }
  __syncthreads();
  const int moves = min(live - below, free_pages);  // equal unless refs holds negative counts
  for (int i = threadIdx.x; i < moves; i += kIdxThreads) {
    const int src = page_of(ws.live_list, sh.live_at, st.seg, below + i);
    const int dst = page_of(ws.free_list, sh.free_at, st.seg, i);
    ws.src[i] = src;
    ws.dst[i] = dst;
    ws.map[src] = dst;
    st.refs[dst] = st.refs[src];
    st.refs[src] = 0;
  }
  if (threadIdx.x == 0) {
    info[0] = moves;
    info[1] = live;
    ws.head->moves = moves;
    ws.head->live = live;
  }
}

struct CopyParams {
  char* base[8];
  int64_t group_stride[8], page_stride[8];
  int first_group[9];  // groups before pool i
  int pools, groups, pages;
  int vecs;            // 16-byte vectors a page
  const int *src, *dst;
  const int* count;    // device count of pairs, or null: n
  int n;
  int* status;
};

CopyParams copy_params(const gemm_cache_t& c, int* status) {
  CopyParams p{};
  p.pools = c.pool_count;
  for (int i = 0; i < c.pool_count; ++i) {
    p.base[i] = static_cast<char*>(c.pools[i]);
    p.group_stride[i] = c.pool_group_stride[i];
    p.page_stride[i] = c.pool_page_stride[i];
    p.first_group[i + 1] = p.first_group[i] + static_cast<int>(c.pool_groups[i]);
  }
  p.groups = p.first_group[c.pool_count];
  p.pages = static_cast<int>(c.num_pages);
  p.vecs = static_cast<int>(c.page_bytes / 16);
  p.status = status;
  return p;
}

// A warp copies pieces of 32 x kCopyVecs vectors (4 KB), all loads before the
// first store; pieces of one page lie next to one another.
__device__ void copy_pairs(const CopyParams& p, int64_t warp, int64_t warps) {
  const int lane = threadIdx.x & 31;
  const int n = p.count != nullptr ? *p.count : p.n;
  const int pieces = (p.vecs + 32 * kCopyVecs - 1) / (32 * kCopyVecs);
  const int64_t per_pair = static_cast<int64_t>(pieces) * p.groups;
  for (int64_t w = warp; w < per_pair * n; w += warps) {
    const int pair = static_cast<int>(w / per_pair);
    const int rest = static_cast<int>(w - pair * per_pair);
    const int group = rest / pieces, piece = rest - group * pieces;
    const int src = p.src[pair], dst = p.dst[pair];
    if (src < 0 || src >= p.pages || dst < 0 || dst >= p.pages) {
      if (lane == 0) atomicExch(p.status, kDevBadIndex);
      continue;
    }
    int pool = 0;
    while (group >= p.first_group[pool + 1]) ++pool;
    char* base = p.base[pool] + (group - p.first_group[pool]) * p.group_stride[pool];
    const uint4* from = reinterpret_cast<const uint4*>(base + src * p.page_stride[pool]);
    uint4* to = reinterpret_cast<uint4*>(base + dst * p.page_stride[pool]);
    const int v0 = piece * 32 * kCopyVecs + lane;
    uint4 x[kCopyVecs];
#pragma unroll
    for (int u = 0; u < kCopyVecs; ++u)
      if (v0 + 32 * u < p.vecs) x[u] = from[v0 + 32 * u];
#pragma unroll
    for (int u = 0; u < kCopyVecs; ++u)
      if (v0 + 32 * u < p.vecs) to[v0 + 32 * u] = x[u];
  }
}

__global__ void __launch_bounds__(kCopyThreads) cache_copy_kernel(const __grid_constant__ CopyParams p) {
  grid_dep_wait();
  grid_dep_launch();
  copy_pairs(p, static_cast<int64_t>(blockIdx.x) * (kCopyThreads / 32) + (threadIdx.x >> 5),
             static_cast<int64_t>(gridDim.x) * (kCopyThreads / 32));
}

// The children's rows of the table (a warp each), then the pages.
__global__ void __launch_bounds__(kCopyThreads)
    cache_fork_copy_kernel(const PageState st, const Scratch ws, int n, const int32_t* parents,
                           const int32_t* children, const int32_t* copied, const __grid_constant__ CopyParams p) {
  grid_dep_wait();
  grid_dep_launch();
  if (ws.head->ok == 0) return;
  const int lane = threadIdx.x & 31;
  const int64_t warp = static_cast<int64_t>(blockIdx.x) * (kCopyThreads / 32) + (threadIdx.x >> 5);
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kCopyThreads / 32);
  for (int64_t i = warp; i < n; i += warps) {
    const int len = ws.before[i], full = len / st.page_size, last = copied[i];
    const int32_t* from = st.table + parents[i] * st.table_row;
    int32_t* to = st.table + children[i] * st.table_row;
    for (int j = lane; j < st.width; j += 32) {
      int page = -1;
      if (j < full) {
        page = checked_page(st, from[j]);
      } else if (j == full) {
        page = last;
      }
      if (page >= 0) atomicAdd(st.refs + page, 1);
      to[j] = page;
    }
  }
  copy_pairs(p, warp, warps);
}

// The table's entries of pages that move, then the pages.
__global__ void __launch_bounds__(kCopyThreads)
    cache_compact_copy_kernel(const PageState st, const Scratch ws, const __grid_constant__ CopyParams p) {
  grid_dep_wait();
  grid_dep_launch();
  const int live = ws.head->live, moves = ws.head->moves;
  if (moves == 0) return;
  const int64_t entries = static_cast<int64_t>(st.sequences) * st.width;
  const int64_t threads = static_cast<int64_t>(gridDim.x) * kCopyThreads;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x; e < entries; e += threads) {
    int32_t* entry = st.table + e / st.width * st.table_row + e % st.width;
    const int page = *entry;
    if (page < live) continue;  // stays (or -1)
    // in use, as a table holds it, and so moved; a page that refs calls free
    // has no new place
    const int to = page < st.pages ? ws.map[page] : -1;
    if (to >= 0)
      *entry = to;
    else
      atomicExch(st.status, kDevBadIndex);
  }
  copy_pairs(p, static_cast<int64_t>(blockIdx.x) * (kCopyThreads / 32) + (threadIdx.x >> 5),
             static_cast<int64_t>(gridDim.x) * (kCopyThreads / 32));
}

// Eight blocks an SM at most: 64 warps x 4 KB in flight.
int copy_grid(const CopyParams& p, int64_t pairs, int64_t other_warps, int sms) {
  const int pieces = (p.vecs + 32 * kCopyVecs - 1) / (32 * kCopyVecs);
  const int64_t warps = std::max<int64_t>(pairs * pieces * p.groups, other_warps);
  const int64_t blocks = (warps + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(blocks, 8 * static_cast<int64_t>(sms))));
}

}  // namespace

size_t cache_scratch_bytes(int64_t num_pages, int64_t n) {
  const int64_t np = round_256(num_pages), nn = round_256(n + 1);
  return kHeaderBytes + static_cast<size_t>(3 * np + 2 * std::max(np, nn) + 3 * nn) * sizeof(int32_t);
}

cudaError_t launch_cache_grow(const gemm_cache_t& c, int64_t n, const int32_t* seqs, const int32_t* counts,
                              int64_t tokens, int64_t* positions, int64_t* slots, int32_t* info, void* scratch,
                              int sms, int* status, cudaStream_t stream) {
  const PageState st = state_of(c, status);
  const Scratch ws = scratch_at(scratch, c.num_pages, n);
  const cudaError_t e =
      launch_pdl(cache_grow_kernel, dim3(idx_blocks(st)), dim3(kIdxThreads), 0, stream, st, ws, static_cast<int>(n),
                 seqs, counts, static_cast<int>(tokens), positions, slots, info, c.pool_count > 0 ? 1 : 0);
  if (e != cudaSuccess || c.pool_count == 0) return e;
  // the pages that became a sequence's own, which the device alone knows: hardly ever one
  CopyParams p = copy_params(c, status);
  p.src = ws.src;
  p.dst = ws.dst;
  p.count = &ws.head->moves;
  return launch_pdl(cache_copy_kernel, dim3(copy_grid(p, n, 1, sms)), dim3(kCopyThreads), 0, stream, p);
}

cudaError_t launch_cache_shrink(const gemm_cache_t& c, int64_t n, const int32_t* seqs, const int32_t* counts,
                                int* status, cudaStream_t stream) {
  return launch_pdl(cache_shrink_kernel, dim3(static_cast<unsigned>((n + 7) / 8)), dim3(256), 0, stream,
                    state_of(c, status), static_cast<int>(n), seqs, counts);
}

cudaError_t launch_cache_fork(const gemm_cache_t& c, int64_t n, const int32_t* parents, const int32_t* children,
                              int32_t* copied, int32_t* info, void* scratch, int sms, int* status,
                              cudaStream_t stream) {
  const PageState st = state_of(c, status);
  const Scratch ws = scratch_at(scratch, c.num_pages, n);
  cudaError_t e = launch_pdl(cache_fork_kernel, dim3(idx_blocks(st)), dim3(kIdxThreads), 0, stream, st, ws,
                             static_cast<int>(n), parents, children, copied, info);
  if (e != cudaSuccess) return e;
  CopyParams p = copy_params(c, status);
  p.src = ws.src;
  p.dst = ws.dst;
  p.count = &ws.head->moves;
  return launch_pdl(cache_fork_copy_kernel, dim3(copy_grid(p, n, n, sms)), dim3(kCopyThreads), 0, stream, st, ws,
                    static_cast<int>(n), parents, children, static_cast<const int32_t*>(copied), p);
}

cudaError_t launch_cache_compact(const gemm_cache_t& c, int32_t* info, void* scratch, int sms, int* status,
                                 cudaStream_t stream) {
  const PageState st = state_of(c, status);
  const Scratch ws = scratch_at(scratch, c.num_pages, 0);
  cudaError_t e =
      launch_pdl(cache_compact_kernel, dim3(idx_blocks(st)), dim3(kIdxThreads), 0, stream, st, ws, info);
  if (e != cudaSuccess) return e;
  CopyParams p = copy_params(c, status);
  p.src = ws.src;
  p.dst = ws.dst;
  p.count = &ws.head->moves;
  const int64_t entries = static_cast<int64_t>(c.sequences) * c.table_width;
  return launch_pdl(cache_compact_copy_kernel, dim3(copy_grid(p, c.num_pages / 2, entries / 32, sms)),
                    dim3(kCopyThreads), 0, stream, st, ws, p);
}

cudaError_t launch_cache_copy(const gemm_cache_t& c, int64_t n, const int32_t* src, const int32_t* dst, int sms,
                              int* status, cudaStream_t stream) {
  CopyParams p = copy_params(c, status);
  p.src = src;
  p.dst = dst;
  p.n = static_cast<int>(n);
  return launch_pdl(cache_copy_kernel, dim3(copy_grid(p, n, 1, sms)), dim3(kCopyThreads), 0, stream, p);
}

}  // namespace dgt
