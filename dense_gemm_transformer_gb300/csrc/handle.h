// handle.h -- what a gemm_handle_t points to (internal).
#pragma once

#include <cstddef>
#include <cstdint>
#include <mutex>

#include "gemm.h"
#include "kernels.h"
#include "skinny.cuh"

namespace dgt {
// Scratch of the paged attention and of the page management for the calls on
// one stream, or for those that graphs have captured on it, by size (block i
// holds 2^i MiB), zeroed when allocated.  It holds counters that a call leaves
// at zero, so two calls that run at the same time need one each.  A block that
// has become too small stays, so that a captured graph that uses it stays
// valid.
struct StreamScratch {
  // cudaStreamGetId, never that of another stream; in a capture, where that
  // call is an error, the handle
  unsigned long long stream;
  bool captured;
  void* attn[kScratchBlocks];
  void* cache[kScratchBlocks];
  StreamScratch* next;
};
}  // namespace dgt

struct gemm_handle_s {
  int device = 0;
  int sms = 0;
  int* d_status = nullptr;   // the status word, then (from word kSkCntOffset) the SIMT stream-K arrival counters
  void* ws = nullptr;
  size_t ws_bytes = 0;
  void* ws_t = nullptr;  // the transposed result of a weight-gradient-shaped TF32 product (run_checked)
  size_t ws_t_bytes = 0;
  int opt_family = GEMM_FAMILY_AUTO;
  int opt_split_k = 0;
  int opt_tile_n = 0;
  int opt_pretranspose = 0;
  int opt_pair = 0;
  int64_t opt_wait_us = 0;   // bounded-wait limit of the tcgen05 kernel (0: the default)
  int opt_fault_skip = 0;    // test hook (GEMM_OPT_FAULT_SKIP_STAGE)
  int opt_sk_fixup = 0;      // GEMM_OPT_SK_FIXUP
  int sk_active[5][dgt::kSkinnyMaxCluster + 1];  // small-M kernel per mode (TF32, BF16, FP8, MXFP8, NVFP4): resident clusters (-1: not queried)
  dgt::TmaCache* tma_cache = nullptr;             // TMA descriptors of earlier calls
  std::mutex paged_lock;  // of what the operators on a paged cache change here: they may run from several threads
  dgt::StreamScratch* paged_scratch = nullptr;
  gemm_plan_t plan{};
  dgt::LaunchShape null_shape;  // main kernel of the last successful gemm_run (for gemm_launch_null)
};
