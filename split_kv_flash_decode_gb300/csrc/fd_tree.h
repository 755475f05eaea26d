// Internal definitions of a step of speculative decoding: the handle and the attention's parameters.
#pragma once

#include "fd_common.h"
#include "fd_host.h"

struct fd_tree_s {
  int B, Hq, Hkv, d, dtype, page_size, max_pages, max_drafts, num_sms;
  int64_t T, n_tokens, n_blocks;
  uint64_t kv_bytes;
  int32_t cu_q[FD_MAX_BATCH + 1];  // prefix sums of drafts
  int32_t len[FD_MAX_BATCH];       // L_b
  int32_t base[FD_MAX_BATCH];      // contiguous caches: cache row (in tokens) of the sequence's row 0
  int ctas;
  size_t ws_bytes;
};

namespace fd {

struct TreeParams {
  const void *q, *k, *v;
  const uint64_t* mask;
  void* out;
  float* lse;
  uint32_t* status;
  const int32_t* block_table;
  int32_t bt_stride, page_shift, num_pages;
  int32_t B, Hq, Hkv;
  float scale_log2;  // log2(e) / sqrt(d)
  int32_t cu_q[FD_MAX_BATCH + 1];
  int32_t len[FD_MAX_BATCH];
  int32_t base[FD_MAX_BATCH];
};

cudaError_t launch_tree(const TreeParams& p, int dtype, int d, int T, cudaStream_t s);

}  // namespace fd
