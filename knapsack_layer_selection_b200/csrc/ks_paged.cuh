// The paged key/value cache (ks_page_plan, ks_rope_append_bf16,
// ks_paged_attention_bf16): what its sources share.
#pragma once

#include "ks_common.cuh"

namespace ks {

constexpr int kMaxRequests = 16384;

// Host checks of a pool that every call makes before anything is enqueued.
ks_status check_pool(const ks_page_pool* pool, const char* call);

// One step's attention (arguments checked; see ks_paged_attention_bf16).
struct PagedAttnArgs {
  const void* q;
  const ks_page_pool* pool;
  const int32_t *block_table, *cu_new, *kv_len;
  int max_blocks, B, n_tokens, max_new, Hq, window, n_sinks;
  void* out;
  void* workspace;
  int32_t* status;
};
ks_status launch_paged_attention(const PagedAttnArgs& a, cudaStream_t st);
size_t paged_attention_workspace_bytes();

}  // namespace ks
