// Attention of a step's new tokens over the paged cache: which kernel, and its
// parameters.
#include <math.h>

#include <algorithm>

#include "ks_paged_sched.cuh"
#include "ks_tc.cuh"

namespace ks {

size_t paged_attention_workspace_bytes() { return paged::kWorkspaceBytes; }

ks_status launch_paged_attention(const PagedAttnArgs& a, cudaStream_t st) {
  const ks_page_pool& pool = *a.pool;
  paged::Params p{};
  p.table = a.block_table;
  p.cu = a.cu_new;
  p.kv_len = a.kv_len;
  p.out = (__nv_bfloat16*)a.out;
  p.ws = (unsigned char*)a.workspace;
  p.status = a.status;
  p.B = a.B;
  p.n_tokens = a.n_tokens;
  p.max_new = std::min(a.max_new, a.n_tokens);
  p.max_blocks = a.max_blocks;
  p.page_size = pool.page_size;
  p.cap = a.max_blocks * pool.page_size;
  p.Hq = a.Hq;
  p.Hkv = pool.n_kv_heads;
  p.grp = a.Hq / pool.n_kv_heads;
  p.n_pages = pool.n_pages;
  p.n_slots = pool.n_pages * pool.page_size;
  p.box = std::min(paged::kBlock, pool.page_size & -pool.page_size);
  while (p.box << p.log2_boxes < paged::kBlock) ++p.log2_boxes;
  p.window = a.window;
  p.sinks = a.n_sinks;
  p.scale_log2 = (float)(1.4426950408889634 / sqrt((double)pool.head_dim));
  // Up to 64 rows the keys' traffic bounds a step and the few-row kernel is the faster; above, its
  // scores no longer fit the registers.  64 requests over up to 8,192 keys, 8 kv heads, few-row and
  // chunk kernel in us: heads of 128, 4 rows 170 and 184, 32 rows 178 and 196, 64 rows 189 and 204;
  // heads of 64, 4 rows 139 and 161, 32 rows 149 and 167, 64 rows 173 and 175.
  const bool few = (long long)p.grp * p.max_new <= 64;
  p.tile_tokens = few ? p.max_new : paged::kTileRows / p.grp;
  // a CTA per SM, or fewer where the step cannot have as many key blocks
  const long long tiles = (long long)p.B * ceil_div(p.max_new, p.tile_tokens);
  const long long most = tiles * p.Hkv * std::max(1, ceil_div(p.cap, paged::kBlock));
  const int grid = (int)std::min<long long>(std::min(sm_count(), paged::kMaxCtas), most);
  return few ? launch_paged_decode(a, p, grid, st) : launch_paged_chunk(a, p, grid, st);
}

}  // namespace ks
