// Attention of a chunk of new tokens over the paged cache: the plain form, one
// warp per (token, query head) that walks its visible keys with a running
// maximum and sum.
#include <math.h>

#include <algorithm>

#include "ks_paged_sched.cuh"
#include "ks_tc.cuh"

namespace ks {

namespace {

struct Simple {
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16* out;
  const int32_t *table, *cu, *kv_len;
  int32_t* status;
  int max_blocks, B, n_tokens, max_new, Hq, Hkv, page_size, n_pages, window, sinks;
  float scale;
};

template <int HD>
__global__ void __launch_bounds__(128) paged_attn_kernel(const Simple p) {
  constexpr int E = HD / 32;
  const int i = blockIdx.x, lane = threadIdx.x & 31;
  const int h = blockIdx.y * 4 + (threadIdx.x >> 5);
  if (h >= p.Hq) return;
  int lo = 0, hi = p.B;                      // the request whose rows hold token i
  if (i >= p.cu[p.B]) return;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.cu[mid] <= i) lo = mid;
    else hi = mid;
  }
  const int b = lo, g = h / (p.Hq / p.Hkv);
  const int n = p.cu[b + 1] - p.cu[b], t = i - p.cu[b];
  const int cap = p.max_blocks * p.page_size;
  const int kv = max(0, min(p.kv_len[b], cap));
  if ((n > p.max_new || kv != p.kv_len[b]) && lane == 0) raise_status(p.status, KS_ERR_INVALID_ARG);
  if (t >= p.max_new) return;
  const int pos = kv - min(n, p.max_new) + t;
  const __nv_bfloat16* q = p.q + ((long long)i * p.Hq + h) * HD + lane * E;
  float qf[E], acc[E] = {};
  for (int e = 0; e < E; ++e) qf[e] = __bfloat162float(q[e]) * p.scale;
  float m = -INFINITY, l = 0.f;
  const int from = p.window ? max(0, pos - p.window + 1) : 0;
  const int sinks = min(p.sinks, from);
  for (int s = 0; s < sinks + pos + 1 - from; ++s) {
    const int j = s < sinks ? s : from + s - sinks;
    const int page = p.table[(long long)b * p.max_blocks + j / p.page_size];
    const bool good = (unsigned)page < (unsigned)p.n_pages;
    if (!good && lane == 0) raise_status(p.status, KS_ERR_INVALID_ARG);
    const long long row =
        (((long long)(good ? page : 0) * p.page_size + j % p.page_size) * p.Hkv + g) * HD + lane * E;
    float d = 0.f, vf[E];
    for (int e = 0; e < E; ++e) {
      d += good ? qf[e] * __bfloat162float(p.k[row + e]) : 0.f;
      vf[e] = good ? __bfloat162float(p.v[row + e]) : 0.f;
    }
    for (int o = 16; o; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    const float mn = fmaxf(m, d), a = expf(m - mn), w = expf(d - mn);
    l = l * a + w;
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * a + w * vf[e];
    m = mn;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  __nv_bfloat16* out = p.out + ((long long)i * p.Hq + h) * HD + lane * E;
  for (int e = 0; e < E; ++e) out[e] = __float2bfloat16_rn(acc[e] * inv);
}

}  // namespace

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
  p.window = a.window < p.cap ? a.window : 0;   // a window that no position outruns hides nothing
  p.sinks = a.n_sinks;
  p.scale_log2 = (float)(1.4426950408889634 / sqrt((double)pool.head_dim));
  if ((long long)p.grp * p.max_new <= 128) {
    p.tile_tokens = p.max_new;
    const long long most = (long long)p.B * p.Hkv * std::max(1, ceil_div(p.cap, paged::kBlock));
    const int grid = (int)std::min<long long>(std::min(sm_count(), paged::kMaxCtas), most);
    return launch_paged_decode(a, p, grid, st);
  }
  const Simple s{(const __nv_bfloat16*)a.q, (const __nv_bfloat16*)pool.k_pages,
                 (const __nv_bfloat16*)pool.v_pages, (__nv_bfloat16*)a.out, a.block_table,
                 a.cu_new, a.kv_len, a.status, a.max_blocks, a.B, a.n_tokens, a.max_new, a.Hq,
                 pool.n_kv_heads, pool.page_size, pool.n_pages, a.window, a.n_sinks,
                 1.0f / sqrtf((float)pool.head_dim)};
  const dim3 grid(a.n_tokens, (a.Hq + 3) / 4);
  if (pool.head_dim == 128) paged_attn_kernel<128><<<grid, 128, 0, st>>>(s);
  else paged_attn_kernel<64><<<grid, 128, 0, st>>>(s);
  KS_LAUNCH_CHECK();
  return KS_OK;
}

}  // namespace ks
