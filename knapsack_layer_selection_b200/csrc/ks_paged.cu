// The paged cache's C ABI, and the two memory-bound operators before its
// attention: the step's layout and the rotary append.
#include <math.h>

#include <algorithm>
#include <cmath>

#include "ks_paged.cuh"
#include "ks_prof.cuh"
#include "ks_tc.cuh"

namespace ks {

namespace {

constexpr int kPlanThreads = 512;

struct PlanArgs {
  const int32_t *ctx_len, *new_len, *free_pages;
  int32_t *block_table, *cu_new, *kv_len, *positions, *slots, *n_taken, *status;
  int B, n_free, n_pages, page_size, max_blocks, max_tokens;
  int32_t* n_held;                           // NULL: what the cached tokens fill
  int32_t* free_start;                       // NULL: 0
  // pages in front of request r's row that are its own; the cached tokens fill the first of them
  __device__ __forceinline__ int filled(long long ctx) const {
    return (int)((ctx + page_size - 1) / page_size);
  }
  __device__ __forceinline__ int held(int r) const { return n_held ? n_held[r] : filled(ctx_len[r]); }
};

// Last index r of off[0 .. n] with off[r] <= i (off ascending, off[n] > i).
__device__ __forceinline__ int find_segment(const int32_t* off, int n, int i) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

// One launch: every CTA scans the requests' token and page counts into its own
// shared memory (two prefix sums of at most 16384 entries; a second launch or a
// grid-wide wait would cost more than the repeated reads, which come from L2),
// then the CTAs share the packed tokens and the taken pages between them, each
// finding its request by bisection.  A token reads a table entry only of a page
// that its request held before, and only entries of taken pages are written, so
// no CTA reads what another writes.
__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const PlanArgs p) {
  extern __shared__ int32_t plan_smem[];
  int32_t* tok = plan_smem;                  // [B+1] new tokens, then their prefix sums
  int32_t* pag = plan_smem + p.B + 1;        // [B+1] pages to take, then their prefix sums
  __shared__ long long warp_tok[kPlanThreads / 32], warp_pag[kPlanThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long row_cap = (long long)p.max_blocks * p.page_size;

  const int start = p.free_start ? *p.free_start : 0;
  bool bad = start < 0 || start > p.n_free;
  for (int b = tid; b < p.B; b += kPlanThreads) {
    const long long c = p.ctx_len[b], n = p.new_len[b];
    bool wrong = c < 0 || n < 0 || c + n > row_cap;
    int held = 0;
    if (!wrong) {
      held = p.filled(c);
      if (p.n_held) {
        const int h = p.n_held[b];
        wrong = h < held || h > p.max_blocks;
        held = h;
      }
    }
    bad |= wrong;
    tok[b] = wrong ? 0 : (int32_t)n;
    pag[b] = wrong ? 0 : max(0, p.filled(c + n) - held);
  }
  bad = __syncthreads_or(bad);

  // each thread's contiguous share, then a scan of the shares
  const int per = (p.B + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  long long st = 0, sp = 0;
  for (int b = b0; b < b1; ++b) {
    st += tok[b];
    sp += pag[b];
  }
  long long it = st, ip = sp;                // inclusive within the warp
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long ut = __shfl_up_sync(0xffffffffu, it, d), up = __shfl_up_sync(0xffffffffu, ip, d);
    if (lane >= d) {
      it += ut;
      ip += up;
    }
  }
  if (lane == 31) {
    warp_tok[warp] = it;
    warp_pag[warp] = ip;
  }
  __syncthreads();
  long long total_tok = 0, total_pag = 0, base_tok = 0, base_pag = 0;
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w == warp) {
      base_tok = total_tok;
      base_pag = total_pag;
    }
    total_tok += warp_tok[w];
    total_pag += warp_pag[w];
  }
  const int32_t code = bad || total_tok > p.max_tokens ? KS_ERR_INVALID_ARG
                       : total_pag > p.n_free - start  ? KS_ERR_WORKSPACE
                                                       : KS_OK;
  const bool ok = code == KS_OK;
  if (!ok) total_tok = total_pag = 0;        // an empty step
  if (ok) {                                  // both totals fit 32 bits from here on
    int rt = (int)(base_tok + it - st), rp = (int)(base_pag + ip - sp);
    for (int b = b0; b < b1; ++b) {
      const int t = tok[b], g = pag[b];
      tok[b] = rt;
      pag[b] = rp;
      rt += t;
      rp += g;
    }
  }
  if (tid == 0) {
    tok[p.B] = (int32_t)total_tok;
    pag[p.B] = (int32_t)total_pag;
  }
  __syncthreads();

  const int first = blockIdx.x * kPlanThreads + tid, step = gridDim.x * kPlanThreads;
  if (first == 0) {
    *p.n_taken = (int32_t)total_pag;
    if (!ok) raise_status(p.status, code);
  }
  for (int b = first; b <= p.B; b += step) {
    p.cu_new[b] = ok ? tok[b] : 0;
    if (b < p.B) p.kv_len[b] = ok ? p.ctx_len[b] + p.new_len[b] : 0;
  }
  for (long long i = first; i < total_pag; i += step) {
    const int r = find_segment(pag, p.B, (int)i);
    const int held = p.held(r);
    int page = p.free_pages[start + i];
    if ((unsigned)page >= (unsigned)p.n_pages) {
      page = -1;
      raise_status(p.status, KS_ERR_INVALID_ARG);
    }
    p.block_table[(long long)r * p.max_blocks + held + ((int)i - pag[r])] = page;
  }
  for (long long i = first; i < p.max_tokens; i += step) {
    int pos = -1, slot = -1;
    if (i < total_tok) {
      const int r = find_segment(tok, p.B, (int)i);
      const int ctx = p.ctx_len[r];
      pos = ctx + ((int)i - tok[r]);
      const int held = p.held(r), blk = pos / p.page_size;
      const int page = blk < held ? p.block_table[(long long)r * p.max_blocks + blk]
                                  : p.free_pages[start + pag[r] + (blk - held)];
      if ((unsigned)page < (unsigned)p.n_pages) slot = page * p.page_size + (pos - blk * p.page_size);
      else raise_status(p.status, KS_ERR_INVALID_ARG);
    }
    p.positions[i] = pos;
    p.slots[i] = slot;
  }
}

// The counts that the plan carries on, in a launch of their own: every CTA of the plan reads them all,
// so none of them may be written there.  A refused step has kv_len = 0 and n_taken = 0 and changes
// nothing.
__global__ void __launch_bounds__(kPlanThreads) plan_carry_kernel(const PlanArgs p) {
  const int b = blockIdx.x * kPlanThreads + threadIdx.x;
  if (b == 0 && p.free_start) *p.free_start += *p.n_taken;
  if (b >= p.B || !p.n_held) return;
  const int filled = p.filled(p.kv_len[b]);
  if (filled > 0 && filled > p.n_held[b]) p.n_held[b] = filled;
}

constexpr int kAppendThreads = 256;            // at most

struct AppendArgs {
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16 *q_out, *k_pages, *v_pages;
  const int32_t *positions, *slots;
  int32_t* status;
  long long q_stride, k_stride, v_stride;
  int n_tokens, Hq, Hkv, n_slots;
  double turns[64];                          // theta_j / (2 pi): turns of pair j per position
};

// One CTA per token: its head_dim/2 rotations are computed once (angle in fp64
// turns, reduced to (-1/2, 1/2] exactly, so the fp32 sine and cosine see a small
// argument at any position) and serve all its heads.
template <int HD>
__global__ void __launch_bounds__(kAppendThreads) rope_append_kernel(const AppendArgs p) {
  constexpr int HALF = HD / 2, PC = HALF / 8, VC = HD / 8;   // 8-element chunks of a half, a head
  __shared__ float2 cs[HALF];
  const int i = blockIdx.x;
  const int pos = p.positions[i];
  if (pos < 0) return;                       // padding row
  const int slot = p.slots[i];
  const bool cached = slot >= 0 && slot < p.n_slots;
  if (slot >= p.n_slots && threadIdx.x == 0) raise_status(p.status, KS_ERR_INVALID_ARG);
  if (threadIdx.x < HALF) {
    const double t = (double)pos * p.turns[threadIdx.x];
    float s, c;
    sincospif((float)(2.0 * (t - rint(t))), &s, &c);
    cs[threadIdx.x] = make_float2(c, s);
  }
  __syncthreads();
  const int nq = p.q ? p.Hq * PC : 0, nk = cached ? p.Hkv * PC : 0, nv = cached ? p.Hkv * VC : 0;
  for (int u = threadIdx.x; u < nq + nk + nv; u += blockDim.x) {
    if (u < nq + nk) {
      const bool is_q = u < nq;
      const int e = is_q ? u : u - nq;
      const int h = e / PC, c = (e % PC) * 8;
      const __nv_bfloat16* src = (is_q ? p.q + i * p.q_stride : p.k + i * p.k_stride) + h * HD + c;
      __nv_bfloat16* dst = is_q ? p.q_out + ((long long)i * p.Hq + h) * HD + c
                                : p.k_pages + ((long long)slot * p.Hkv + h) * HD + c;
      uint4 a4 = *reinterpret_cast<const uint4*>(src);
      uint4 b4 = *reinterpret_cast<const uint4*>(src + HALF);
      __nv_bfloat162* a = reinterpret_cast<__nv_bfloat162*>(&a4);
      __nv_bfloat162* b = reinterpret_cast<__nv_bfloat162*>(&b4);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float2 fa = __bfloat1622float2(a[x]), fb = __bfloat1622float2(b[x]);
        const float2 r0 = cs[c + 2 * x], r1 = cs[c + 2 * x + 1];
        a[x] = __floats2bfloat162_rn(fa.x * r0.x - fb.x * r0.y, fa.y * r1.x - fb.y * r1.y);
        b[x] = __floats2bfloat162_rn(fb.x * r0.x + fa.x * r0.y, fb.y * r1.x + fa.y * r1.y);
      }
      *reinterpret_cast<uint4*>(dst) = a4;
      *reinterpret_cast<uint4*>(dst + HALF) = b4;
    } else {
      const int e = u - nq - nk;
      const long long off = (long long)(e / VC) * HD + (e % VC) * 8;
      *reinterpret_cast<uint4*>(p.v_pages + (long long)slot * p.Hkv * HD + off) =
          *reinterpret_cast<const uint4*>(p.v + i * p.v_stride + off);
    }
  }
}

template <int HD>
ks_status launch_append(const AppendArgs& a, cudaStream_t st) {
  // Tokens enough for several CTAs per SM: three warps each, so that more tokens' loads are in flight
  // past the angles' barrier (8,900 tokens of 32/8 heads of 128: 38.2 us, 5.7 TB/s, against 41.7
  // with eight warps; heads of 64: 9.4 against 13.5).  Few tokens: eight warps, a token's latency
  // counts (32 tokens: 2.8 us against 3.6).
  const int threads = a.n_tokens >= 4 * sm_count() ? 96 : kAppendThreads;
  rope_append_kernel<HD><<<a.n_tokens, threads, 0, st>>>(a);
  KS_LAUNCH_CHECK();
  return KS_OK;
}

}  // namespace

ks_status check_pool(const ks_page_pool* pool, const char* call) {
  const std::string c(call);
  if (!pool || !pool->k_pages || !pool->v_pages) return fail(KS_ERR_INVALID_ARG, c + ": pool is NULL");
  KS_TRY(check_aligned16({pool->k_pages, pool->v_pages}, call));
  if (pool->n_pages < 1 || pool->page_size < 1 || pool->n_kv_heads < 1)
    return fail(KS_ERR_INVALID_ARG, c + ": bad pool size");
  if (pool->head_dim != 64 && pool->head_dim != 128)
    return fail(KS_ERR_UNSUPPORTED, c + ": head_dim must be 64 or 128");
  if (pool->page_size % 8) return fail(KS_ERR_UNSUPPORTED, c + ": page_size must be a multiple of 8");
  if ((long long)pool->n_pages * pool->page_size > 2147483647ll - 255)
    return fail(KS_ERR_UNSUPPORTED, c + ": n_pages * page_size must be at most 2^31 - 256");
  if ((long long)pool->n_kv_heads * pool->head_dim > (1 << 20))
    return fail(KS_ERR_UNSUPPORTED, c + ": n_kv_heads * head_dim must be at most 2^20");
  return KS_OK;
}

}  // namespace ks

using namespace ks;

extern "C" {

ks_status ks_page_plan(const int32_t* ctx_len, const int32_t* new_len, int32_t B,
                       const int32_t* free_pages, int32_t n_free, int32_t n_pages,
                       int32_t page_size, int32_t* block_table, int32_t max_blocks,
                       int32_t max_tokens, int32_t* cu_new, int32_t* kv_len, int32_t* positions,
                       int32_t* slots, int32_t* n_taken, int32_t* status, ks_stream_t stream) {
  return ks_page_plan_carried(ctx_len, new_len, B, free_pages, n_free, n_pages, page_size, block_table,
                              max_blocks, max_tokens, cu_new, kv_len, positions, slots, n_taken, nullptr,
                              nullptr, status, stream);
}

ks_status ks_page_plan_carried(const int32_t* ctx_len, const int32_t* new_len, int32_t B,
                               const int32_t* free_pages, int32_t n_free, int32_t n_pages,
                               int32_t page_size, int32_t* block_table, int32_t max_blocks,
                               int32_t max_tokens, int32_t* cu_new, int32_t* kv_len,
                               int32_t* positions, int32_t* slots, int32_t* n_taken, int32_t* n_held,
                               int32_t* free_start, int32_t* status, ks_stream_t stream) {
  if (B < 0 || n_free < 0 || n_pages < 1 || page_size < 1 || max_blocks < 0 || max_tokens < 0)
    return fail(KS_ERR_INVALID_ARG, "page plan: bad size");
  if (B > kMaxRequests) return fail(KS_ERR_UNSUPPORTED, "page plan: at most 16384 requests");
  if (page_size % 8) return fail(KS_ERR_UNSUPPORTED, "page plan: page_size must be a multiple of 8");
  if ((long long)n_pages * page_size > 2147483647ll - 255)
    return fail(KS_ERR_UNSUPPORTED, "page plan: n_pages * page_size must be at most 2^31 - 256");
  if ((long long)max_blocks * page_size > 2147483647ll - 255)
    return fail(KS_ERR_UNSUPPORTED, "page plan: max_blocks * page_size must be at most 2^31 - 256");
  if (!cu_new || !n_taken || (B && (!ctx_len || !new_len || !kv_len)) ||
      (B && max_blocks && !block_table) || (max_tokens && (!positions || !slots)) ||
      (n_free && !free_pages))
    return fail(KS_ERR_INVALID_ARG, "page plan: NULL pointer");
  const cudaStream_t st = (cudaStream_t)stream;
  const size_t smem = 2 * sizeof(int32_t) * ((size_t)B + 1);
  static std::atomic<unsigned long long> attr{0};
  KS_TRY(once_per_device(attr, [&]() -> ks_status {
    KS_CUDA_TRY(cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)(2 * sizeof(int32_t) * (kMaxRequests + 1))));
    return KS_OK;
  }));
  const PlanArgs a{ctx_len, new_len, free_pages, block_table, cu_new,  kv_len,    positions,  slots,
                   n_taken, status,  B,          n_free,      n_pages, page_size, max_blocks, max_tokens,
                   n_held,  free_start};
  const int rows = max_tokens > B + 1 ? max_tokens : B + 1;
  const int grid = std::min(ceil_div(rows, kPlanThreads), sm_count());
  const bool carried = (n_held && B) || free_start;
  ProfScope prof(KK_PAGE_PLAN, st, 0.0, 16.0 * B + 8.0 * max_tokens, carried ? 2 : 1);
  page_plan_kernel<<<grid, kPlanThreads, smem, st>>>(a);
  KS_LAUNCH_CHECK();
  if (carried) {
    plan_carry_kernel<<<std::max(1, ceil_div(B, kPlanThreads)), kPlanThreads, 0, st>>>(a);
    KS_LAUNCH_CHECK();
  }
  return KS_OK;
}

ks_status ks_rope_append_bf16(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                              const void* v, int64_t v_stride, int32_t n_tokens, int32_t n_q_heads,
                              const ks_page_pool* pool, const int32_t* positions,
                              const int32_t* slots, double rope_base, void* q_out, int32_t* status,
                              ks_stream_t stream) {
  KS_TRY(check_pool(pool, "rope append"));
  const int hd = pool->head_dim, Hkv = pool->n_kv_heads;
  if (n_tokens < 0 || n_q_heads < 1) return fail(KS_ERR_INVALID_ARG, "rope append: bad size");
  if ((long long)n_q_heads * hd > (1 << 20))
    return fail(KS_ERR_UNSUPPORTED, "rope append: n_q_heads * head_dim must be at most 2^20");
  if ((q == nullptr) != (q_out == nullptr))
    return fail(KS_ERR_INVALID_ARG, "rope append: q and q_out go together");
  if (!(rope_base > 0.0) || !std::isfinite(rope_base))
    return fail(KS_ERR_INVALID_ARG, "rope append: rope_base must be > 0");
  if (n_tokens == 0) return KS_OK;
  if (!k || !v || !positions || !slots) return fail(KS_ERR_INVALID_ARG, "rope append: NULL pointer");
  KS_TRY(check_aligned16({q, k, v, q_out}, "rope append"));
  const long long qs = q ? q_stride : (long long)n_q_heads * hd;
  if (qs % 8 || k_stride % 8 || v_stride % 8 || qs < (long long)n_q_heads * hd ||
      k_stride < (long long)Hkv * hd || v_stride < (long long)Hkv * hd)
    return fail(KS_ERR_INVALID_ARG, "rope append: strides must be multiples of 8 and hold a row");
  const cudaStream_t st = (cudaStream_t)stream;
  AppendArgs a;
  a.q = (const __nv_bfloat16*)q;
  a.k = (const __nv_bfloat16*)k;
  a.v = (const __nv_bfloat16*)v;
  a.q_out = (__nv_bfloat16*)q_out;
  a.k_pages = (__nv_bfloat16*)pool->k_pages;
  a.v_pages = (__nv_bfloat16*)pool->v_pages;
  a.positions = positions;
  a.slots = slots;
  a.status = status;
  a.q_stride = qs;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.n_tokens = n_tokens;
  a.Hq = n_q_heads;
  a.Hkv = Hkv;
  a.n_slots = pool->n_pages * pool->page_size;
  // base^(-2 (8 a + b) / hd) as a product: 16 calls of pow instead of 64, half an ulp more
  double lo[8];
  for (int b = 0; b < 8; ++b) lo[b] = pow(rope_base, -2.0 * b / hd) * 0.15915494309189535;   // 1 / (2 pi)
  for (int j = 0; j < hd / 2; j += 8) {
    const double hi = j ? pow(rope_base, -2.0 * j / hd) : 1.0;
    for (int b = 0; b < 8; ++b) a.turns[j + b] = hi * lo[b];
  }
  const double heads = (q ? n_q_heads : 0) + 2.0 * Hkv;
  ProfScope prof(KK_ROPE_APPEND, st, 3.0 * n_tokens * (heads - Hkv) * hd, 4.0 * n_tokens * heads * hd);
  return hd == 128 ? launch_append<128>(a, st) : launch_append<64>(a, st);
}

ks_status ks_paged_attention_workspace_size(size_t* bytes) {
  if (!bytes) return fail(KS_ERR_INVALID_ARG, "paged attention: bytes is NULL");
  *bytes = paged_attention_workspace_bytes();
  return KS_OK;
}

ks_status ks_paged_attention_bf16(const void* q, const ks_page_pool* pool,
                                  const int32_t* block_table, int32_t max_blocks,
                                  const int32_t* cu_new, const int32_t* kv_len, int32_t B,
                                  int32_t n_tokens, int32_t max_new, int32_t n_q_heads,
                                  int32_t window, int32_t n_sinks, void* out, void* workspace,
                                  size_t workspace_bytes, int32_t* status, ks_stream_t stream) {
  KS_TRY(check_pool(pool, "paged attention"));
  if (B < 0 || n_tokens < 0 || max_new < 0 || max_blocks < 0 || n_q_heads < 1 || window < 0 ||
      n_sinks < 0)
    return fail(KS_ERR_INVALID_ARG, "paged attention: bad size");
  if (B > kMaxRequests) return fail(KS_ERR_UNSUPPORTED, "paged attention: at most 16384 requests");
  if (n_q_heads % pool->n_kv_heads)
    return fail(KS_ERR_INVALID_ARG, "paged attention: n_q_heads must be a multiple of n_kv_heads");
  if (n_q_heads / pool->n_kv_heads > 128)
    return fail(KS_ERR_UNSUPPORTED, "paged attention: at most 128 query heads per kv head");
  if ((long long)n_q_heads * pool->head_dim > (1 << 20))
    return fail(KS_ERR_UNSUPPORTED, "paged attention: n_q_heads * head_dim must be at most 2^20");
  if ((long long)max_blocks * pool->page_size > 2147483647ll - 255)
    return fail(KS_ERR_UNSUPPORTED,
                "paged attention: max_blocks * page_size must be at most 2^31 - 256");
  if (B == 0 || n_tokens == 0 || max_new == 0) return KS_OK;
  if (!q || !out || !cu_new || !kv_len || !workspace || (max_blocks && !block_table))
    return fail(KS_ERR_INVALID_ARG, "paged attention: NULL pointer");
  KS_TRY(check_aligned16({q, out}, "paged attention"));
  if (reinterpret_cast<uintptr_t>(workspace) & 255)
    return fail(KS_ERR_INVALID_ARG, "paged attention: the workspace must be 256-byte aligned");
  if (workspace_bytes < paged_attention_workspace_bytes())
    return fail(KS_ERR_WORKSPACE, "paged attention: workspace smaller than "
                                  "ks_paged_attention_workspace_size()");
  const PagedAttnArgs a{q,     pool,     block_table, cu_new,    kv_len, max_blocks, B,
                        n_tokens, max_new, n_q_heads, window, n_sinks,    out,
                        workspace, status};
  // the lengths stay on the device: the launch accounting counts the call, not its work
  ProfScope prof(KK_PAGED_ATTN, (cudaStream_t)stream, 0.0, 0.0);
  return launch_paged_attention(a, (cudaStream_t)stream);
}

}  // extern "C"
