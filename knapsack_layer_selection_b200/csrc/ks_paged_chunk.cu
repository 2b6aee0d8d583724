// Attention over the paged cache for prompt chunks: query tiles of up to 128
// rows (whole tokens x the query heads of one kv head), sm_100a tcgen05 + TMEM +
// TMA.
//
// Many rows meet every key, so the tensor core bounds it (and, at the same
// height, the exponentials): S = Q K^T, O = P V with query rows on the tensor
// core's 128 rows.  The pipeline inside a tile is that of the contiguous
// cache's attention (two softmax groups of one thread per row that take the even
// and the odd key blocks, P in TMEM, row sums from a panel of ones after V,
// references kept until the maximum grows by 2^8); what differs is the work: a
// persistent CTA per SM walks an equal share of the step's key blocks
// (ks_paged_sched.cuh), so that a chunk whose tiles see different numbers of
// keys, and one with fewer tiles than SMs, still fill the GPU.  384 threads:
//   warp 0    -- walks the share, publishes its pieces and loads their K blocks
//                (TMA, 3-slot ring);
//   warp 1    -- S_i = Q K_i^T; loads the next piece's Q tile itself once its
//                last S is done, so that no load of K or V waits behind it;
//   warp 2    -- TMEM owner; [O | l] += P_i [V_i | 1], after zeroing what nobody
//                sees in a ragged block of V;
//   warp 3    -- V blocks into a 2-slot ring; in both rings each lane loads the box
//                of one page of one 64-column panel (issuing a box costs ~57 cycles, so
//                16-key pages would hold one warp for longer than a block takes);
//   warps 4-7, 8-11 -- the softmax groups; blocks are numbered over the whole
//                share, so a piece's first block runs beside its predecessor's last.
// Registers: a softmax thread holds a block's 128 scores, so the kernel launches
// with 168 registers a thread and moves them with setmaxnreg from the first
// warpgroup (REGS_LOW) to the softmax warpgroups (REGS_HIGH), whose shares add up to the
// launch's allocation; the host refuses a build of another register count.
// Rounding: P is bf16 for the tensor core, and the row sums are of the rounded values
// (in fp32), so that what rounding adds to a weight it adds to the sum too; S, O and
// references are fp32 (2.3e-3 from fp64 in all, 1.7e-3 of it the output's own rounding).
// Measured: two chunks of up to 2,047 tokens over 8,192 cached keys (32/8 heads of
// 128, 550 GFLOP) 546 us among other work (1.01 PFLOP/s), 465 back to back (1.18); 8
// requests of 72 rows over up to 16,384 keys 102 and 96 us, where the few-row kernel's
// 128-column form took 354.
#include <algorithm>

#include "ks_paged_sched.cuh"
#include "ks_tc.cuh"

namespace ks {

using namespace paged;

namespace {

constexpr int kThreads = 384;
constexpr float kStale = 8.0f;                 // a new reference once the maximum grows by > 2^8

struct Tail {
  SchedSmem sched;
  uint64_t q_full, q_empty;                                // one phase per piece
  uint64_t k_full[3], k_empty[3], v_full[2], v_empty[2];
  uint64_t s_full[2], s_free[2];                           // [softmax group = S buffer]
  uint64_t p_full;                                         // one phase per block
  uint64_t pv_done[2];                                     // [block parity]
  uint64_t m_ready[2];                                     // [group of the publishing block]
  uint64_t o_free;                                         // one phase per piece
  uint64_t gsync[2];                                       // meetings of a group's warps
  uint64_t drain[2];                                       // [S issuer, PV issuer]
  uint32_t tmem_base;
  int abort;
  int last[2];
  float m_pub[2][128];                                     // references, by group
};

template <int HD>
struct Cfg {
  static constexpr int BM = 128, BN = kBlock, KST = 3, VST = 2;
  static constexpr int PANELS = HD / 64;
  static constexpr int Q_PANEL = BM * 128, Q_TILE = PANELS * Q_PANEL;
  static constexpr int KV_PANEL = BN * 128, KV_BLOCK = PANELS * KV_PANEL;
  static constexpr int V_SLOT = (PANELS + 1) * KV_PANEL;   // the panel of ones after V
  static constexpr int N_O = HD + 16;
  static constexpr int OFF_K = Q_TILE;
  static constexpr int OFF_V = OFF_K + KST * KV_BLOCK;
  static constexpr int OFF_TAIL = OFF_V + VST * V_SLOT;
  static constexpr int USED = OFF_TAIL + (int)((sizeof(Tail) + 255) / 256 * 256);
  static constexpr int SMEM = USED > 118784 ? USED : 118784;   // one CTA holds an SM's TMEM
  static constexpr int REGS = 168, REGS_LOW = 72, REGS_HIGH = 216;
  static_assert(128 * REGS_LOW + 256 * REGS_HIGH == kThreads * REGS, "register split");
  static constexpr int TMEM_S = 0, TMEM_P = 2 * BN, TMEM_O = 2 * BN + BN / 2;
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t IDESC_S = idesc_bf16_f32(BM, BN);
  static constexpr uint32_t IDESC_O = idesc_bf16_f32(BM, N_O) | (1u << 16);   // B (V) MN-major
  static_assert(TMEM_O + N_O <= (int)TMEM_COLS, "TMEM budget");
  static_assert(USED <= 232448, "shared memory budget");
};

template <int HD>
__global__ void __launch_bounds__(kThreads, 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap tmQ,
                       const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const __grid_constant__ Params p) {
  using C = Cfg<HD>;
  extern __shared__ __align__(1024) unsigned char smem[];
  // the 128-byte-swizzled tiles need a 1024-aligned base; refuse rather than realign
  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) raise_status(p.status, KS_ERR_INTERNAL);
    return;
  }
  Tail* tail = reinterpret_cast<Tail*>(smem + C::OFF_TAIL);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &tail->abort;
  const uint32_t sbase = smem_u32(smem);

  if (threadIdx.x == kThreads - 32) {          // the first warps have requests to read
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
    for (int s = 0; s < kSegRing; ++s) {
      mbar_init(smem_u32(&tail->sched.full[s]), 1);
      mbar_init(smem_u32(&tail->sched.empty[s]), 11);    // V, S, P.V and 8 softmax warps
    }
    mbar_init(smem_u32(&tail->q_full), 1);
    mbar_init(smem_u32(&tail->q_empty), 1);
    for (int s = 0; s < C::KST; ++s) {
      mbar_init(smem_u32(&tail->k_full[s]), 1);
      mbar_init(smem_u32(&tail->k_empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&tail->v_full[b]), 1);
      mbar_init(smem_u32(&tail->v_empty[b]), 1);
      mbar_init(smem_u32(&tail->s_full[b]), 1);
      mbar_init(smem_u32(&tail->s_free[b]), 4);          // one arrival per softmax warp
      mbar_init(smem_u32(&tail->m_ready[b]), 4);
      mbar_init(smem_u32(&tail->pv_done[b]), 1);
      mbar_init(smem_u32(&tail->gsync[b]), 4);
      mbar_init(smem_u32(&tail->drain[b]), 1);
    }
    mbar_init(smem_u32(&tail->p_full), 4);
    mbar_init(smem_u32(&tail->o_free), 4);
    tail->abort = 0;
    fence_barrier_init();
  }
  if (warp == 2) {
    tmem_alloc(smem_u32(&tail->tmem_base), C::TMEM_COLS);
    tmem_relinquish();
  }
  // the ones panel of each V slot (every element 1.0, so its swizzle is moot);
  // the TMA only ever writes the V panels before it
  for (int s = 0; s < C::VST; ++s) {
    uint4* ones = reinterpret_cast<uint4*>(smem + C::OFF_V + s * C::V_SLOT + C::PANELS * C::KV_PANEL);
    for (int e = threadIdx.x; e < C::KV_PANEL / 16; e += kThreads)
      ones[e] = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // visible to the tensor core
  locate<kThreads / 32>(p, tail->sched);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tail->tmem_base;

  if (warp < 4) {
    regs_dec<C::REGS_LOW>();
    if (warp == 0 || warp == 3) {
      // ---------------------------------------------------------- TMA: the walk and K; V
      const bool is_k = warp == 0;
      const Ring ring{is_k ? &tmK : &tmV, is_k ? tail->k_full : tail->v_full,
                      is_k ? tail->k_empty : tail->v_empty, sbase + (is_k ? C::OFF_K : C::OFF_V),
                      is_k ? C::KST : C::VST, is_k ? C::KV_BLOCK : C::V_SLOT};
      load_share<HD>(p, tail->sched, ring, is_k, abort, [](const Seg&) { return true; });
    } else if (warp == 1) {
      // ---------------------------------------------------------- Q loads and S
      SegReader rd;
      Seg s;
      uint32_t n_seg = 0;
      int i = 0, ks = 0;
      uint32_t kph = 0;
      bool ok = true;
      const int box_rows = p.grp * p.tile_tokens;
      const uint64_t dq0 = desc_kmajor_sw128(sbase);
      const uint64_t dk0 = desc_kmajor_sw128(sbase + C::OFF_K);
      while (ok) {
        if (!rd.take(p, tail->sched, abort, s) || s.nb == 0) break;
        if (n_seg > 0 && !KS_PAGED_WAIT(tail->q_empty, (n_seg - 1) & 1)) break;
        if (lane == 0) {
          const uint32_t qf = smem_u32(&tail->q_full);
          mbar_arrive_expect_tx(qf, C::PANELS * box_rows * 128);
          for (int pn = 0; pn < C::PANELS; ++pn)
            tma_load_3d(sbase + pn * C::Q_PANEL, &tmQ, pn * 64, s.g * p.grp, s.row0, qf);
        }
        ++n_seg;
        ok = KS_PAGED_WAIT(tail->q_full, (n_seg - 1) & 1);
        for (int e = 0; ok && e < s.nb; ++e, ++i) {
          // S_i into S buffer i % 2, free once the softmax has copied S_{i-2}
          const int b = i & 1;
          if (i >= 2 && !(ok = KS_PAGED_WAIT(tail->s_free[b], ((i - 2) >> 1) & 1))) break;
          if (!(ok = KS_PAGED_WAIT(tail->k_full[ks], kph))) break;
          tc_fence_after();
          if (lane == 0) {
            const uint64_t dk = dk0 + (uint64_t)((ks * C::KV_BLOCK) >> 4);
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk)
              mma_bf16(tmem + C::TMEM_S + b * C::BN,
                       dq0 + (uint64_t)((kk / 4) * (C::Q_PANEL >> 4) + 2 * (kk % 4)),
                       dk + (uint64_t)((kk / 4) * (C::KV_PANEL >> 4) + 2 * (kk % 4)), C::IDESC_S,
                       kk > 0);
            // the softmax group that sees S_i complete frees K slot ks
            mma_commit(smem_u32(&tail->s_full[b]));
            if (e == s.nb - 1) mma_commit(smem_u32(&tail->q_empty));
          }
          __syncwarp();
          if (++ks == C::KST) {
            ks = 0;
            kph ^= 1;
          }
        }
      }
      if (lane == 0) {
        if (n_seg > 0) mbar_wait_drain(smem_u32(&tail->q_full), (n_seg - 1) & 1, p.status);
        mma_commit(smem_u32(&tail->drain[0]));
        mbar_wait_drain(smem_u32(&tail->drain[0]), 0, p.status);
      }
    } else if (warp == 2) {
      // ---------------------------------------------------------- P.V
      SegReader rd;
      Seg s;
      uint32_t n_seg = 0;
      int i = 0;
      bool ok = true;
      const uint64_t dv0 = desc_mnmajor_sw128(sbase + C::OFF_V, C::KV_PANEL);
      while (ok) {
        if (!rd.take(p, tail->sched, abort, s) || s.nb == 0) break;
        // O still holds the piece before this one until its rows have been read
        if (n_seg > 0 && !KS_PAGED_WAIT(tail->o_free, (n_seg - 1) & 1)) break;
        ++n_seg;
        for (int e = 0; e < s.nb; ++e, ++i) {
          const int vs = i % C::VST, kb = s.key_block(e);
          if (!(ok = KS_PAGED_WAIT(tail->v_full[vs], (i / C::VST) & 1))) break;
          if (s.ragged(kb)) zero_unseen<C::PANELS>(p, s, kb, smem + C::OFF_V + vs * C::V_SLOT, lane);
          if (!(ok = KS_PAGED_WAIT(tail->p_full, i & 1))) break;
          tc_fence_after();
          if (lane == 0) {
            const uint64_t dv = dv0 + (uint64_t)((vs * C::V_SLOT) >> 4);
#pragma unroll
            for (int kk = 0; kk < C::BN / 16; ++kk)
              // 16 keys = 8 packed TMEM columns of P, 16 rows of 128 bytes further along V
              mma_bf16_tmem_a(tmem + C::TMEM_O, tmem + C::TMEM_P + kk * 8,
                              dv + (uint64_t)(kk * ((16 * 128) >> 4)), C::IDESC_O,
                              (e > 0 || kk > 0) ? 1u : 0u);
            mma_commit(smem_u32(&tail->pv_done[i & 1]));
            mma_commit(smem_u32(&tail->v_empty[vs]));
          }
          __syncwarp();
        }
      }
      if (lane == 0) {
        mma_commit(smem_u32(&tail->drain[1]));
        mbar_wait_drain(smem_u32(&tail->drain[1]), 0, p.status);
      }
    }
  } else {
    regs_inc<C::REGS_HIGH>();
    // ------------------------------------------------------------ softmax groups (warps 4-11)
    const int G = (warp - 4) >> 2;               // group: blocks i with i % 2 == G
    const int q4 = warp & 3;                     // TMEM lane quarter this warp may access
    const int r = q4 * 32 + lane;                // row of the tile = TMEM lane
    const int rt = r / p.grp;                    // its token in the tile
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const uint32_t ts = tmem + lane_off + C::TMEM_S + G * C::BN;
    const uint32_t tp = tmem + lane_off + C::TMEM_P;
    constexpr int NC = C::BN;                    // scores per row and block
    const float sl2 = p.scale_log2;
    SegReader rd;
    int i0 = 0;                                  // number of the piece's first block
    uint32_t syncs = 0;
    bool ok = true;
    // waits until PV_q has completed.  PV_q commits to pv_done[q % 2], whose phases
    // are PV_{q-2}, PV_q, PV_{q+2}...; at every wait below PV_{q-2} has completed
    // (this group waited for it, or for a later P.V, whose commit covers it) and
    // PV_{q+2} cannot have (it needs a P this group has not yet written), so a
    // parity wait sees the right phase
    auto wait_pv = [&](int q) -> bool {
      if (!KS_PAGED_WAIT(tail->pv_done[q & 1], (q >> 1) & 1)) return false;
      tc_fence_after();
      return true;
    };
    auto meet = [&]() -> bool {                  // this group's four warps
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&tail->gsync[G]));
      return KS_PAGED_WAIT(tail->gsync[G], syncs++ & 1);
    };
    while (ok) {
      const Seg* sp = rd.peek(p, tail->sched, abort);
      if (!sp || sp->nb == 0) break;
      const Seg& s = *sp;
      const bool idle = q4 * 32 >= s.tokens * p.grp;   // no row of this warp is in the tile
      const int lead = i0 + s.lead - s.k0, trail = i0 + s.trail - s.k0;   // blocks to mask: outside
      float m_new = kNoRef;
      for (int i = i0 + ((i0 ^ G) & 1); i < i0 + s.nb; i += 2) {
        if (!KS_PAGED_WAIT(tail->s_full[G], (i >> 1) & 1)) {
          ok = false;
          break;
        }
        if (idle) {                              // keep in step, and leave the exponentials to the others
          if (lane == 0) mbar_arrive(smem_u32(&tail->s_free[G]));
          ok = i == 0 || KS_PAGED_WAIT(tail->m_ready[1 - G], ((i - 1) >> 1) & 1);
          if (ok && lane == 0) mbar_arrive(smem_u32(&tail->m_ready[G]));
          if (ok && i >= 1) ok = wait_pv(i - 1);
          if (!ok) break;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&tail->p_full));
          continue;
        }
        if (q4 == 0 && lane == 0) mbar_arrive(smem_u32(&tail->k_empty[i % C::KST]));   // K_i read
        tc_fence_after();
        float sc[NC];
#pragma unroll
        for (int c = 0; c < NC / 32; ++c)
          tmem_ld32(ts + c * 32, *reinterpret_cast<float(*)[32]>(&sc[c * 32]));
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < NC / 32; ++c) reg_fence32(*reinterpret_cast<float(*)[32]>(&sc[c * 32]));
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&tail->s_free[G]));   // S_{i+2} may be computed now
        if (i < lead || i >= trail) {
          const int kb = s.key_block(i - i0);
          // a row sees keys of the table up to its position that are in its window or among the
          // first; as ranges of this block: e <= last, and e >= wlo or e < sinks
          const int key0 = kb * C::BN;
          const int pos = s.p_first + rt, last = min(pos, s.last_key) - key0;
          const int wlo = p.window > 0 && pos >= p.window ? pos - p.window + 1 - key0 : 0;
          const int sk = p.window > 0 ? p.sinks - key0 : 0;
#pragma unroll
          for (int e = 0; e < NC; ++e)
            if (e > last || (e < wlo && e >= sk)) sc[e] = -INFINITY;
        }
        float mx[4] = {sc[0], sc[1], sc[2], sc[3]};
#pragma unroll
        for (int e = 4; e < NC; e += 2)          // columns 4 .. NC-1, two at a time
          mx[(e >> 1) & 3] = fmax3(mx[(e >> 1) & 3], sc[e], sc[e + 1]);
        const float bmax = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        // the reference of the previous block, from the other group (waited for on a piece's first
        // block too, which keeps the groups within a phase of each other)
        float m_in = kNoRef;
        if (i > 0) {
          if (!KS_PAGED_WAIT(tail->m_ready[1 - G], ((i - 1) >> 1) & 1)) {
            ok = false;
            break;
          }
          if (i > i0) m_in = tail->m_pub[1 - G][r];
        }
        const bool grow = (bmax - m_in) * sl2 > kStale;
        m_new = grow ? bmax : m_in;
        tail->m_pub[G][r] = m_new;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&tail->m_ready[G]));
        if (__any_sync(0xffffffffu, grow && i > i0)) {
          // O and its row sums hold the P.V of the piece's blocks < i relative to m_in: rescale
          // them once PV_{i-1} has landed
          if (!wait_pv(i - 1)) {
            ok = false;
            break;
          }
          const float a = grow ? ex2((m_in - m_new) * sl2) : 1.0f;
          float v[32];
#pragma unroll
          for (int c = 0; c < HD / 32; ++c) {
            const uint32_t to = tmem + lane_off + C::TMEM_O + c * 32;
            tmem_ld32(to, v);
            tmem_wait_ld();
            reg_fence32(v);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] *= a;
            tmem_st32(to, v);
          }
          {
            const uint32_t to = tmem + lane_off + C::TMEM_O + HD;   // the 16 row-sum columns
            tmem_wait_st();                        // the stores above land before this reload
            tmem_ld32(to - 16, v);                 // 32 columns ending at the sums: HD-16 .. HD+15
            tmem_wait_ld();
            reg_fence32(v);
#pragma unroll
            for (int e = 16; e < 32; ++e) v[e] *= a;   // the first 16 were rescaled above
            tmem_st32(to - 16, v);
          }
        }
        const uint64_t scale2 = pk2(sl2, sl2);
        const uint64_t moff2 = pk2(-m_new * sl2, -m_new * sl2);
        uint32_t pk[NC / 2];                       // P of the block as bf16 pairs
#pragma unroll
        for (int e = 0; e < NC; e += 2) {
          float x0, x1, p0, p1;
          upk2(fma2(pk2(sc[e], sc[e + 1]), scale2, moff2), x0, x1);
          p0 = ex2(x0);
          p1 = ex2(x1);
          pk[e >> 1] = pack2(p0, p1);
        }
        // the P buffer was last read by PV_{i-1}: wait for it only now, with P in registers
        if (i >= 1 && !wait_pv(i - 1)) {
          ok = false;
          break;
        }
#pragma unroll
        for (int c = 0; c < NC / 32; ++c) tmem_st16u(tp + c * 16, &pk[c * 16]);
        tmem_wait_st();                            // P and any O rescale stores complete
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&tail->p_full));
      }
      const int last = i0 + s.nb - 1;
      i0 += s.nb;
      if (!ok) break;
      if (G != (last & 1)) {
        rd.release(tail->sched);
        continue;
      }
      // the group of the piece's last block reads O and its row sum
      if (!wait_pv(last)) break;
      const bool cut = s.nb < s.blocks;
      const int rows = s.tokens * p.grp;
      float v[32];
      tmem_ld32(tmem + lane_off + C::TMEM_O + HD - 16, v);   // HD-16 .. HD+15: the sum at 16
      tmem_wait_ld();
      reg_fence32(v);
      const float sum = v[16], inv = sum > 0.f ? 1.0f / sum : 0.f;
      unsigned char* pc = own_piece(p, s);
      uint4* dst = reinterpret_cast<uint4*>(
          p.out + ((long long)(s.row0 + rt) * p.Hq + s.g * p.grp + (r - rt * p.grp)) * HD);
      float4* part = reinterpret_cast<float4*>(reinterpret_cast<float*>(pc + kPieceStats) + r * HD);
#pragma unroll
      for (int c = 0; c < HD / 32; ++c) {
        tmem_ld32(tmem + lane_off + C::TMEM_O + c * 32, v);
        tmem_wait_ld();
        reg_fence32(v);
        if (r < rows) {
          if (cut) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              __stcg(part + c * 8 + e,
                     make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]));
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              dst[c * 4 + e] = make_uint4(pack2(v[8 * e] * inv, v[8 * e + 1] * inv),
                                          pack2(v[8 * e + 2] * inv, v[8 * e + 3] * inv),
                                          pack2(v[8 * e + 4] * inv, v[8 * e + 5] * inv),
                                          pack2(v[8 * e + 6] * inv, v[8 * e + 7] * inv));
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&tail->o_free));
      if (!cut) {
        rd.release(tail->sched);
        continue;
      }
      if (r < rows) __stcg(reinterpret_cast<float2*>(pc) + r, make_float2(m_new * sl2, sum));
      if (!meet()) break;
      if (q4 == 0 && lane == 0) tail->last[G] = arrive_piece(p, s);
      if (!meet()) break;
      if (tail->last[G]) {
        join_pieces<HD>(p, s, q4, 4, lane);
      }
      rd.release(tail->sched);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <int HD>
ks_status launch(const Params& p, const CUtensorMap& tq, const CUtensorMap& tk,
                 const CUtensorMap& tv, int grid, cudaStream_t st) {
  using C = Cfg<HD>;
  static std::atomic<unsigned long long> attr{0};
  auto k = paged_chunk_kernel<HD>;
  KS_TRY(once_per_device(attr, [&]() -> ks_status {
    // the setmaxnreg split assumes exactly C::REGS registers a thread at launch
    cudaFuncAttributes fa;
    KS_CUDA_TRY(cudaFuncGetAttributes(&fa, k));
    if (fa.numRegs != C::REGS)
      return fail(KS_ERR_INTERNAL, "paged attention: kernel built with " + std::to_string(fa.numRegs) +
                                       " registers a thread, the register split needs " +
                                       std::to_string(C::REGS));
    KS_CUDA_TRY(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM));
    return KS_OK;
  }));
  k<<<grid, kThreads, C::SMEM, st>>>(tq, tk, tv, p);
  KS_LAUNCH_CHECK();
  return KS_OK;
}

}  // namespace

ks_status launch_paged_chunk(const PagedAttnArgs& a, const Params& p, int grid, cudaStream_t st) {
  const int hd = a.pool->head_dim;
  const long long kvd = (long long)p.Hkv * hd;
  CUtensorMap tq, tk, tv;
  KS_TRY(make_tmap_heads(&tq, a.q, a.n_tokens, a.Hq, hd, p.grp, p.tile_tokens));
  KS_TRY(make_tmap_2d(&tk, a.pool->k_pages, p.n_slots, kvd, kvd, 64, p.box));
  KS_TRY(make_tmap_2d(&tv, a.pool->v_pages, p.n_slots, kvd, kvd, 64, p.box));
  return hd == 128 ? launch<128>(p, tq, tk, tv, grid, st) : launch<64>(p, tq, tk, tv, grid, st);
}

}  // namespace ks
