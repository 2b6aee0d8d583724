// Attention over the paged cache for up to 64 query rows per request and kv
// head: one token each (a drafting step), a few (a verification), a short chunk
// (sm_100a, tcgen05 + TMEM + TMA).
//
// Every key and value is read once, and a row of them meets few queries, so the
// keys' traffic bounds it.  The products are turned round so that the keys fill
// the tensor core's 128 rows and the queries are its (16 .. 64) columns:
//   S^T = K Q^T      A = K block [128 keys][hd],       B = Q [rows][hd]
//   O^T += V^T P^T   A = V block read MN-major [hd][128], B = P [rows][128 keys]
// A thread of the softmax is then a key, and its work is one exponential per
// query row: with 4 rows a block costs a thread 4 to 8 exponentials, where query
// rows on the lanes would leave 28 of 32 lanes idle behind 128 each.
//
// One persistent CTA per SM takes an equal share of the step's key blocks
// (ks_paged_sched.cuh); 512 threads:
//   warp 0    -- walks the share, publishes its pieces, loads their Q (two buffers)
//                and K blocks (TMA, a ring);
//   warp 2    -- TMEM owner; V blocks into a ring of their own.  In both rings each
//                lane loads the box of one page (the largest power of two of keys,
//                up to 128, that divides the page) of one 64-column panel; issuing
//                a box costs ~57 cycles, so 16-key pages would hold a single warp
//                for longer than a block's bytes take;
//   warp 1    -- S_i; warp 3 -- P.V_i: an issue of eight products with its waits and
//                commits takes ~750 cycles, so one warp for both would be the
//                bottleneck.  Blocks are numbered over the whole share: a short
//                piece's tail runs beside its successor's first products;
//   warps 4-11 -- two softmax groups, each half of the query rows (TMEM columns),
//                thread = key.  P goes to shared memory (two buffers);
//   warps 12-15 -- read a finished piece's O (two buffers in TMEM), write the output
//                or leave the piece and join: the fence and the atomic of a cut
//                piece take ~3 us while memory is busy, which the softmax would
//                otherwise wait out.
// setmaxnreg moves registers between these warpgroups (kRegs* below).
// The softmax reference of a row is kept until a score exceeds it by 2^24, so a
// block needs no maximum: each thread only compares, one vote of the group finds
// the rare block that moves a reference, and only then are maxima taken over the
// keys and O rescaled; a piece begins with the largest score of four keys.  An
// exponent is one fma, score * scale - reference, so it is off by the reference's
// rounding (2^-25 of it, the same for all of a row's keys): scores up to 2^30 cost
// nothing, from 2^32 on 2^that would leave fp32.  Row sums stay with the keys'
// threads in fp32 and are added up once per piece; P is rounded to bf16 for the
// tensor core, O is fp32.
// Measured: 64 requests of one token (32/8 heads of 128, up to 8,192 keys, 1.06 GB)
// 173 us, 6.1 TB/s of the 6.47 of a copy; 32 requests of up to 44 rows, 0.52 GB,
// 106 us.  Heads of 64 move half the bytes a block at the same work per block: the 64
// requests, 530 MB, 139 us.
#include <algorithm>

#include "ks_paged_sched.cuh"
#include "ks_tc.cuh"

namespace ks {

using namespace paged;

namespace {

constexpr int kThreads = 512, kRegs = 128;      // registers a thread at launch
constexpr int kRegsRoles = 72, kRegsSoftmax = 160, kRegsOutput = 120;   // and after setmaxnreg
static_assert(kRegsRoles + 2 * kRegsSoftmax + kRegsOutput == 4 * kRegs, "register split");
// References move once a score exceeds them by 2^24: P and its sums have fp32's and
// bf16's range to grow in, and lose no precision by it.
constexpr float kStale = 24.0f;
constexpr int kMaxRing = 6;                    // slots of the K ring, and of the V ring
constexpr int kSmemLimit = 232448;
constexpr int kSmemFloor = 118784;             // one CTA holds an SM and its 512 TMEM columns

struct Tail {
  SchedSmem sched;
  uint64_t k_full[kMaxRing], k_empty[kMaxRing], v_full[kMaxRing], v_empty[kMaxRing];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2], s_free[2], p_full[2], pv_done[2];   // by block parity
  uint64_t o_full[2], l_full[2], o_free[2];               // by piece parity
  uint64_t esync, drain[2];                               // meetings of the output warps; MMA drains
  uint32_t tmem_base;
  int abort, last;
  // each softmax group's own, by its rows of the piece: the groups do not wait for each other, and
  // the next piece may divide its rows between them differently
  struct alignas(16) {
    float nref[32], alpha[32], wmax[4][32];               // -reference, rescale factor, maxima by warp
  } refs[2];
  float lsum[2][4][64], ref[2][64];                       // a finished piece's, by its parity
};
constexpr int kTailBytes = (int)((sizeof(Tail) + 255) / 256 * 256);

template <int HD>
constexpr int slot_bytes() { return HD / 64 * kBlock * 128; }

// 8 consecutive fp32 columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float* v) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
                 "=f"(v[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
               "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}
// Ties registers filled by tcgen05.ld to the point after its wait.
__device__ __forceinline__ void reg_fence8(float* v) {
  asm volatile(""
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]),
                 "+f"(v[7]));
}

// Largest of the warp's values; floats compare like integers once the negative
// ones' lower bits are flipped.
__device__ __forceinline__ float warp_max(float x) {
  int i = __float_as_int(x);
  i ^= (i >> 31) & 0x7fffffff;
  i = __reduce_max_sync(0xffffffffu, i);
  return __int_as_float(i ^ ((i >> 31) & 0x7fffffff));
}

// Sums of 8 values over the warp's lanes: lane l returns the sum of v[l / 4].
// Each exchange halves the values a lane still carries, so 8 sums take 9 shuffles.
__device__ __forceinline__ float warp_sum8(const float* v, int lane) {
  float a[4], b[2], c;
  const bool h16 = lane & 16, h8 = lane & 8, h4 = lane & 4;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    a[i] = (h16 ? v[i + 4] : v[i]) + __shfl_xor_sync(0xffffffffu, h16 ? v[i] : v[i + 4], 16);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    b[i] = (h8 ? a[i + 2] : a[i]) + __shfl_xor_sync(0xffffffffu, h8 ? a[i] : a[i + 2], 8);
  c = (h4 ? b[1] : b[0]) + __shfl_xor_sync(0xffffffffu, h4 ? b[0] : b[1], 4);
  c += __shfl_xor_sync(0xffffffffu, c, 2);
  return c + __shfl_xor_sync(0xffffffffu, c, 1);
}

// CPG: most query rows that one softmax group handles (half of a tile's).
template <int HD, int CPG>
__global__ void __launch_bounds__(kThreads, 1)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tmQ,
                        const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const __grid_constant__ Params p) {
  constexpr int PANELS = HD / 64, SLOT = slot_bytes<HD>(), NCH = CPG / 8;
  extern __shared__ __align__(1024) unsigned char smem[];
  // the 128-byte-swizzled tiles need a 1024-aligned base; refuse rather than realign
  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) raise_status(p.status, KS_ERR_INTERNAL);
    return;
  }
  const int N = p.q_rows, row_panel = N * 128;           // a 64-column panel of N rows
  const int q_tile = PANELS * row_panel, p_tile = 2 * row_panel;
  const int off_v = p.k_slots * SLOT, off_q = off_v + p.v_slots * SLOT, off_p = off_q + 2 * q_tile;
  Tail* tail = reinterpret_cast<Tail*>(smem + off_p + 2 * p_tile);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &tail->abort;
  const uint32_t sbase = smem_u32(smem);

  if (threadIdx.x == kThreads - 32) {          // the first warps have requests to read
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
    for (int s = 0; s < kMaxRing; ++s) {
      mbar_init(smem_u32(&tail->k_full[s]), 1);
      mbar_init(smem_u32(&tail->k_empty[s]), 1);
      mbar_init(smem_u32(&tail->v_full[s]), 1);
      mbar_init(smem_u32(&tail->v_empty[s]), 1);
    }
    for (int s = 0; s < kSegRing; ++s) {
      mbar_init(smem_u32(&tail->sched.full[s]), 1);
      mbar_init(smem_u32(&tail->sched.empty[s]), 15);    // V, S, P.V, 8 softmax and 4 output warps
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&tail->q_full[b]), 1);
      mbar_init(smem_u32(&tail->q_empty[b]), 1);
      mbar_init(smem_u32(&tail->s_full[b]), 1);
      mbar_init(smem_u32(&tail->s_free[b]), 8);
      mbar_init(smem_u32(&tail->p_full[b]), 8);
      mbar_init(smem_u32(&tail->pv_done[b]), 1);
      mbar_init(smem_u32(&tail->o_full[b]), 1);
      mbar_init(smem_u32(&tail->l_full[b]), 8);
      mbar_init(smem_u32(&tail->o_free[b]), 4);
    }
    mbar_init(smem_u32(&tail->esync), 4);
    mbar_init(smem_u32(&tail->drain[0]), 1);
    mbar_init(smem_u32(&tail->drain[1]), 1);
    tail->abort = 0;
    fence_barrier_init();
  }
  if (warp == 2) {
    tmem_alloc(smem_u32(&tail->tmem_base), 512);
    tmem_relinquish();
  }
  // rows of a Q tile that no load writes (the tile's rows rounded up to 16)
  const int box_rows = p.grp * p.tile_tokens;
  for (int e = threadIdx.x; e < 2 * PANELS * (N - box_rows) * 8; e += kThreads) {
    const int pn = e / ((N - box_rows) * 8), o = e - pn * ((N - box_rows) * 8);
    reinterpret_cast<uint4*>(smem + off_q + pn * row_panel + box_rows * 128)[o] =
        make_uint4(0, 0, 0, 0);
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  locate<kThreads / 32>(p, tail->sched);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tail->tmem_base;
  constexpr uint32_t kS = 0, kO = 256;         // TMEM columns: S[b] at 128 b, O[piece parity] from 256

  if (warp < 4) {
    regs_dec<kRegsRoles>();
    if (warp == 0 || warp == 2) {
      // ---------------------------------------------------------- TMA: the walk, Q and K; V
      const bool is_k = warp == 0;
      const Ring ring{is_k ? &tmK : &tmV, is_k ? tail->k_full : tail->v_full,
                      is_k ? tail->k_empty : tail->v_empty, sbase + (is_k ? 0 : off_v),
                      is_k ? p.k_slots : p.v_slots, SLOT};
      int n_seg = 0;
      load_share<HD>(p, tail->sched, ring, is_k, abort, [&](const Seg& s) -> bool {
        const int qb = n_seg & 1;
        if (!KS_PAGED_WAIT(tail->q_empty[qb], ((n_seg >> 1) & 1) ^ 1)) return false;
        if (lane == 0) {
          const uint32_t qf = smem_u32(&tail->q_full[qb]);
          mbar_arrive_expect_tx(qf, PANELS * box_rows * 128);
          for (int pn = 0; pn < PANELS; ++pn)
            tma_load_3d(sbase + off_q + qb * q_tile + pn * row_panel, &tmQ, pn * 64, s.g * p.grp,
                        s.row0, qf);
        }
        __syncwarp();
        ++n_seg;
        return true;
      });
      if (lane == 0)
        for (int n = n_seg > 2 ? n_seg - 2 : 0; n < n_seg; ++n)
          mbar_wait_drain(smem_u32(&tail->q_full[n & 1]), (n >> 1) & 1, p.status);
    } else if (warp == 1) {
      // ------------------------------------------------------------ S_i = K_i Q^T
      SegReader rd;
      int slot = 0;
      uint32_t phase = 0, i = 0, n_seg = 0;
      bool ok = true;
      const uint32_t idesc = idesc_bf16_f32(128, N);
      const uint64_t dk0 = desc_kmajor_sw128(sbase), dq0 = desc_kmajor_sw128(sbase + off_q);
      const uint32_t rp16 = row_panel >> 4;
      while (ok) {
        const Seg* s = rd.peek(p, tail->sched, abort);
        const int nb = s ? s->nb : 0;
        if (nb == 0) break;
        rd.release(tail->sched);
        const uint32_t qb = n_seg & 1;
        ok = KS_PAGED_WAIT(tail->q_full[qb], (n_seg >> 1) & 1);
        ++n_seg;
        for (int e = 0; ok && e < nb; ++e, ++i) {
          // into S buffer i % 2, free once the softmax has copied S_{i-2}
          const uint32_t b = i & 1;
          if (i >= 2 && !(ok = KS_PAGED_WAIT(tail->s_free[b], ((i - 2) >> 1) & 1))) break;
          if (!(ok = KS_PAGED_WAIT(tail->k_full[slot], phase))) break;
          tc_fence_after();
          if (lane == 0) {
            const uint64_t dk = dk0 + (uint64_t)((slot * SLOT) >> 4);
            const uint64_t dq = dq0 + (uint64_t)((qb * q_tile) >> 4);
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk)
              mma_bf16(tmem + kS + b * 128, dk + (uint64_t)((kk / 4) * ((kBlock * 128) >> 4) + 2 * (kk % 4)),
                       dq + (uint64_t)((kk / 4) * rp16 + 2 * (kk % 4)), idesc, kk > 0);
            mma_commit(smem_u32(&tail->s_full[b]));
            mma_commit(smem_u32(&tail->k_empty[slot]));
            if (e == nb - 1) mma_commit(smem_u32(&tail->q_empty[qb]));
          }
          __syncwarp();
          if (++slot == p.k_slots) {
            slot = 0;
            phase ^= 1;
          }
        }
      }
      if (lane == 0) {
        mma_commit(smem_u32(&tail->drain[0]));
        mbar_wait_drain(smem_u32(&tail->drain[0]), 0, p.status);
      }
    } else if (warp == 3) {
      // ------------------------------------------------------------ O^T += V_i^T P_i
      SegReader rd;
      Seg s;
      int slot = 0;
      uint32_t phase = 0, i = 0, n_seg = 0;
      bool ok = true;
      const uint32_t idesc = idesc_bf16_f32(128, N) | (1u << 15);   // A (V) MN-major
      const uint64_t dp0 = desc_kmajor_sw128(sbase + off_p);
      // head_dim 64: rows 64 .. 127 of the product repeat V's columns some keys further on; nobody
      // reads them
      const uint64_t dv0 = desc_mnmajor_sw128(sbase + off_v, PANELS == 2 ? kBlock * 128 : 1024);
      const uint32_t rp16 = row_panel >> 4;
      while (ok) {
        if (!rd.take(p, tail->sched, abort, s) || s.nb == 0) break;
        // O holds the piece before the last until its rows have been read
        const uint32_t ob = n_seg & 1;
        if (n_seg >= 2 && !KS_PAGED_WAIT(tail->o_free[ob], ((n_seg - 2) >> 1) & 1)) break;
        ++n_seg;
        for (int e = 0; e < s.nb; ++e, ++i) {
          const uint32_t b = i & 1;
          const int kb = s.key_block(e);
          if (!(ok = KS_PAGED_WAIT(tail->v_full[slot], phase))) break;
          if (s.ragged(kb)) zero_unseen<PANELS>(p, s, kb, smem + off_v + slot * SLOT, lane);
          if (!(ok = KS_PAGED_WAIT(tail->p_full[b], (i >> 1) & 1))) break;
          tc_fence_after();
          if (lane == 0) {
            const uint64_t dv = dv0 + (uint64_t)((slot * SLOT) >> 4);
            const uint64_t dp = dp0 + (uint64_t)((b * p_tile) >> 4);
#pragma unroll
            for (int kk = 0; kk < kBlock / 16; ++kk)
              mma_bf16(tmem + kO + ob * 64, dv + (uint64_t)(kk * ((16 * 128) >> 4)),
                       dp + (uint64_t)((kk / 4) * rp16 + 2 * (kk % 4)), idesc, e > 0 || kk > 0);
            mma_commit(smem_u32(&tail->v_empty[slot]));
            mma_commit(smem_u32(&tail->pv_done[b]));
            if (e == s.nb - 1) mma_commit(smem_u32(&tail->o_full[ob]));
          }
          __syncwarp();
          if (++slot == p.v_slots) {
            slot = 0;
            phase ^= 1;
          }
        }
      }
      if (lane == 0) {
        mma_commit(smem_u32(&tail->drain[1]));
        mbar_wait_drain(smem_u32(&tail->drain[1]), 0, p.status);
      }
    }
  } else if (warp < 12) {
    regs_inc<kRegsSoftmax>();
    // ------------------------------------------------------------ softmax
    const int G = (warp - 4) >> 2, q4 = warp & 3;
    const int key = q4 * 32 + lane;            // key of the block = TMEM lane
    const uint32_t lanes = (uint32_t)(q4 * 32) << 16;
    const float sl2 = p.scale_log2;
    // byte of this key in a row of P: 64-key panel, and the swizzled 16-byte chunk of row e % 8
    const uint32_t p_key = (key >> 6) * row_panel + (key & 7) * 2;
    const uint32_t p_chunk = (key & 63) >> 3;
    auto& refs = tail->refs[G];
    SegReader rd;
    uint32_t j = 0;
    bool ok = true;
    // The group's four warps meet at a hardware barrier (shorter than an mbarrier's round trip) and
    // vote: the count is 0, 1 .. 4 when some of them ask for new references, 32 or more when one
    // has given up.  A barrier has no time limit, so a warp that leaves, for whatever reason but
    // such a vote, comes to one more: its partners are then never left waiting.
    bool voted_out = false, finished = false;
    auto vote = [&](bool mine) -> int {
      int n;
      asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
                   "bar.red.popc.u32 %0, %1, 128, q;\n\t}"
                   : "=r"(n)
                   : "r"(1 + G), "r"((int)mine)
                   : "memory");
      voted_out = n >= 32;
      return n;
    };
    auto meet = [&]() -> bool { return vote(false) < 32; };
    // PV_q commits to pv_done[q % 2]; whoever waits for it has waited for PV_{q-2} before, and
    // PV_{q+2} needs a P that this warp has not written, so the parity is unambiguous
    auto wait_pv = [&](uint32_t q) -> bool {
      if (!KS_PAGED_WAIT(tail->pv_done[q & 1], (q >> 1) & 1)) return false;
      tc_fence_after();
      return true;
    };
    while (ok) {
      const Seg* cur = rd.peek(p, tail->sched, abort);
      if (!cur) break;
      const Seg& s = *cur;
      const int nb = s.nb;
      if (nb == 0) {
        finished = true;
        break;
      }
      const uint32_t par = rd.n & 1, to_o = tmem + lanes + kO + par * 64;
      const int rows = s.tokens * p.grp, chunks = (rows + 7) >> 3, half = (chunks + 1) >> 1;
      const int r0 = G ? half * 8 : 0;         // this group's first row
      const int nch = G ? chunks - half : half;
      const int lead = s.lead - s.k0, trail = s.trail - s.k0;   // blocks to mask: outside
      float l[CPG];
#pragma unroll
      for (int c = 0; c < CPG; ++c) l[c] = 0.f;
      for (int i = 0; i < nb; ++i, ++j) {
        const uint32_t b = j & 1;
        if (!KS_PAGED_WAIT(tail->s_full[b], (j >> 1) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        float sc[CPG];
#pragma unroll
        for (int c = 0; c < NCH; ++c)
          if (c < nch) tmem_ld8(tmem + lanes + kS + b * 128 + r0 + c * 8, &sc[c * 8]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < NCH; ++c) reg_fence8(&sc[c * 8]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&tail->s_free[b]));   // S_{j+2} may be computed now
        if (nch > 0) {
          if (i < lead || i >= trail) {
            // row r is token r / grp at p_first + r / grp: it sees key k from row (k - p_first) grp
            // on, and while the key is in its window up to row (k - p_first + window) grp; keys past
            // the table's row are nobody's
            const int k = s.key_block(i) * kBlock + key;
            const long long d = (long long)k - s.p_first;
            const int from = (int)(d < 0 ? 0 : d > 128 ? 128 : d) * p.grp;
            int to = 1 << 20;
            if (p.window > 0 && k >= p.sinks) {
              const long long e = d + p.window;
              to = (int)(e < 0 ? 0 : e > 128 ? 128 : e) * p.grp;
            }
            if (k > s.last_key) to = 0;
#pragma unroll
            for (int c = 0; c < CPG; ++c)
              if (r0 + c < from || r0 + c >= to) sc[c] = -INFINITY;
          }
          if (i == 0) {
            // a piece's first references: the largest score of four of its keys will do, since
            // a row's P and sums may grow to 2^kStale times the reference's before it moves
            if (lane == 0) {
#pragma unroll
              for (int c = 0; c < NCH; ++c)
                if (c < nch)
#pragma unroll
                  for (int e = 0; e < 8; e += 4)
                    *reinterpret_cast<float4*>(&refs.wmax[q4][c * 8 + e]) = make_float4(
                        sc[c * 8 + e], sc[c * 8 + e + 1], sc[c * 8 + e + 2], sc[c * 8 + e + 3]);
            }
            if (!meet()) {
              ok = false;
              break;
            }
            if (key < nch * 8) {
              const float mx = sl2 * fmaxf(fmaxf(refs.wmax[0][key], refs.wmax[1][key]),
                                           fmaxf(refs.wmax[2][key], refs.wmax[3][key]));
              refs.nref[key] = -fmaxf(mx, kNoRef);
            }
            if (!meet()) {
              ok = false;
              break;
            }
          }
          // has a score outgrown its row's reference?
          bool any = false;
#pragma unroll
          for (int c = 0; c < NCH; ++c)
            if (c < nch) {
              const float4 n0 = *reinterpret_cast<const float4*>(&refs.nref[c * 8]);
              const float4 n1 = *reinterpret_cast<const float4*>(&refs.nref[c * 8 + 4]);
              const float* x = &sc[c * 8];
              const float m0 =
                  fmax3(fmaf(x[0], sl2, n0.x), fmaf(x[1], sl2, n0.y), fmaf(x[2], sl2, n0.z));
              const float m1 =
                  fmax3(fmaf(x[3], sl2, n0.w), fmaf(x[4], sl2, n1.x), fmaf(x[5], sl2, n1.y));
              any |= fmax3(m0, m1, fmaxf(fmaf(x[6], sl2, n1.z), fmaf(x[7], sl2, n1.w))) > kStale;
            }
          any = __any_sync(0xffffffffu, any);
          const int votes = vote(any && lane == 0);
          if (votes >= 32) {
            ok = false;
            break;
          }
          const bool grow = votes > 0;
          if (grow) {
            // maxima over the keys, and the rows' new references
#pragma unroll
            for (int c0 = 0; c0 < CPG; c0 += 32) {
              float m = 0.f;
#pragma unroll
              for (int c = c0; c < c0 + 32 && c < CPG; ++c)
                if (c < nch * 8) {
                  const float w = warp_max(sc[c]);
                  if (lane == c - c0) m = w;
                }
              if (c0 + lane < nch * 8) refs.wmax[q4][c0 + lane] = m;
            }
            if (!meet()) {
              ok = false;
              break;
            }
            if (key < nch * 8) {
              const float mx = sl2 * fmaxf(fmaxf(refs.wmax[0][key], refs.wmax[1][key]),
                                           fmaxf(refs.wmax[2][key], refs.wmax[3][key]));
              const float old = -refs.nref[key];
              const bool up = mx - old > kStale;
              refs.alpha[key] = up ? ex2(old - mx) : 1.0f;
              refs.nref[key] = up ? -mx : -old;
            }
            if (!meet()) {
              ok = false;
              break;
            }
            if (i > 0) {
              // sums and O hold the blocks before relative to the old references
              if (!wait_pv(j - 1)) {
                ok = false;
                break;
              }
#pragma unroll
              for (int c = 0; c < NCH; ++c)
                if (c < nch) {
                  float v[8];
                  const uint32_t to = to_o + r0 + c * 8;
                  tmem_ld8(to, v);
                  tmem_wait_ld();
                  reg_fence8(v);
#pragma unroll
                  for (int e = 0; e < 8; ++e) {
                    const float a = refs.alpha[c * 8 + e];
                    v[e] *= a;
                    l[c * 8 + e] *= a;
                  }
                  tmem_st8(to, v);
                }
              tmem_wait_st();
            }
          }
          // the P buffer was last read by PV_{j-2}
          if (j >= 2 && !wait_pv(j - 2)) {
            ok = false;
            break;
          }
          unsigned char* pt = smem + off_p + b * p_tile + p_key + r0 * 128;
#pragma unroll
          for (int c = 0; c < NCH; ++c)
            if (c < nch) {
              const float4 n0 = *reinterpret_cast<const float4*>(&refs.nref[c * 8]);
              const float4 n1 = *reinterpret_cast<const float4*>(&refs.nref[c * 8 + 4]);
              const float n[8] = {n0.x, n0.y, n0.z, n0.w, n1.x, n1.y, n1.z, n1.w};
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float w = ex2(fmaf(sc[c * 8 + e], sl2, n[e]));
                l[c * 8 + e] += w;
                *reinterpret_cast<__nv_bfloat16*>(pt + (c * 8 + e) * 128 + ((p_chunk ^ e) << 4)) =
                    __float2bfloat16_rn(w);
              }
            }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        } else if (j >= 2 && !wait_pv(j - 2)) {   // keep in step
          ok = false;
          break;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&tail->p_full[b]));
      }
      if (!ok) break;
      // the piece's sums and references, for the output warps
      if (rd.n >= 2 && !KS_PAGED_WAIT(tail->o_free[par], ((rd.n - 2) >> 1) & 1)) break;
#pragma unroll
      for (int c = 0; c < NCH; ++c)
        if (c < nch) {
          const float w = warp_sum8(&l[c * 8], lane);
          if ((lane & 3) == 0) tail->lsum[par][q4][r0 + c * 8 + (lane >> 2)] = w;
        }
      if (key < nch * 8) tail->ref[par][r0 + key] = -refs.nref[key];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&tail->l_full[par]));
      rd.release(tail->sched);
    }
    if (!voted_out) vote(!finished);
  } else {
    regs_dec<kRegsOutput>();
    // ------------------------------------------------------------ output
    const int q4 = warp & 3, d = q4 * 32 + lane;   // d: column of the output = TMEM lane
    const uint32_t lanes = (uint32_t)(q4 * 32) << 16;
    SegReader rd;
    uint32_t syncs = 0;
    auto meet = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&tail->esync));
      return KS_PAGED_WAIT(tail->esync, syncs++ & 1);
    };
    while (true) {
      const Seg* cur = rd.peek(p, tail->sched, abort);
      if (!cur || cur->nb == 0) break;
      const Seg& s = *cur;
      const uint32_t par = rd.n & 1, phase = (rd.n >> 1) & 1;
      const int rows = s.tokens * p.grp;
      const bool cut = s.nb < s.blocks;
      unsigned char* pc = own_piece(p, s);
      int hh = 0;
      float* part = reinterpret_cast<float*>(pc + kPieceStats) + d;
      __nv_bfloat16* dst = p.out + ((long long)s.row0 * p.Hq + s.g * p.grp) * HD + d;
      const long long next = (long long)(p.Hq - p.grp + 1) * HD;
      if (!KS_PAGED_WAIT(tail->l_full[par], phase)) break;
      float inv[2];                            // of rows lane and lane + 32
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = lane + 32 * h;
        const float sum = (tail->lsum[par][0][r] + tail->lsum[par][1][r]) +
                          (tail->lsum[par][2][r] + tail->lsum[par][3][r]);
        inv[h] = sum > 0.f ? 1.0f / sum : 0.f;
        if (cut && q4 == 0 && r < rows)
          __stcg(reinterpret_cast<float2*>(pc) + r, make_float2(tail->ref[par][r], sum));
      }
      if (!KS_PAGED_WAIT(tail->o_full[par], phase)) break;
      tc_fence_after();
#pragma unroll 1
      for (int r0 = 0; r0 < rows; r0 += 8) {
        float o[8];
        tmem_ld8(tmem + lanes + kO + par * 64 + r0, o);
        tmem_wait_ld();
        reg_fence8(o);
        const float iv = r0 < 32 ? inv[0] : inv[1];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float f = __shfl_sync(0xffffffffu, iv, (r0 + e) & 31);
          if (r0 + e < rows && d < HD) {
            if (cut) {
              __stcg(part + (r0 + e) * HD, o[e]);
            } else {
              *dst = __float2bfloat16_rn(o[e] * f);
              if (++hh == p.grp) {
                hh = 0;
                dst += next;
              } else {
                dst += HD;
              }
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&tail->o_free[par]));
      if (cut) {
        if (!meet()) break;
        if (warp == 12 && lane == 0) tail->last = arrive_piece(p, s);
        if (!meet()) break;
        if (tail->last) join_pieces<HD>(p, s, q4, 4, lane);
      }
      rd.release(tail->sched);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int HD, int CPG>
ks_status launch(Params p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                 int grid, cudaStream_t st) {
  static std::atomic<unsigned long long> attr{0};
  auto k = paged_decode_kernel<HD, CPG>;
  KS_TRY(once_per_device(attr, [&]() -> ks_status {
    // the setmaxnreg split assumes exactly kRegs registers a thread at launch
    cudaFuncAttributes fa;
    KS_CUDA_TRY(cudaFuncGetAttributes(&fa, k));
    if (fa.numRegs != kRegs)
      return fail(KS_ERR_INTERNAL, "paged attention: kernel built with " + std::to_string(fa.numRegs) +
                                       " registers a thread, the register split needs " +
                                       std::to_string(kRegs));
    KS_CUDA_TRY(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit));
    return KS_OK;
  }));
  const int tiles = (2 * (HD / 64) + 4) * p.q_rows * 128 + kTailBytes;   // Q, P and the rest
  const int slots = std::min(2 * kMaxRing, (kSmemLimit - tiles) / slot_bytes<HD>());
  p.v_slots = (slots + 1) / 2;                 // a V block waits for its P, a K block for nothing
  p.k_slots = slots / 2;
  const int smem = std::max(kSmemFloor, slots * slot_bytes<HD>() + tiles);
  k<<<grid, kThreads, smem, st>>>(tq, tk, tv, p);
  KS_LAUNCH_CHECK();
  return KS_OK;
}

template <int HD>
ks_status launch_hd(const Params& p, const CUtensorMap& tq, const CUtensorMap& tk,
                    const CUtensorMap& tv, int grid, cudaStream_t st) {
  const int rows = p.grp * p.tile_tokens;
  if (rows <= 16) return launch<HD, 8>(p, tq, tk, tv, grid, st);
  if (rows <= 32) return launch<HD, 16>(p, tq, tk, tv, grid, st);
  return launch<HD, 32>(p, tq, tk, tv, grid, st);
}

}  // namespace

ks_status launch_paged_decode(const PagedAttnArgs& a, Params p, int grid, cudaStream_t st) {
  const int hd = a.pool->head_dim;
  p.q_rows = (p.grp * p.tile_tokens + 15) / 16 * 16;
  const long long kvd = (long long)p.Hkv * hd;
  CUtensorMap tq, tk, tv;
  KS_TRY(make_tmap_heads(&tq, a.q, a.n_tokens, a.Hq, hd, p.grp, p.tile_tokens));
  KS_TRY(make_tmap_2d(&tk, a.pool->k_pages, p.n_slots, kvd, kvd, 64, p.box));
  KS_TRY(make_tmap_2d(&tv, a.pool->v_pages, p.n_slots, kvd, kvd, 64, p.box));
  return hd == 128 ? launch_hd<128>(p, tq, tk, tv, grid, st) : launch_hd<64>(p, tq, tk, tv, grid, st);
}

}  // namespace ks
