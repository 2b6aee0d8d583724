// What the two paged-attention kernels share on the device: how a step's
// requests become work, how a CTA walks its share, and how pieces are joined.
//
// Work is counted in key blocks (128 positions).  A unit is one tile of query
// rows (whole tokens x the query heads of one kv head) with the key blocks that
// its tokens see, after kUnitCost blocks' worth of its own cost; units are ordered
// by request, kv head, tile, and concatenated.  CTA c takes the c-th of G equal
// shares of that sequence, whatever the lengths; a unit that crosses a border is
// cut into pieces there, at most two per CTA.  The lengths
// are on the device: every CTA adds the requests' block counts up itself (they
// come from L2) and finds its first block, which costs about as much as reading
// them once and saves a launch.
//
// A piece leaves its unnormalised output, reference and row sum in the
// workspace; the last CTA of a unit to arrive joins the pieces in their order,
// so the result does not depend on who arrives last.
#pragma once

#include "ks_paged.cuh"
#include "ks_sm100.cuh"

namespace ks {
namespace paged {

using namespace sm100;

constexpr int kBlock = 128;                  // keys per block
constexpr int kMaxCtas = 148;                // one CTA per SM of a B200
constexpr int kTileRows = 128;               // query rows of a tile, at most
constexpr int kMaxWarps = 16;
constexpr float kNoRef = -1e30f;             // reference of a row that has seen no key

// Workspace: one arrival counter per CTA (of the unit whose first piece it
// holds), then two pieces per CTA: reference and sum of 128 rows, and the rows.
constexpr size_t kCounterBytes = 1024;
constexpr size_t kPieceStats = 128 * sizeof(float2);
constexpr size_t kPieceBytes = kPieceStats + 128 * 128 * sizeof(float);
constexpr size_t kWorkspaceBytes = kCounterBytes + 2 * kMaxCtas * kPieceBytes;
static_assert(kMaxCtas * sizeof(uint32_t) <= kCounterBytes, "counters");
// Arrivals are counted in steps of kArrival (odd, so it has an inverse modulo 2^32): n arrivals read
// n kArrival, and a word that no arrivals made, a small number above all, stands for a count far past
// any unit's pieces.  In steps of one, a leftover count c < pieces would make the unit's last arrival
// but c join pieces that are not there yet, and be c again afterwards.
constexpr uint32_t kArrival = 0x4164d839u, kArrivalInv = 0xc4db9609u;
static_assert(kArrival * kArrivalInv == 1u, "inverse");

struct Params {
  const int32_t *table, *cu, *kv_len;
  __nv_bfloat16* out;
  unsigned char* ws;
  int32_t* status;
  int B, n_tokens, max_new, max_blocks, cap;   // cap = max_blocks * page_size positions a row
  int Hq, Hkv, grp, page_size, n_pages, n_slots;
  int box, log2_boxes;                         // keys of a TMA box, boxes of a block
  int window, sinks;
  int tile_tokens;                             // tokens per query tile
  int q_rows;                                  // decode kernel: rows of a Q / P tile (N)
  int k_slots, v_slots;                        // decode kernel: ring slots
  float scale_log2;
};

// A request's rows after every clamp that keeps broken lengths inside the
// buffers.  pos0, the position of its first token, follows from the lengths as
// given, so that the rows that are left keep their places whatever is dropped: it
// is negative where kv_len is shorter than the chunk, and past the table's row
// where kv_len is longer than that.
struct Req {
  int row0, n, pos0;
};

__device__ __forceinline__ Req load_req(const Params& p, int b, bool* bad) {
  const long long c0 = p.cu[b], c1 = p.cu[b + 1];
  const int kv_in = p.kv_len[b];
  const long long raw = c1 - c0;
  long long n = raw < p.max_new ? raw : p.max_new;
  if (c0 < 0 || c0 > p.n_tokens) n = 0;
  else if (n > p.n_tokens - c0) n = p.n_tokens - c0;
  if (n < 0) n = 0;
  *bad = n != raw || kv_in < 0 || kv_in > p.cap;
  Req r;
  r.row0 = (int)c0;
  r.n = (int)n;
  r.pos0 = n > 0 ? (int)(max(0, kv_in) - raw) : 0;   // c0 >= 0 here, so raw < 2^31
  return r;
}

// What a unit costs beside its key blocks, in blocks: its query tile, its table
// entries, its output.  Without it CTAs with many short units finish last (128
// requests of up to 500 keys: 70 us against 60; longer ones do not notice).
constexpr int kUnitCost = 2;

struct Tile {
  int row0, tokens, p_first;                   // p_first: position of its first token
  int p_end, last_key;                         // of its last token; the same inside the table's row
  int lo, sinks;                               // its tokens see [0, sinks) and [lo, last_key]
  int sink_blocks, blocks;                     // blocks before block lo / 128, blocks in all
  __device__ __forceinline__ int cost() const { return kUnitCost + blocks; }
};

__device__ __forceinline__ Tile make_tile(const Params& p, const Req& r, int tile) {
  Tile t;
  const int t0 = tile * p.tile_tokens;
  t.row0 = r.row0 + t0;
  t.tokens = min(p.tile_tokens, r.n - t0);
  t.p_first = r.pos0 + t0;
  t.p_end = t.p_first + t.tokens - 1;
  t.last_key = min(t.p_end, p.cap - 1);
  t.lo = p.window > 0 && t.p_first >= p.window ? min(t.p_first - p.window + 1, p.cap) : 0;
  t.sinks = p.window > 0 ? min(p.sinks, t.lo) : 0;
  const int b0 = t.lo / kBlock;
  t.sink_blocks = min((t.sinks + kBlock - 1) / kBlock, b0);
  // a tile whose tokens see nothing still has one (masked) block: its rows are zeros
  t.blocks = max(1, t.sink_blocks + (t.last_key >= 0 ? t.last_key / kBlock - b0 + 1 : 0));
  return t;
}

__device__ __forceinline__ int n_tiles(const Params& p, const Req& r) {
  return r.n <= p.tile_tokens ? (r.n > 0) : (r.n + p.tile_tokens - 1) / p.tile_tokens;
}

// One piece of a unit, as the roles of a CTA read it from the ring.
struct alignas(16) Seg {
  int b, g, row0, tokens;
  int p_first, last_key, lo, sinks;
  int sink_blocks, k0, nb, blocks;             // blocks k0 .. k0+nb-1 of the unit's `blocks`; nb = 0 ends
  int first_cta, pieces;                       // of a cut unit (pieces = 1 otherwise)
  int lead, trail;                             // unit blocks k with some key hidden from some token:
                                               // k < lead or k >= trail
  __device__ __forceinline__ int key_block(int i) const {   // i counts from k0
    const int k = k0 + i;
    return k < sink_blocks ? k : lo / kBlock + (k - sink_blocks);
  }
  // Keys [j0, j1] of which no token of the tile sees any.
  __device__ __forceinline__ bool unseen(int j0, int j1) const {
    return j0 > last_key || (j1 < lo && j0 >= sinks);
  }
  // Some key of this block is hidden from every token.
  __device__ __forceinline__ bool ragged(int kb) const {
    const int j0 = kb * kBlock, j1 = j0 + kBlock - 1;
    return j1 > last_key || (j0 < lo && j1 >= sinks);
  }
};
static_assert(sizeof(Seg) == 64, "segments are copied as four uint4");

constexpr int kSegRing = 8;

struct Start {                                 // a CTA's share, and where the walk stands
  long long first, end, total;                 // the share; the step's whole cost
  long long unit;                              // where the current unit begins
  int ctas;                                    // CTAs that have a share
  int b, g, tile;
};

struct SchedSmem {
  Seg seg[kSegRing];
  uint64_t full[kSegRing], empty[kSegRing];
  Start start;                                 // later: where the walk stands
  Req held[32];                                // requests base .. base + 31
  int base, published;
  long long warp_sum[kMaxWarps];
};

// Quotient of non-negative numbers.  Block numbers almost always fit 32 bits, and a
// 64-bit division costs hundreds of cycles of a kernel that may take ten thousand.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}
__device__ __forceinline__ long long warp_sum_ll(long long v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}
__device__ __forceinline__ long long warp_scan_ll(long long v, int lane) {   // inclusive
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += u;
  }
  return v;
}
__device__ __forceinline__ Req shfl_req(const Req& r, int src) {
  Req o;
  o.row0 = __shfl_sync(0xffffffffu, r.row0, src);
  o.n = __shfl_sync(0xffffffffu, r.n, src);
  o.pos0 = __shfl_sync(0xffffffffu, r.pos0, src);
  return o;
}

// Cost of one kv head of the lane's request.  Lanes with few tiles add theirs
// up alone; a request of many tiles is shared by the warp.
__device__ __forceinline__ long long head_cost(const Params& p, const Req& r, int lane) {
  const int T = n_tiles(p, r);
  long long w = 0;
  if (T <= 4)
    for (int t = 0; t < T; ++t) w += make_tile(p, r, t).cost();
  unsigned many = __ballot_sync(0xffffffffu, T > 4);
  while (many) {
    const int src = __ffs(many) - 1;
    many &= many - 1;
    const Req q = shfl_req(r, src);
    const int Tq = n_tiles(p, q);
    long long s = 0;
    for (int t = lane; t < Tq; t += 32) s += make_tile(p, q, t).cost();
    s = warp_sum_ll(s);
    if (lane == src) w = s;
  }
  return w;
}

// Finds the CTA's share (all W warps; sm.start is valid after the caller's next
// __syncthreads).
template <int W>
__device__ __forceinline__ void locate(const Params& p, SchedSmem& sm) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = (p.B + W - 1) / W;
  const int r0 = min(warp * per, p.B), r1 = min(r0 + per, p.B);
  long long mine = 0, w_first = 0;
  Req r_first{0, 0, 0};
  for (int base = r0; base < r1; base += 32) {
    Req r{0, 0, 0};
    bool bad = false;
    if (base + lane < p.B) r = load_req(p, base + lane, &bad);
    if (bad) raise_status(p.status, KS_ERR_INVALID_ARG);
    // lanes past r1 hold another warp's requests, which the walk may come to
    const long long w = head_cost(p, base + lane < r1 ? r : Req{0, 0, 0}, lane) * p.Hkv;
    if (base == r0) {
      r_first = r;
      w_first = w;
    }
    mine += warp_sum_ll(w);
  }
  if (threadIdx.x == 0) {
    sm.start.unit = sm.start.end = 0;
    sm.published = 0;
  }
  if (lane == 0) sm.warp_sum[warp] = mine;
  __syncthreads();
  long long total = 0, before = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w == warp) before = total;
    total += sm.warp_sum[w];
  }
  const int ctas = (int)(total < gridDim.x ? total : gridDim.x);
  const int c = blockIdx.x;
  if (c >= ctas) return;                       // no share (or no work at all)
  const long long first = quotient(total * c, ctas), end = quotient(total * (c + 1), ctas);
  if (first < before || first >= before + mine) return;
  long long at = before;
  for (int base = r0; base < r1; base += 32) {
    Req r = r_first;
    long long w = w_first;
    if (base != r0) {
      bool bad;
      r = Req{0, 0, 0};
      if (base + lane < p.B) r = load_req(p, base + lane, &bad);
      w = head_cost(p, base + lane < r1 ? r : Req{0, 0, 0}, lane) * p.Hkv;
    }
    const long long upto = at + warp_scan_ll(w, lane);
    const unsigned hit = __ballot_sync(0xffffffffu, first < upto);
    if (!hit) {
      at = __shfl_sync(0xffffffffu, upto, 31);
      continue;
    }
    const int src = __ffs(hit) - 1;
    const Req q = shfl_req(r, src);
    const long long head = quotient(__shfl_sync(0xffffffffu, w, src), p.Hkv);
    const long long off = first - __shfl_sync(0xffffffffu, upto - w, src);
    const int g = (int)quotient(off, head), T = n_tiles(p, q);
    long long rest = off - g * head;
    for (int t0 = 0; t0 < T; t0 += 32) {
      const long long nb = t0 + lane < T ? make_tile(p, q, t0 + lane).cost() : 0;
      const long long s = warp_scan_ll(nb, lane);
      const unsigned in = __ballot_sync(0xffffffffu, rest < s);
      if (in) {
        const int l = __ffs(in) - 1;
        const long long in_unit = rest - __shfl_sync(0xffffffffu, s - nb, l);
        sm.held[lane] = r;                     // the walk begins with these requests
        if (lane == 0) {
          sm.start = Start{first, end, total, first - in_unit, ctas, base + src, g, t0 + l};
          sm.base = base;
        }
        return;
      }
      rest -= __shfl_sync(0xffffffffu, s, 31);
    }
    return;
  }
}

// Warp-uniform wait that also reports a lane's timeout to the others.
#define KS_PAGED_WAIT(bar, parity) warp_wait(smem_u32(&(bar)), (uint32_t)(parity), abort, p.status)

// The walk over a CTA's share, by the warp that loads its keys.  Its state lies in
// shared memory: the loading loop has few registers.
__device__ __forceinline__ void hold_requests(const Params& p, SchedSmem& sm, int base, int lane) {
  bool bad;
  Req r{0, 0, 0};
  if (base + lane < p.B) r = load_req(p, base + lane, &bad);
  sm.held[lane] = r;
  if (lane == 0) sm.base = base;
  __syncwarp();
}
// The first request from b on whose offsets grow (p.B if there is none).  Only such a one can have
// tokens; 256 are looked at per round trip, since a step of a large batch may have thousands of idle
// requests in a row (16,376 of them between live ones: 1,340 us at 32 per round trip, 45 us now).
__device__ __forceinline__ int next_growing(const Params& p, int b, int lane) {
  constexpr int N = 8;
  for (; b < p.B; b += 32 * N) {
    int last = p.cu[b], next[N];               // past the batch's end the offsets do not grow
#pragma unroll
    for (int e = 0; e < N; ++e) next[e] = p.cu[min(b + 32 * e + lane + 1, p.B)];
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const int before = __shfl_up_sync(0xffffffffu, next[e], 1);
      const unsigned m = __ballot_sync(0xffffffffu, next[e] > (lane ? before : last));
      if (m) return b + 32 * e + __ffs(m) - 1;
      last = __shfl_sync(0xffffffffu, next[e], 31);
    }
  }
  return p.B;
}
// Publishes the next piece (nb = 0: the end) and returns it, or NULL to give up.
__device__ __forceinline__ const Seg* walk(const Params& p, SchedSmem& sm, volatile int* abort) {
  const int lane = threadIdx.x & 31, n = sm.published, slot = n % kSegRing;
  if (!KS_PAGED_WAIT(sm.empty[slot], ((n / kSegRing) & 1) ^ 1)) return nullptr;
  Seg* seg = &sm.seg[slot];
  Start& st = sm.start;
  // block x of a unit that begins at u lies at u + kUnitCost + x
  const bool over = st.unit + kUnitCost >= st.end || st.b >= p.B;
  bool next_request = false;
  if (lane == 0) {
    sm.published = n + 1;
    if (over) {
      seg->nb = 0;
    } else {
      const Req r = sm.held[st.b - sm.base];
      const Tile t = make_tile(p, r, st.tile);
      const long long x0 = st.unit + kUnitCost;
      const int k = (int)max(0ll, st.first - x0);
      const int nb = (int)min((long long)t.blocks, st.end - x0) - k;
      Seg s;
      s.b = st.b;
      s.g = st.g;
      s.row0 = t.row0;
      s.tokens = t.tokens;
      s.p_first = t.p_first;
      s.last_key = t.last_key;
      s.lo = t.lo;
      s.sinks = t.sinks;
      s.sink_blocks = t.sink_blocks;
      s.k0 = k;
      s.nb = nb;
      s.blocks = t.blocks;
      s.first_cta = blockIdx.x;
      s.pieces = 1;
      // keys up to p_first that the table holds are seen by every token; the window's lower edge
      // crosses the blocks from lo's to the one of the last token's first key
      const int b0 = t.lo / kBlock;
      s.trail = t.p_first < 0 ? 0 : t.sink_blocks + max(0, (min(t.p_first, p.cap - 1) + 1) / kBlock - b0);
      s.lead = p.window > 0 && t.p_end >= p.window
                   ? t.sink_blocks + (t.p_end - p.window) / kBlock + 1 - b0
                   : 0;
      if (nb < t.blocks) {
        // position y belongs to CTA ((y + 1) ctas - 1) / total
        const long long x1 = x0 + t.blocks;
        s.first_cta = (int)quotient((x0 + 1) * st.ctas - 1, st.total);
        s.pieces = (int)quotient(x1 * st.ctas - 1, st.total) - s.first_cta + 1;
      }
      *seg = s;
      st.unit += t.cost();
      if (++st.tile == n_tiles(p, r)) {
        st.tile = 0;
        if (++st.g == p.Hkv) {
          st.g = 0;
          next_request = st.unit + kUnitCost < st.end;   // nobody asks for it once the share is used up
        }
      }
    }
    mbar_arrive(smem_u32(&sm.full[slot]));
  }
  __syncwarp();
  if (__shfl_sync(0xffffffffu, (int)next_request, 0)) {   // the next request with a token
    int b = st.b + 1;
    for (;;) {
      const int base = sm.base;
      const unsigned live = __ballot_sync(0xffffffffu, base + lane >= b && sm.held[lane].n > 0);
      if (live) {
        b = base + __ffs(live) - 1;
        break;
      }
      b = next_growing(p, base + 32, lane);
      if (b >= p.B) break;
      hold_requests(p, sm, b, lane);
    }
    __syncwarp();
    if (lane == 0) st.b = b;
    __syncwarp();
  }
  return seg;
}

// A role's reader of the ring: take() copies the next piece (false: give up);
// one lane of each role must be counted in the ring's `empty` barriers.
struct SegReader {
  uint32_t n = 0;
  __device__ __forceinline__ bool take(const Params& p, SchedSmem& sm, volatile int* abort, Seg& s) {
    const int slot = n % kSegRing;
    if (!KS_PAGED_WAIT(sm.full[slot], (n / kSegRing) & 1)) return false;
    const uint4* src = reinterpret_cast<const uint4*>(&sm.seg[slot]);
    uint4* dst = reinterpret_cast<uint4*>(&s);
#pragma unroll
    for (int i = 0; i < 4; ++i) dst[i] = src[i];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&sm.empty[slot]));
    ++n;
    return true;
  }
  // The piece in place, for roles without registers to spare; release() gives it back.
  __device__ __forceinline__ const Seg* peek(const Params& p, SchedSmem& sm, volatile int* abort) {
    const int slot = n % kSegRing;
    return KS_PAGED_WAIT(sm.full[slot], (n / kSegRing) & 1) ? &sm.seg[slot] : nullptr;
  }
  __device__ __forceinline__ void release(SchedSmem& sm) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&sm.empty[n % kSegRing]));
    ++n;
  }
};

// Where the boxes of a piece's key blocks lie in the pool.  A block has n boxes
// (each inside one page); lane l looks up box l % n of block i + l / n, so one fetch
// serves 32 / n blocks, and it is asked for that long before its use: under load a
// table entry takes microseconds to come.  A box that no token of the tile sees and
// a page that is none give a row past the pool, where the tensor map reads zeros
// without touching memory.
struct BoxRows {
  int page, in_page;                           // of the fetch under way; in_page < 0: unseen
  int rows;                                    // first pool row of the lane's box, after use()
  __device__ __forceinline__ void fetch(const Params& p, const Seg& s, int i, int lane) {
    i += lane >> p.log2_boxes;
    in_page = -1;
    if (i >= s.nb) return;
    const int j0 = s.key_block(i) * kBlock + (lane & ((1 << p.log2_boxes) - 1)) * p.box;
    if (s.unseen(j0, j0 + p.box - 1)) return;
    const int blk = j0 / p.page_size;          // a key that is seen lies inside the table's row
    in_page = j0 - blk * p.page_size;
    page = p.table[(long long)s.b * p.max_blocks + blk];
  }
  __device__ __forceinline__ void use(const Params& p) {
    rows = p.n_slots;
    if (in_page < 0) return;
    if ((unsigned)page < (unsigned)p.n_pages) rows = page * p.page_size + in_page;
    else raise_status(p.status, KS_ERR_INVALID_ARG);
  }
};

// One warp that loads the share's K blocks (and walks it) or its V blocks into a
// ring; lane l loads the box l % 16 of panel l / 16.  on_piece(s), K only: before a
// piece's first block; false gives up.
struct Ring {
  const CUtensorMap* tm;
  uint64_t *full, *empty;
  uint32_t base;                               // shared address of slot 0
  int slots, stride;
};
template <int HD, typename F>
__device__ __forceinline__ void load_share(const Params& p, SchedSmem& sm, const Ring& r, bool is_k,
                                           volatile int* abort, F&& on_piece) {
  constexpr int PANELS = HD / 64;
  const int lane = threadIdx.x & 31, lb = p.log2_boxes, per = 32 >> lb;
  const bool mine = (lane & 15) >> lb == 0 && (lane >> 4) < PANELS;
  const uint32_t box_off = r.base + (lane >> 4) * (kBlock * 128) + (lane & 15) * p.box * 128;
  SegReader rd;
  int slot = 0, n_loads = 0;
  uint32_t phase = 1;
  BoxRows at;
  const Seg* s = is_k ? walk(p, sm, abort) : rd.peek(p, sm, abort);
  if (s && s->nb > 0) at.fetch(p, *s, 0, lane);
  while (s && s->nb > 0) {
    if (is_k && !on_piece(*s)) break;
    const Seg* following = nullptr;
    const int nb = s->nb, x = s->g * HD + (lane >> 4) * 64;
    int i = 0;
    do {
      at.use(p);
      const int m = min(per, nb - i);
      if (i + m < nb) at.fetch(p, *s, i + m, lane);
      int e = 0;
      for (; e < m; ++e) {
        if (!KS_PAGED_WAIT(r.empty[slot], phase)) break;
        const uint32_t fb = smem_u32(&r.full[slot]);
        const int row = __shfl_sync(0xffffffffu, at.rows, (e << lb) + (lane & ((1 << lb) - 1)));
        if (lane == 0) mbar_arrive_expect_tx(fb, PANELS * kBlock * 128);
        __syncwarp();
        if (mine) tma_load_2d(box_off + slot * r.stride, r.tm, x, row, fb);
        ++n_loads;
        if (++slot == r.slots) {
          slot = 0;
          phase ^= 1;
        }
      }
      if (e < m) break;
      i += m;
    } while (i < nb);
    if (i < nb) break;
    if (!is_k) rd.release(sm);
    following = is_k ? walk(p, sm, abort) : rd.peek(p, sm, abort);
    if (following && following->nb > 0) at.fetch(p, *following, 0, lane);
    s = following;
  }
  // wait for the copies still in flight before leaving
  if (lane == 0)
    for (int n = n_loads > r.slots ? n_loads - r.slots : 0; n < n_loads; ++n)
      mbar_wait_drain(smem_u32(&r.full[n % r.slots]), (uint32_t)(n / r.slots) & 1, p.status);
}

// Zeroes the rows of a V block that no token of the tile sees (their weights are
// zero, but zero times what the page holds there need not be); one warp.  Boxes of
// which nothing is seen hold zeros already, so what is left lies behind the last
// seen key in its box, and at either end of the gap between sinks and window.
template <int PANELS>
__device__ __forceinline__ void zero_rows(unsigned char* v, int from, int to, int lane) {
  for (int r = from + (lane >> 3); r < to; r += 4)
#pragma unroll
    for (int pn = 0; pn < PANELS; ++pn)
      *reinterpret_cast<uint4*>(v + pn * kBlock * 128 + r * 128 + (lane & 7) * 16) =
          make_uint4(0, 0, 0, 0);
}
template <int PANELS>
__device__ __forceinline__ void zero_unseen(const Params& p, const Seg& s, int kb, unsigned char* v,
                                            int lane) {
  const int j0 = kb * kBlock, up = p.box - 1;
  const int tail = max(0, min(kBlock, s.last_key + 1 - j0));
  zero_rows<PANELS>(v, tail, min(kBlock, (tail + up) & ~up), lane);
  const int g0 = max(0, min(kBlock, s.sinks - j0)), g1 = max(0, min(kBlock, s.lo - j0));
  if (g0 < g1) {                               // the gap [g0, g1)
    zero_rows<PANELS>(v, g0, min(g1, (g0 + up) & ~up), lane);
    zero_rows<PANELS>(v, max(g0, g1 & ~up), g1, lane);
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
}

__device__ __forceinline__ unsigned char* piece(const Params& p, int cta, int second) {
  return p.ws + kCounterBytes + (size_t)(2 * cta + second) * kPieceBytes;
}
// The piece that this CTA leaves for a segment, and the one that CTA `cta` left.
__device__ __forceinline__ unsigned char* own_piece(const Params& p, const Seg& s) {
  return piece(p, blockIdx.x, s.k0 == 0);
}

// One thread, after the CTA's writers of the piece have met (its fence then covers
// their stores too): true for the unit's last arrival.  The counter is zero again
// afterwards.  The readers of the pieces meet it again before they read.  A counter that
// did not start out zero is reported by the first arrival that finds it.
__device__ __forceinline__ bool arrive_piece(const Params& p, const Seg& s) {
  uint32_t* counter = reinterpret_cast<uint32_t*>(p.ws) + s.first_cta;
  __threadfence();
  const uint32_t before = atomicAdd(counter, kArrival) * kArrivalInv, pieces = s.pieces;
  if (before >= pieces) raise_status(p.status, KS_ERR_WORKSPACE);
  const bool last = before == pieces - 1;
  if (last) *counter = 0;
  __threadfence();
  return last;
}

// Joins a unit's pieces: with M the largest reference of a row,
//   out = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s, pieces in order.
// Nothing here depends on bytes, only on how many loads a warp keeps in flight: few rows go one
// to a warp with 8 pieces at a time (19 pieces of 4 rows: 12 us one piece at a time), many rows 8
// to a warp (2 pieces of 128 rows: 60 us one row at a time).
constexpr int kJoinBatch = 8;

template <int HD>
__device__ __forceinline__ void store_row(const Params& p, const Seg& s, int r, int lane,
                                          const float* acc, float f) {
  constexpr int E = HD / 32;
  const int t = r / p.grp;
  __nv_bfloat16* dst =
      p.out + ((long long)(s.row0 + t) * p.Hq + s.g * p.grp + (r - t * p.grp)) * HD + lane * E;
  uint32_t o[E / 2];
#pragma unroll
  for (int e = 0; e < E / 2; ++e) o[e] = pack2(acc[2 * e] * f, acc[2 * e + 1] * f);
  if (E == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(o[0], o[E / 2 - 1]);
  else *reinterpret_cast<uint32_t*>(dst) = o[0];
}

template <int HD>
__device__ __forceinline__ void join_pieces(const Params& p, const Seg& s, int warp, int n_warps,
                                            int lane) {
  constexpr int E = HD / 32, NB = kJoinBatch;
  const int rows = s.tokens * p.grp, n = s.pieces;
  const size_t next = 2 * kPieceBytes;         // from a piece to the unit's next one, after the first
  const unsigned char* first = piece(p, s.first_cta, 1);
  const unsigned char* rest = piece(p, s.first_cta, 0);   // + i * next, i >= 1
  auto stats = [&](int i, int r) {
    return __ldcg(reinterpret_cast<const float2*>(i ? rest + i * next : first) + r);
  };
  auto load = [&](int i, int r, float* v) {
    const float* src =
        reinterpret_cast<const float*>((i ? rest + i * next : first) + kPieceStats) + r * HD + lane * E;
    if (E == 4) *reinterpret_cast<float4*>(v) = __ldcg(reinterpret_cast<const float4*>(src));
    else *reinterpret_cast<float2*>(v) = __ldcg(reinterpret_cast<const float2*>(src));
  };
  alignas(16) float v[NB][E];
  if (rows <= 2 * n_warps) {
    for (int r = warp; r < rows; r += n_warps) {
      float M = kNoRef, L = 0.f, acc[E] = {};
      for (int i = lane; i < n; i += 32) M = fmaxf(M, stats(i, r).x);
#pragma unroll
      for (int d = 16; d; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
#pragma unroll 1
      for (int i0 = 0; i0 < n; i0 += NB) {
        const bool on = lane < NB && i0 + lane < n;
        const float2 ml = stats(min(i0 + (lane & (NB - 1)), n - 1), r);
#pragma unroll
        for (int k = 0; k < NB; ++k) load(min(i0 + k, n - 1), r, v[k]);
        const float w = on ? ex2(ml.x - M) : 0.f, wl = w * ml.y;
#pragma unroll
        for (int k = 0; k < NB; ++k) {
          const float wk = __shfl_sync(0xffffffffu, w, k);
          L += __shfl_sync(0xffffffffu, wl, k);
          if (i0 + k < n)
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] += wk * v[k][e];
        }
      }
      store_row<HD>(p, s, r, lane, acc, L > 0.f ? 1.0f / L : 0.f);
    }
    return;
  }
  for (int r0 = warp * NB; r0 < rows; r0 += n_warps * NB) {
    // lane l: row r0 + l % 8 of pieces l / 8, l / 8 + 4, ...
    const int row = min(r0 + (lane & (NB - 1)), rows - 1);
    float M = kNoRef, L = 0.f, acc[NB][E] = {};
    for (int i = lane >> 3; i < n; i += 4) M = fmaxf(M, stats(i, row).x);
    M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 8));
    M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 16));
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const float2 ml = stats(i, row);
#pragma unroll
      for (int k = 0; k < NB; ++k) load(i, min(r0 + k, rows - 1), v[k]);
      const float w = ex2(ml.x - M);
      L += w * ml.y;
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const float wk = __shfl_sync(0xffffffffu, w, k);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[k][e] += wk * v[k][e];
      }
    }
    const float inv = L > 0.f ? 1.0f / L : 0.f;
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const float f = __shfl_sync(0xffffffffu, inv, k);
      if (r0 + k < rows) store_row<HD>(p, s, r0 + k, lane, acc[k], f);
    }
  }
}

}  // namespace paged

// Every request's new tokens in one tile of at most 64 rows.
ks_status launch_paged_decode(const PagedAttnArgs& a, paged::Params p, int grid, cudaStream_t st);
// Any step, in tiles of at most 128 rows.
ks_status launch_paged_chunk(const PagedAttnArgs& a, const paged::Params& p, int grid,
                             cudaStream_t st);

}  // namespace ks
