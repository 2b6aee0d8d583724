"""The paged key/value cache of a draft-and-verify loop: three operators and their plain forms.

* plan:   block tables, slots and positions of the next tokens, from the requests' lengths
          (``binding.page_plan``);
* append: rotary positions on the new tokens' queries and keys, and the keys and values
          written into their pages (``binding.rope_append_bf16``);
* attend: causal grouped-query attention of a chunk of new tokens over the paged cache, with an
          optional sliding window and first tokens that stay visible
          (``binding.paged_attention_bf16``).

``own`` selects what ``run`` does: False computes the plain form with elementary torch
operations, True calls the library.
"""
import math
import random

import torch

own = False

# (query heads, key/value heads, head dim): the repository's workloads (small, 8B and 32B shapes),
# and generic ones: no sharing, all heads shared, a group that does not divide a tile
HEADS = ((16, 4, 64), (32, 8, 128), (64, 8, 128), (4, 4, 64), (8, 1, 128), (12, 4, 128))


def _case(name, kind, B, ctx, new, heads=(32, 8, 128), page=16, window=0, sinks=0):
    """B requests with ctx[0] .. ctx[1] cached tokens and new[0] .. new[1] new ones each."""
    return {"name": name, "kind": kind, "B": B, "ctx_lo": ctx[0], "ctx_hi": ctx[1],
            "new_lo": new[0], "new_hi": new[1], "Hq": heads[0], "Hkv": heads[1], "hd": heads[2],
            "page": page, "window": window, "sinks": sinks}


def listed():
    return [
        # a verification step of 64 requests: 1 .. 11 tokens each (a draft of up to 10 and its root)
        _case("plan_verify_64", "plan", 64, (0, 8192), (1, 11)),
        # a step that mixes decoding requests, idle ones and prompt chunks
        _case("plan_mixed_301", "plan", 301, (0, 32768), (0, 255), page=64),
        # one draft token of 32 requests: latency counts
        _case("append_draft_32", "append", 32, (100, 8192), (1, 1)),
        # a verification step in the small model's heads, pages that do not divide 128
        _case("append_verify_small_heads", "append", 61, (0, 2048), (1, 9), (16, 4, 64), 48),
        # prompt chunks: the bandwidth-bound end
        _case("append_chunks", "append", 5, (0, 32768), (1500, 2047), page=64),
        # one request, one token, a short context: the smallest call
        _case("attend_draft_single", "attend", 1, (700, 1100), (1, 1), (16, 4, 64)),
        # batched drafting: one token each over ragged contexts
        _case("attend_draft_64", "attend", 64, (200, 8192), (1, 1)),
        # one request with a long context: the keys have to be split over the GPU
        _case("attend_draft_long", "attend", 1, (120000, 131000), (1, 1), page=64),
        # verification of drafts of up to 10 tokens
        _case("attend_verify_32", "attend", 32, (500, 8192), (1, 11), page=32),
        # verification with 64 query heads (8 to a key head): 72 rows per key head
        _case("attend_verify_wide", "attend", 8, (9000, 16384), (9, 9), (64, 8, 128)),
        # prompt chunks over a long context: the matrix units bound it
        _case("attend_chunks", "attend", 2, (6000, 8192), (1900, 2047), page=64),
        # cheap drafting over long contexts: a window of 1,024 keys and 4 first tokens
        _case("attend_window_48", "attend", 48, (3000, 32768), (1, 6), window=1024, sinks=4),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(("plan", "append", "append", "attend", "attend", "attend", "attend"))
    heads = rng.choice(HEADS)
    page = rng.choice((16, 32, 48, 64, 128))
    if kind == "plan":
        B = _log_int(rng, 1, 512)
        return _strip(_case("", kind, B, (0, _log_int(rng, 64, 32768)),
                            (rng.randint(0, 1), _log_int(rng, 1, max(1, 40000 // B))), page=page))
    if kind == "append":
        B = _log_int(rng, 1, 128)
        hi = _log_int(rng, 1, max(1, 10000 // B))
        return _strip(_case("", kind, B, (0, _log_int(rng, 64, 32768)), (rng.randint(1, hi), hi),
                            heads, page))
    what = rng.choice(("draft", "verify", "chunk"))
    if what == "chunk":
        B = rng.randint(1, 4)
        hi = _log_int(rng, 12, 2047 // B)
        ctx = _log_int(rng, 64, 16384)
        new = (rng.randint(1, hi), hi)
    else:
        B = _log_int(rng, 1, 96)
        # at most about 400,000 cached tokens in all
        ctx = _log_int(rng, 64, min(65536, 400000 // B))
        new = (1, 1) if what == "draft" else (1, rng.randint(2, 11))
    win = rng.random() < 0.35
    return _strip(_case("", kind, B, (rng.randint(1, ctx), ctx), new, heads, page,
                        _log_int(rng, 17, 4096) if win else 0,
                        rng.choice((0, 1, 4, 63, 130)) if win else 0))


def _strip(case):
    del case["name"]
    return case


def _lengths(case, seed=None):
    """Cached and new tokens of each request.  The case fixes the lengths (the longest context and
    the largest chunk among them); the seed gives them to the requests in another order."""
    r, B = random.Random(20), case["B"]
    pairs = [(r.randint(case["ctx_lo"], case["ctx_hi"]), r.randint(case["new_lo"], case["new_hi"]))
             for _ in range(B)]
    pairs[0] = (case["ctx_hi"], case["new_hi"])
    if seed is not None:
        random.Random(seed).shuffle(pairs)
    return [c for c, _ in pairs], [n for _, n in pairs]


def _ceil(a, b):
    return -(-a // b)


class _State:
    pass


def prepare(case, seed):
    s = _State()
    s.case, kind = case, case["kind"]
    dev = "cuda"
    ctx, new = _lengths(case, seed)
    B, ps, Hq, Hkv, hd = (case[k] for k in ("B", "page", "Hq", "Hkv", "hd"))
    kv = [c + n for c, n in zip(ctx, new)]
    s.B, s.page, s.n_tokens, s.max_new, s.max_kv = B, ps, sum(new), max(max(new), 1), max(kv)
    held = [_ceil(c, ps) for c in ctx]
    need = [_ceil(k, ps) for k in kv]
    s.max_blocks = max(max(need), 1)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    g = torch.Generator(device=dev).manual_seed(seed)
    # pages lie scattered in the pool, as after many requests have come and gone; a few are spare
    s.n_pages = sum(need) + 7
    order = torch.randperm(s.n_pages, generator=g, device=dev).to(torch.int32)
    s.ctx_len, s.new_len = i32(ctx), i32(new)
    s.status = torch.zeros(1, dtype=torch.int32, device=dev)
    full = kind != "plan"
    have = i32(need if full else held)
    start = torch.cumsum(have, 0) - have
    cols = torch.arange(s.max_blocks, device=dev)
    # entries past a request's pages hold -1
    s.table = torch.where(cols[None, :] < have[:, None],
                          order[(start[:, None] + cols[None, :]).clamp(max=s.n_pages - 1)],
                          torch.full((), -1, dtype=torch.int32, device=dev))
    if kind == "plan":
        s.free = order[sum(held):].contiguous()
        # the buffers are sized for a step's largest batch, not for this one's tokens
        s.cap = s.n_tokens + 37
        s.cu, s.kv_len = torch.empty(B + 1, dtype=torch.int32, device=dev), torch.empty_like(s.ctx_len)
        s.positions = torch.empty(s.cap, dtype=torch.int32, device=dev)
        s.slots = torch.empty(s.cap, dtype=torch.int32, device=dev)
        s.taken = torch.empty(1, dtype=torch.int32, device=dev)
        return s
    s.kv_len = i32(kv)
    s.cu = torch.zeros(B + 1, dtype=torch.int32, device=dev)
    s.cu[1:] = torch.cumsum(s.new_len, 0)
    randn = lambda *shape: torch.randn(*shape, generator=g, device=dev, dtype=torch.bfloat16)
    pool = (s.n_pages, ps, Hkv, hd)
    if kind == "append":
        # a pool as allocated, so that what comes back is what the pass wrote
        s.k_pages = torch.zeros(pool, dtype=torch.bfloat16, device=dev)
        s.v_pages = torch.zeros_like(s.k_pages)
        # one fused projection's output: queries, keys and values of a token side by side
        qkv = randn(s.n_tokens, Hq + 2 * Hkv, hd)
        s.q, s.k, s.v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s.q_out = torch.empty(s.n_tokens, Hq, hd, dtype=torch.bfloat16, device=dev)
        s.base = 500000.0
        tok = torch.arange(s.n_tokens, device=dev)
        r = torch.searchsorted(s.cu[1:].contiguous(), tok.to(torch.int32), right=True)
        pos = s.ctx_len[r] + tok - s.cu[r]
        s.positions = pos.to(torch.int32)
        s.slots = (s.table[r, pos // ps] * ps + pos % ps).to(torch.int32)
        return s
    s.k_pages, s.v_pages = randn(*pool), randn(*pool)
    s.window, s.sinks = case["window"], case["sinks"]
    s.q = randn(s.n_tokens, Hq, hd) * 1.3
    s.out = torch.empty_like(s.q)
    # scratch that a serving program keeps from step to step, zero before its first use
    s.ws = torch.zeros(20 << 20, dtype=torch.uint8, device=dev)
    return s


# ------------------------------------------------------------------ plain forms
def _plain_plan(s):
    ps, dev = s.page, s.ctx_len.device
    ctx, new = s.ctx_len.long(), s.new_len.long()
    kv = ctx + new
    held, need = (ctx + ps - 1) // ps, (kv + ps - 1) // ps
    cu = torch.zeros(s.B + 1, dtype=torch.long, device=dev)
    cu[1:] = torch.cumsum(new, 0)
    first = torch.cumsum(need - held, 0) - (need - held)      # of each request, in the free list
    col = torch.arange(s.table.shape[1], device=dev)[None, :]
    fresh = (col >= held[:, None]) & (col < need[:, None])
    take = (first[:, None] + col - held[:, None]).clamp(0, s.free.numel() - 1)
    table = torch.where(fresh, s.free[take], s.table)
    tok = torch.arange(s.cap, device=dev)
    live = tok < cu[-1]
    r = torch.searchsorted(cu[1:], tok, right=True).clamp(max=s.B - 1)
    pos = torch.where(live, ctx[r] + tok - cu[r], torch.full_like(tok, -1))
    p0 = pos.clamp(min=0)
    slot = torch.where(live, table[r, p0 // ps].long() * ps + p0 % ps, torch.full_like(tok, -1))
    return {"table": table, "cu": cu.int(), "kv_len": kv.int(), "positions": pos.int(),
            "slots": slot.int(), "taken": (need - held).sum().reshape(1).int()}


def _rotate(x, cos, sin):
    a, b = x.float().chunk(2, dim=-1)
    return torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1).to(torch.bfloat16)


def _plain_append(s):
    hd = s.q.shape[-1]
    # angles of far positions lose their fraction in 32 bits
    freq = s.base ** (-2.0 * torch.arange(hd // 2, device=s.q.device, dtype=torch.float64) / hd)
    angle = s.positions.double()[:, None, None] * freq
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    s.q_out.copy_(_rotate(s.q, cos, sin))
    where = s.slots.long()
    s.k_pages.view(-1, *s.k.shape[1:])[where] = _rotate(s.k, cos, sin)
    s.v_pages.view(-1, *s.v.shape[1:])[where] = s.v
    return {"q": s.q_out, "k_pages": s.k_pages, "v_pages": s.v_pages}


def _plain_attend(s):
    Hq, hd = s.q.shape[1:]
    Hkv, dev, ps = s.k_pages.shape[2], s.q.device, s.page
    grp, N, J = Hq // Hkv, s.max_new, s.max_kv
    key = torch.arange(J, device=dev)
    rows = (s.table[:, key // ps].clamp(min=0).long() * ps + key % ps)            # [B][J]
    k = s.k_pages.view(-1, Hkv, hd)[rows].float()                                  # [B][J][Hkv][hd]
    v = s.v_pages.view(-1, Hkv, hd)[rows].float()
    new = (s.cu[1:] - s.cu[:-1]).long()
    t = torch.arange(N, device=dev)
    tok = (s.cu[:-1].long()[:, None] + t).clamp(max=s.n_tokens - 1)               # [B][N]
    q = s.q[tok].view(s.B, N, Hkv, grp, hd).float()
    score = torch.einsum("bnghd,bjgd->bgnhj", q, k) / math.sqrt(hd)
    pos = (s.kv_len.long() - new)[:, None] + t                                     # [B][N]
    seen = key <= pos[:, :, None]
    if s.window:
        seen = seen & ((key > pos[:, :, None] - s.window) | (key < s.sinks))
    score.masked_fill_(~seen[:, None, :, None, :], float("-inf"))
    score -= score.amax(dim=-1, keepdim=True).clamp(min=-3e38)
    score.exp_()
    total = score.sum(dim=-1, keepdim=True)
    out = torch.einsum("bgnhj,bjgd->bnghd", score, v)
    out = out / total.permute(0, 2, 1, 3, 4).clamp(min=1e-30)
    live = t < new[:, None]
    return out.reshape(s.B, N, Hq, hd)[live].to(torch.bfloat16)                    # packed


# ------------------------------------------------------------------ one pass
def run(s):
    kind = s.case["kind"]
    if not own:
        return {"plan": _plain_plan, "append": _plain_append, "attend": _plain_attend}[kind](s)
    from knapsack_layer_selection_b200 import binding as B
    if kind == "plan":
        B.page_plan(s.ctx_len, s.new_len, s.free, s.table, s.page, s.n_pages, s.cu, s.kv_len,
                    s.positions, s.slots, s.taken, s.status)
        return {"table": s.table, "cu": s.cu, "kv_len": s.kv_len, "positions": s.positions,
                "slots": s.slots, "taken": s.taken}
    if kind == "append":
        B.rope_append_bf16(s.q, s.k, s.v, s.positions, s.slots, s.k_pages, s.v_pages, s.base,
                           s.q_out, s.status)
        return {"q": s.q_out, "k_pages": s.k_pages, "v_pages": s.v_pages}
    B.paged_attention_bf16(s.q, s.k_pages, s.v_pages, s.table, s.cu, s.kv_len, s.max_new, s.out,
                           s.ws, window=s.window, sinks=s.sinks, status=s.status)
    return s.out


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    Hq, Hkv, hd, ps, B = (case[k] for k in ("Hq", "Hkv", "hd", "page", "B"))
    pairs = list(zip(*_lengths(case)))
    tokens = sum(n for _, n in pairs)
    if case["kind"] == "plan":
        touched = sum(_ceil(c + n, ps) - c // ps for c, n in pairs if n)
        # lengths in; offsets and lengths out; positions and slots; a page's entry read, or taken
        # from the free list and written
        return {"bytes": 4 * (2 * B + 2 * B + 1) + 8 * (tokens + 37) + 8 * touched, "flops": 0}
    if case["kind"] == "append":
        return {"bytes": tokens * (2 * 2 * (Hq + 2 * Hkv) * hd + 8),
                "flops": tokens * 3 * (Hq + Hkv) * hd}
    w, sinks = case["window"] or 1 << 40, case["sinks"]
    seen = lambda p: p + 1 if p < w else w + min(sinks, p + 1 - w)       # by position p
    rows = sum(seen(p) for c, n in pairs for p in range(c, c + n))
    # a request's keys: those that one of its tokens sees
    keys = sum(c + n if c < w else min(c + n, w + n - 1 + sinks) for c, n in pairs)
    return {"bytes": 4 * Hkv * hd * keys + 4 * Hq * hd * tokens + 4 * keys // ps + 8 * B,
            "flops": 4 * Hq * hd * rows}


# ------------------------------------------------------------------ 64 bits, from the definitions
def exact(case, seed):
    s = prepare(case, seed)
    ctx, new = _lengths(case, seed)
    ps = case["page"]
    if case["kind"] == "plan":
        return _exact_plan(s, ctx, new, ps)
    if case["kind"] == "append":
        return _exact_append(s, case)
    return _exact_attend(s, ctx, new, case)


def _exact_plan(s, ctx, new, ps):
    table, free = s.table.cpu().tolist(), s.free.cpu().tolist()
    cu, kv, positions, slots, used = [0], [], [], [], 0
    for r, (c, n) in enumerate(zip(ctx, new)):
        for p in range(c, c + n):
            if p % ps == 0:                        # a page begins: the next free one
                table[r][p // ps] = free[used]
                used += 1
            positions.append(p)
            slots.append(table[r][p // ps] * ps + p % ps)
        cu.append(cu[-1] + n)
        kv.append(c + n)
    pad = [-1] * (s.cap - len(slots))
    i = lambda x: torch.tensor(x, dtype=torch.int32)
    return {"table": i(table), "cu": i(cu), "kv_len": i(kv), "positions": i(positions + pad),
            "slots": i(slots + pad), "taken": i([used])}


def _exact_append(s, case):
    hd, half = case["hd"], case["hd"] // 2
    j = torch.arange(half, device="cuda", dtype=torch.float64)
    theta = s.positions.to(torch.float64)[:, None] / torch.pow(torch.tensor(s.base, dtype=torch.float64,
                                                                            device="cuda"), 2 * j / hd)
    turn = torch.polar(torch.ones_like(theta), theta)[:, None, :]

    def rotated(x):                                # element i and element i + hd/2 are one complex number
        z = torch.complex(x[..., :half].double(), x[..., half:].double()) * turn
        return torch.cat((z.real, z.imag), dim=-1)

    k, v = s.k_pages.double(), s.v_pages.double()
    where = s.slots.long()
    k[where // s.page, where % s.page] = rotated(s.k)
    v[where // s.page, where % s.page] = s.v.double()
    return {"q": rotated(s.q), "k_pages": k, "v_pages": v}


def _exact_attend(s, ctx, new, case):
    Hq, Hkv, hd, ps = case["Hq"], case["Hkv"], case["hd"], case["page"]
    grp, out, at = Hq // Hkv, [], 0
    for r, (c, n) in enumerate(zip(ctx, new)):
        pages = s.table[r, :_ceil(c + n, ps)].long()
        q = s.q[at:at + n].double()
        at += n
        k = s.k_pages[pages].flatten(0, 1)[:c + n]
        v = s.v_pages[pages].flatten(0, 1)[:c + n]
        p = torch.arange(c, c + n, device="cuda")[:, None]
        j = torch.arange(c + n, device="cuda")[None, :]
        hidden = j > p
        if case["window"]:
            hidden |= (p - j >= case["window"]) & (j >= case["sinks"])
        heads = []
        for h in range(Hq):
            a = q[:, h] @ k[:, h // grp].double().T / hd ** 0.5
            a = torch.softmax(a.masked_fill(hidden, -math.inf), dim=-1)
            heads.append(a @ v[:, h // grp].double())
        out.append(torch.stack(heads, dim=1))
    return torch.cat(out)
