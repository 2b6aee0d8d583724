"""Paged-cache test helpers: random layouts, and the operators in 64 bits from
their definitions (plain torch, no code shared with the library)."""
import math

import torch

BF16 = torch.bfloat16
HALF_STEP = torch.finfo(BF16).eps / 2          # a bf16 rounding, relative to the value


def ceil(a, b):
    return -(-a // b)


class Layout:
    """Requests [(ctx, new)], their pages scattered over a pool; entries past a
    request's pages hold -1.  full: the table already holds the new tokens'
    pages, else they are at the front of `free`."""

    def __init__(self, lens, page, full=True, extra_blocks=1, spare=5, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.page, self.device = list(lens), page, device
        self.ctx = [c for c, _ in lens]
        self.new = [n for _, n in lens]
        self.kv = [c + n for c, n in lens]
        self.B, self.n_tokens = len(lens), sum(self.new)
        self.max_new = max(self.new + [1])
        need = [ceil(k if full else c, page) for k, c in zip(self.kv, self.ctx)]
        self.max_blocks = max([ceil(k, page) for k in self.kv] + [0]) + extra_blocks
        self.n_pages = sum(ceil(k, page) for k in self.kv) + spare
        order = torch.randperm(self.n_pages, generator=g).tolist()
        self.rows = []
        for n in need:
            self.rows.append(order[:n] + [-1] * (self.max_blocks - n))
            order = order[n:]
        self.free_list = order
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=device)
        self.table = i32(self.rows).reshape(self.B, self.max_blocks)
        self.free = i32(order)
        self.ctx_len, self.new_len, self.kv_len = i32(self.ctx), i32(self.new), i32(self.kv)
        cu = [0]
        for n in self.new:
            cu.append(cu[-1] + n)
        self.cu_list, self.cu = cu, i32(cu)

    def pool(self, Hkv, hd, fill=None, seed=1):
        g = torch.Generator(device=self.device).manual_seed(seed)
        shape = (self.n_pages, self.page, Hkv, hd)
        if fill is not None:
            return torch.full(shape, fill, dtype=BF16, device=self.device)
        return torch.randn(shape, generator=g, device=self.device).to(BF16)


def plan_reference(L, cap):
    """(table, cu, kv_len, positions, slots, n_taken) token by token."""
    table, used = [list(r) for r in L.rows], 0
    pos, slots = [], []
    for b, (c, n) in enumerate(L.lens):
        for p in range(c, c + n):
            if p % L.page == 0:
                table[b][p // L.page] = L.free_list[used]
                used += 1
            pos.append(p)
            slots.append(table[b][p // L.page] * L.page + p % L.page)
    pad = [-1] * (cap - len(pos))
    return table, L.cu_list, L.kv, pos + pad, slots + pad, used


def rope_reference(x, pos, base):
    """Rotate-half RoPE of x [n][H][hd] at pos [n], fp64."""
    hd = x.shape[-1]
    j = torch.arange(hd // 2, dtype=torch.float64, device=x.device)
    a = pos.double()[:, None, None] * (float(base) ** (-2.0 * j / hd))
    x0, x1 = x.double()[..., : hd // 2], x.double()[..., hd // 2:]
    return torch.cat((x0 * a.cos() - x1 * a.sin(), x1 * a.cos() + x0 * a.sin()), -1)


def rope_tolerance(x, ref, pos):
    """One bf16 rounding of the result; the pair's rotation in fp32 (two
    products, a sum, sine and cosine of a reduced angle: under 2^-20 of the
    pair's size in all) and the angle's own error in fp64, a few 2^-53 of it."""
    hd = x.shape[-1]
    pair = x.double()[..., : hd // 2].abs() + x.double()[..., hd // 2:].abs()
    pair = torch.cat((pair, pair), -1)
    return ref.abs() * HALF_STEP + pair * (2.0 ** -20 + pos.double()[:, None, None] * 2.0 ** -50)


def attention_reference(L, q, k_pages, v_pages, window=0, sinks=0, kv=None):
    """(out, tolerance), both fp64 [n_tokens][Hq][hd]; kv overrides the lengths.

    Tolerance: one bf16 rounding of the result, and one of each probability p
    before the product with V.  With p~ = p (1 + d), |d| <= e, and the same p~
    in the row sum, the result moves by at most e / (1 - e) sum_j w_j |v_j - o|
    <= e / (1 - e) (sum_j w_j |v_j| + |o|).  e is the half step plus what fp32
    leaves: a score's error, hd 2^-23 sum|q k| / sqrt(hd) for any order of the
    sum, and 2^-18 for the exponential of a score below 64 in size."""
    hd, Hq = q.shape[-1], q.shape[1]
    Hkv = k_pages.shape[2]
    out, tol = [], []
    for b in range(L.B):
        n = L.new[b]
        S = L.kv[b] if kv is None else kv[b]
        ids = torch.tensor(L.rows[b][: ceil(max(S, 0), L.page)], device=q.device, dtype=torch.long)
        k = k_pages[ids].flatten(0, 1)[: max(S, 0)].double()
        v = v_pages[ids].flatten(0, 1)[: max(S, 0)].double()
        qq = q[L.cu_list[b]: L.cu_list[b] + n].double()
        p = torch.arange(S - n, S, device=q.device)[:, None]
        j = torch.arange(max(S, 0), device=q.device)[None, :]
        seen = j <= p
        if window:
            seen = seen & ((j > p - window) | (j < sinks))
        if S > 0:                              # what nobody sees has no value
            dead = ~seen.any(0)
            k, v = k.clone(), v.clone()
            k[dead] = 0
            v[dead] = 0
        for h in range(Hq):
            kh, vh = k[:, h // (Hq // Hkv)], v[:, h // (Hq // Hkv)]
            s = (qq[:, h] @ kh.T) / math.sqrt(hd)
            s = s.masked_fill(~seen, -math.inf)
            m = s.amax(-1, keepdim=True) if S > 0 else s.new_zeros(n, 1)
            m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
            w = (s - m).exp()
            w = w / w.sum(-1, keepdim=True).clamp(min=1e-300)
            o = w @ vh
            e = HALF_STEP + 2.0 ** -18
            if S > 0:
                big = (qq[:, h].abs() @ kh.abs().T).masked_fill(~seen, 0).amax(-1, keepdim=True)
                e = e + hd * 2.0 ** -23 * big / math.sqrt(hd)
            out.append(o)
            tol.append(HALF_STEP * o.abs() * (1 + 2 * HALF_STEP)
                       + e / (1 - e) * (w @ vh.abs() + o.abs()) + 1e-30)
    split = lambda xs: torch.cat([torch.stack(xs[i * Hq:(i + 1) * Hq], 1) for i in range(L.B)])
    return split(out), split(tol)
