"""ks_page_plan against a token-by-token layout (whole numbers: equal), its
errors, and the rotary append (ks_rope_append_bf16) against fp64."""
import pytest
import torch

from knapsack_layer_selection_b200 import binding as B
from knapsack_layer_selection_b200 import build as BUILD
from tests import _paged as P

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    BUILD.build()
    return B.load()


class Outs:
    def __init__(self, L, cap):
        z = lambda n: torch.full((n,), -99, dtype=I32, device="cuda")
        self.cu, self.kv, self.pos, self.slots, self.taken = z(L.B + 1), z(L.B), z(cap), z(cap), z(1)
        self.status = torch.zeros(1, dtype=I32, device="cuda")


def _plan(L, cap, o=None, table=None, n_pages=None, free=None):
    o = o or Outs(L, cap)
    table = L.table.clone() if table is None else table
    B.page_plan(L.ctx_len, L.new_len, L.free if free is None else free, table, L.page,
                L.n_pages if n_pages is None else n_pages, o.cu, o.kv, o.pos, o.slots, o.taken,
                o.status)
    return o, table


def _ragged(n, hi_ctx, hi_new, seed):
    g = torch.Generator().manual_seed(seed)
    c = torch.randint(0, hi_ctx + 1, (n,), generator=g).tolist()
    w = torch.randint(0, hi_new + 1, (n,), generator=g).tolist()
    return list(zip(c, w))


CASES = [([], 8, 0), ([(0, 0)], 8, 0), ([(0, 1)], 8, 0), ([(7, 1), (8, 1), (9, 1), (16, 17)], 8, 3),
         ([(5, 0), (0, 0), (15, 1), (0, 0)], 16, 40), ([(31, 2), (32, 0), (0, 100)], 48, 0),
         (_ragged(513, 300, 11, 1), 16, 7), (_ragged(1025, 5000, 3, 2), 128, 1),
         (_ragged(3, 40, 9000, 3), 64, 100), (_ragged(16384, 64, 2, 4), 8, 0)]


@pytest.mark.parametrize("lens,page,pad", CASES, ids=lambda x: str(len(x)) if isinstance(x, list) else None)
def test_plan_equals_a_token_by_token_layout(lens, page, pad):
    L = P.Layout(lens, page, full=False)
    cap = L.n_tokens + pad
    o, table = _plan(L, cap)
    rt, cu, kv, pos, slots, used = P.plan_reference(L, cap)
    assert table.tolist() == rt and o.cu.tolist() == cu and o.kv.tolist() == kv
    assert o.pos.tolist() == pos and o.slots.tolist() == slots and o.taken.tolist() == [used]
    assert o.status.item() == 0
    # the same lengths again: the same plan over the updated table
    o2, table2 = _plan(L, cap, table=table.clone())
    assert torch.equal(table2, table) and torch.equal(o2.slots, o.slots)


@pytest.mark.parametrize("what,code", [("negative", 1), ("negative_new", 1), ("long", 1), ("tokens", 1),
                                       ("pages", 2 + 1), ("huge", 1)])
def test_plan_errors_leave_an_empty_step(what, code):
    lens = _ragged(40, 100, 9, 5)
    L = P.Layout(lens, 16, full=False)
    cap, free = L.n_tokens, L.free
    if what == "negative":
        L.ctx_len[3] = -1
    elif what == "negative_new":
        L.new_len[39] = -5
    elif what == "long":
        L.ctx_len[0] = L.max_blocks * 16 + 1
    elif what == "huge":                       # the sum passes 32 bits
        L.ctx_len.fill_(2 ** 31 - 1)
        L.new_len.fill_(2 ** 31 - 1)
    elif what == "tokens":
        cap -= 1
    else:
        used = P.plan_reference(L, cap)[-1]
        free = L.free[: used - 1].contiguous()
    before = L.table.clone()
    o, table = _plan(L, cap, free=free)
    assert o.status.item() == code
    assert torch.equal(table, before)
    assert not o.cu.any() and not o.kv.any() and o.taken.item() == 0
    assert (o.pos == -1).all() and (o.slots == -1).all()


def test_plan_marks_pages_outside_the_pool():
    L = P.Layout([(16, 1), (3, 2), (0, 20), (40, 0)], 16, full=False)
    L.table[3, 0] = 1 << 30                    # not touched by this step: not looked at
    ref = P.plan_reference(L, L.n_tokens)
    free = L.free.clone()
    free[0] = L.n_pages                        # request 0's new page
    table = L.table.clone()
    table[1, 0] = -4                           # request 1 continues in a page that is none
    o, table = _plan(L, L.n_tokens, table=table, free=free)
    assert o.status.item() == 1
    assert o.pos.tolist() == ref[3]
    assert o.slots.tolist() == [-1, -1, -1] + ref[4][3:]
    assert table[0, 1].item() == -1 and table[3, 0].item() == 1 << 30


APPEND = [(1, (4, 4, 64), 8), (5, (8, 1, 128), 48), (257, (12, 4, 128), 16), (33, (16, 4, 64), 64),
          (1000, (32, 8, 128), 128), (3, (1, 1, 64), 16)]


def _append_case(n, heads, page, seed=0, fused=True):
    Hq, Hkv, hd = heads
    g = torch.Generator(device="cuda").manual_seed(seed)
    n_pages = P.ceil(n, page) + 3
    qkv = torch.randn(n, Hq + 2 * Hkv, hd, generator=g, device="cuda").to(P.BF16)
    pos = torch.randint(0, 200000, (n,), generator=g, device="cuda", dtype=I32)
    slots = torch.randperm(n_pages * page, generator=g, device="cuda")[:n].to(I32)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    pools = [torch.full((n_pages, page, Hkv, hd), 7.0, dtype=P.BF16, device="cuda") for _ in range(2)]
    return q, k, v, pos, slots, pools


def _check_append(q, k, v, pos, slots, pools, q_out, base, live=None):
    Hkv, hd = k.shape[1:]
    n_slots = pools[0].numel() // (Hkv * hd)
    keep = torch.ones(len(pos), dtype=torch.bool, device="cuda") if live is None else live
    cached = keep & (slots >= 0) & (slots < n_slots)
    p = pos.long()
    if q_out is not None:
        ref = P.rope_reference(q[keep], p[keep], base)
        err = (q_out[keep].double() - ref).abs()
        assert (err <= P.rope_tolerance(q[keep], ref, p[keep])).all()
    kf, vf = pools[0].view(-1, Hkv, hd), pools[1].view(-1, Hkv, hd)
    w = slots[cached].long()
    ref = P.rope_reference(k[cached], p[cached], base)
    assert ((kf[w].double() - ref).abs() <= P.rope_tolerance(k[cached], ref, p[cached])).all()
    assert torch.equal(vf[w], v[cached])
    rest = torch.ones(n_slots, dtype=torch.bool, device="cuda")
    rest[w] = False
    assert (kf[rest] == 7).all() and (vf[rest] == 7).all()


@pytest.mark.parametrize("fused", [True, False])
@pytest.mark.parametrize("n,heads,page", APPEND)
def test_append_rotates_and_stores(n, heads, page, fused):
    q, k, v, pos, slots, pools = _append_case(n, heads, page, n, fused)
    st = torch.zeros(1, dtype=I32, device="cuda")
    q_out = torch.empty(q.shape, dtype=P.BF16, device="cuda")
    B.rope_append_bf16(q, k, v, pos, slots, *pools, 500000.0, q_out, st)
    _check_append(q, k, v, pos, slots, pools, q_out, 500000.0)
    assert st.item() == 0


def test_append_padding_uncached_and_foreign_slots():
    q, k, v, pos, slots, pools = _append_case(50, (8, 2, 128), 16)
    pos[40:] = -1                              # padding: not even its query is written
    slots[40:45] = -1
    slots[3], slots[7] = -1, -77               # not cached, query still rotated
    slots[11] = pools[0].shape[0] * 16         # one past the pool
    slots[12] = 2 ** 31 - 1
    st = torch.zeros(1, dtype=I32, device="cuda")
    q_out = torch.full(q.shape, 5.0, dtype=P.BF16, device="cuda")
    B.rope_append_bf16(q, k, v, pos, slots, *pools, 1e4, q_out, st)
    _check_append(q, k, v, pos, slots, pools, q_out, 1e4, live=pos >= 0)
    assert (q_out[40:] == 5).all() and st.item() == 1


def test_append_far_positions_and_position_zero():
    q, k, v, pos, slots, pools = _append_case(40, (4, 2, 64), 16)
    pos[:8] = torch.tensor([0, 1, 2 ** 24 + 1, 2 ** 27 + 5, 2 ** 30, 2 ** 31 - 256, 65536, 131071],
                           dtype=I32, device="cuda")
    q_out = torch.empty(q.shape, dtype=P.BF16, device="cuda")
    B.rope_append_bf16(q, k, v, pos, slots, *pools, 1e6, q_out)
    _check_append(q, k, v, pos, slots, pools, q_out, 1e6)
    assert torch.equal(q_out[0], q[0])         # position 0 turns nothing


def test_append_in_place_without_queries_and_without_tokens():
    q, k, v, pos, slots, pools = _append_case(70, (8, 2, 64), 24, fused=False)
    q0 = q.clone()
    B.rope_append_bf16(q, k, v, pos, slots, *pools, 1e4, q)
    _check_append(q0, k, v, pos, slots, pools, q, 1e4)
    again = [torch.full_like(p, 7.0) for p in pools]
    B.rope_append_bf16(None, k, v, pos, slots, *again, 1e4, None)
    assert torch.equal(again[0], pools[0]) and torch.equal(again[1], pools[1])
    none = [torch.full_like(p, 7.0) for p in pools]
    B.rope_append_bf16(q[:0], k[:0], v[:0], pos[:0], slots[:0], *none, 1e4, q[:0])
    assert (none[0] == 7).all()


def test_append_into_a_pool_past_32_bit_offsets():
    """A pool of more than 2^31 elements (4.3 GB): the last slots are its own."""
    Hkv, hd, page = 8, 128, 64
    n_pages = (1 << 31) // (page * Hkv * hd) + 2
    kp = torch.empty(n_pages, page, Hkv, hd, dtype=P.BF16, device="cuda")
    vp = torch.empty_like(kp)
    kp[-2:].fill_(7.0)
    vp[-2:].fill_(7.0)
    _, k, v, pos, _, _ = _append_case(9, (8, Hkv, hd), page)
    slots = (n_pages * page - 1 - 7 * torch.arange(9, device="cuda")).to(I32)
    st = torch.zeros(1, dtype=I32, device="cuda")
    B.rope_append_bf16(None, k, v, pos, slots, kp, vp, 5e5, None, st)
    _check_append(None, k, v, pos, slots - (n_pages - 2) * page, [kp[-2:], vp[-2:]], None, 5e5)
    assert st.item() == 0
