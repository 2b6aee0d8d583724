"""ks_page_plan_carried over many steps: pages are neither lost nor given out
twice when tokens are taken back, against a model on the host (whole numbers:
equal)."""
import pytest
import torch

from knapsack_layer_selection_b200 import binding as B
from knapsack_layer_selection_b200 import build as BUILD
from tests import _paged as P

pytestmark = pytest.mark.gpu
I32 = torch.int32
OK, INVALID, WORKSPACE = 0, 1, 3


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    BUILD.build()
    return B.load()


def _i32(x):
    return torch.tensor(x, dtype=I32, device="cuda")


class Pool:
    """Requests' tables on the device beside the same state on the host."""

    def __init__(self, n_req, page, blocks, n_pages, cap, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.n_req, self.page, self.blocks, self.n_pages, self.cap = n_req, page, blocks, n_pages, cap
        self.free = torch.randperm(n_pages, generator=g).tolist()
        self.rows = [[] for _ in range(n_req)]     # the pages of each request
        self.ctx = [0] * n_req
        self.table = torch.full((n_req, blocks), -1, dtype=I32, device="cuda")
        self.held = _i32([0] * n_req)
        self.out = [_i32([0] * n) for n in (n_req + 1, n_req, cap, cap, 1)]

    def plan(self, new, free=None, held=None, status=OK):
        st = _i32([0])
        B.page_plan(_i32(self.ctx), _i32(new), _i32(self.free) if free is None else free, self.table,
                    self.page, self.n_pages, *self.out, st, n_held=self.held if held is None else held)
        assert st.item() == status
        return [x.tolist() for x in self.out]

    def step(self, new):
        """One plan, checked against the host's; the free list is cut by what it took."""
        pos, slots, used = [], [], 0
        for b, n in enumerate(new):
            for p in range(self.ctx[b], self.ctx[b] + n):
                if p // self.page == len(self.rows[b]):
                    self.rows[b].append(self.free[used])
                    used += 1
                pos.append(p)
                slots.append(self.rows[b][p // self.page] * self.page + p % self.page)
        cu, kv, gpos, gslots, taken = self.plan(new)
        pad = [-1] * (self.cap - len(pos))
        assert cu == [sum(new[:b]) for b in range(self.n_req + 1)]
        assert kv == [c + n for c, n in zip(self.ctx, new)]
        assert gpos == pos + pad and gslots == slots + pad and taken == [used]
        self.free = self.free[used:]
        self.check()

    def check(self):
        """Every page is in the free list or in one row, and the device knows which."""
        held = self.held.tolist()
        assert held == [len(r) for r in self.rows]
        table = self.table.tolist()
        assert [t[:h] for t, h in zip(table, held)] == self.rows
        assert sorted(self.free + sum(self.rows, [])) == list(range(self.n_pages))


def test_a_rejected_draft_keeps_its_page():
    """Page 16, 15 tokens cached, five verified, one accepted: the page that the rejected ones opened is
    the next step's."""
    s = Pool(1, 16, 4, 6, 48)
    s.step([15])
    s.ctx = [15]
    s.step([5])
    s.ctx = [16]
    s.step([5])
    assert s.out[4].item() == 0 and len(s.rows[0]) == 2
    # the same lengths again: the same slots, no page
    s.step([5])
    # all rejected, back inside the first page, then far ahead
    s.ctx = [3]
    s.step([1])
    s.step([40])
    assert len(s.rows[0]) == 3


@pytest.mark.parametrize("n_req,page,steps,hi", [(1, 8, 60, 12), (7, 16, 60, 11), (40, 8, 40, 9), (600, 64, 12, 90)])
def test_pages_are_neither_lost_nor_given_twice(n_req, page, steps, hi):
    g = torch.Generator().manual_seed(n_req)
    r = lambda lo, h: int(torch.randint(lo, h + 1, (1,), generator=g))
    blocks = P.ceil(20 * hi, page) + 1
    s = Pool(n_req, page, blocks, n_req * blocks, n_req * hi + 3, seed=n_req)
    for _ in range(steps):
        new = [min(r(0, hi), blocks * page - c) for c in s.ctx]
        s.step(new)
        # part of the tokens accepted, or even cached ones taken back; some requests end
        s.ctx = [r(max(0, c - 3), c + n) for c, n in zip(s.ctx, new)]
        for b in range(n_req):
            if r(0, 14) == 0:
                s.free += s.rows[b]
                s.rows[b], s.ctx[b] = [], 0
                s.held[b] = 0
    assert any(len(x) > P.ceil(c, page) for x, c in zip(s.rows, s.ctx)) or n_req == 1


def test_without_rejections_it_is_the_plain_plan():
    L = P.Layout([(7, 1), (8, 1), (16, 17), (0, 0), (0, 40), (33, 0)], 8, full=False)
    cap = L.n_tokens + 5
    outs = []
    for held in (None, _i32([P.ceil(c, 8) for c in L.ctx])):
        o, table = [_i32([0] * n) for n in (L.B + 1, L.B, cap, cap, 1)], L.table.clone()
        B.page_plan(L.ctx_len, L.new_len, L.free, table, 8, L.n_pages, *o, n_held=held)
        outs.append([x.tolist() for x in o] + [table.tolist()])
    assert outs[0] == outs[1]
    assert held.tolist() == [P.ceil(k, 8) for k in L.kv]


@pytest.mark.parametrize("held", [[0, 2], [1, 1], [-1, 2], [1, 5], [2 ** 31 - 1, 2], [-2 ** 31, 2]])
def test_counts_that_cannot_be_leave_an_empty_step(held):
    s = Pool(2, 16, 4, 12, 48)
    s.step([10, 20])
    s.ctx = [10, 20]                               # 1 and 2 pages
    before, h = s.table.clone(), _i32(held)
    cu, kv, pos, slots, taken = s.plan([3, 3], held=h, status=INVALID)
    assert cu == [0, 0, 0] and kv == [0, 0] and taken == [0] and set(pos + slots) == {-1}
    assert torch.equal(s.table, before) and h.tolist() == held


def test_too_few_pages_leave_the_counts_as_they_were():
    s = Pool(2, 16, 4, 12, 80)
    s.step([10, 20])
    s.ctx = [10, 20]
    before = s.table.clone()
    s.plan([30, 30], free=_i32(s.free[:2]), status=WORKSPACE)      # three are wanted
    assert torch.equal(s.table, before)
    s.check()
    s.step([30, 30])
    # no page is wanted: an empty list will do
    s.ctx = [33, 20]
    s.plan([7, 0], free=_i32([]))
    assert s.out[4].item() == 0


def test_a_page_that_is_none_stays_counted():
    """Its entry is -1 and its tokens' slots are, in this step and in the next."""
    s = Pool(1, 8, 4, 6, 12)
    _, _, pos, slots, taken = s.plan([10], free=_i32([3, 6, 5]), status=INVALID)
    assert slots[:10] == [24 + i for i in range(8)] + [-1, -1] and taken == [2]
    assert s.table[0].tolist() == [3, -1, -1, -1] and s.held.item() == 2
    s.ctx = [9]
    _, _, _, slots, taken = s.plan([8], free=_i32([5]), status=INVALID)
    assert slots[:8] == [-1] * 7 + [40] and taken == [1]


def test_the_largest_batch():
    n = 16384
    s = Pool(n, 8, 2, 2 * n, n * 2)
    s.step([1] * n)
    s.ctx = [b % 2 for b in range(n)]
    s.step([1 + (b % 3 == 0) for b in range(n)])


# ------------------------------------------------------------- the free list's place on the device
class Replayed:
    """One captured step (plan, append, attention) whose free list nobody touches
    between replays, but to give a request's pages back."""

    def __init__(self, n_req, page, blocks, n_pages, cap, max_new, heads=(8, 2, 64), seed=0):
        self.Hq, self.Hkv, self.hd = heads
        self.n_req, self.page, self.blocks, self.cap = n_req, page, blocks, cap
        g = torch.Generator().manual_seed(seed)
        self.list = torch.randperm(n_pages, generator=g).tolist()
        self.start, self.rows, self.n_pages = 0, [[] for _ in range(n_req)], n_pages
        self.free, self.free_start = _i32(self.list), _i32([0])
        self.ctx, self.new, self.held = (_i32([0] * n_req) for _ in range(3))
        self.table = torch.full((n_req, blocks), -1, dtype=I32, device="cuda")
        self.out = [_i32([0] * n) for n in (n_req + 1, n_req, cap, cap, 1)]
        self.st = _i32([0])
        self.qkv = torch.zeros(cap, self.Hq + 2 * self.Hkv, self.hd, dtype=P.BF16, device="cuda")
        self.kp = torch.zeros(n_pages, page, self.Hkv, self.hd, dtype=P.BF16, device="cuda")
        self.vp = torch.zeros_like(self.kp)
        self.q_rot = torch.zeros(cap, self.Hq, self.hd, dtype=P.BF16, device="cuda")
        self.att = torch.zeros_like(self.q_rot)
        ws = B.paged_attention_workspace()
        q, k, v = self.qkv.split([self.Hq, self.Hkv, self.Hkv], 1)

        def step():
            B.page_plan(self.ctx, self.new, self.free, self.table, page, n_pages, *self.out, self.st,
                        n_held=self.held, free_start=self.free_start)
            B.rope_append_bf16(q, k, v, self.out[2], self.out[3], self.kp, self.vp, 1e4, self.q_rot, self.st)
            B.paged_attention_bf16(self.q_rot, self.kp, self.vp, self.table, self.out[0], self.out[1],
                                   max_new, self.att, ws, status=self.st)

        step()                                     # no tokens yet
        torch.cuda.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            step()

    def replay(self, ctx, new):
        self.ctx.copy_(_i32(ctx))
        self.new.copy_(_i32(new))
        self.st.zero_()
        self.att.fill_(-3)
        self.graph.replay()
        return self.st.item()

    def model(self, ctx, new):
        """The pages that the step takes, on the host; False if there are too few."""
        want = [max(0, P.ceil(c + n, self.page) - len(r)) for c, n, r in zip(ctx, new, self.rows)]
        if sum(want) > self.n_pages - self.start:
            return False
        for b, w in enumerate(want):
            self.rows[b] += self.list[self.start: self.start + w]
            self.start += w
        return True

    def give_back(self, b):
        """A request ends: its pages go in front of the free ones, on the device."""
        n = len(self.rows[b])
        if n:
            self.free_start -= n
            self.free[self.start - n: self.start] = self.table[b, :n]
        self.held[b] = 0
        self.start -= n
        self.list[self.start: self.start + n] = self.rows[b]
        self.rows[b] = []

    def check_books(self):
        assert self.free_start.item() == self.start and self.held.tolist() == [len(r) for r in self.rows]
        assert [t[:len(r)] for t, r in zip(self.table.tolist(), self.rows)] == self.rows
        assert sorted(self.list[self.start:] + sum(self.rows, [])) == list(range(self.n_pages))


def test_two_replays_take_different_pages():
    s = Replayed(3, 16, 4, 12, 40, 20)
    for ctx, new in (([0, 0, 0], [10, 16, 3]), ([10, 16, 3], [10, 1, 0]), ([20, 17, 3], [13, 1, 14])):
        assert s.model(ctx, new) and s.replay(ctx, new) == OK
        s.check_books()
    assert sum(map(len, s.rows)) == 7


def test_a_replayed_loop_with_rejections_keeps_every_request_s_history():
    """Prompt, drafts, verifications of which part is rejected, requests that end and begin: attention
    against fp64 over what was accepted, and the cache holds it unchanged."""
    n_req, page, max_new = 5, 16, 24
    s = Replayed(n_req, page, 10, 24, n_req * max_new, max_new, seed=3)
    g = torch.Generator().manual_seed(1)
    gd = torch.Generator(device="cuda").manual_seed(2)
    r = lambda lo, h: int(torch.randint(lo, h + 1, (1,), generator=g))
    ctx, kept = [0] * n_req, [[] for _ in range(n_req)]    # per request: (k, v) of each accepted token
    refused = rejected = 0
    for step in range(60):
        new = [min(r(5, max_new) if c == 0 else (1 if step % 3 else r(0, 11)), 10 * page - c) for c in ctx]
        s.qkv.normal_(generator=gd)
        fits = s.model(ctx, new)
        st = s.replay(ctx, new)
        assert st == (OK if fits else WORKSPACE)
        s.check_books()
        if not fits:                               # an empty step; the longest request makes room
            refused += 1
            assert not s.out[0].any() and not s.out[1].any() and (s.att == -3).all()
            b = max(range(n_req), key=lambda i: len(s.rows[i]))
            s.give_back(b)
            ctx[b], kept[b] = 0, []
            continue
        n = sum(new)

        class M:
            B, page, rows = n_req, s.page, s.rows
        M.new, M.kv, M.cu_list = new, [c + x for c, x in zip(ctx, new)], s.out[0].tolist()
        pos = s.out[2][:n].long()
        assert pos.tolist() == [c + i for c, x in zip(ctx, new) for i in range(x)]
        ref = P.rope_reference(s.qkv[:n, :s.Hq], pos, 1e4)
        assert ((s.q_rot[:n].double() - ref).abs() <= P.rope_tolerance(s.qkv[:n, :s.Hq], ref, pos)).all()
        if n:
            ref, tol = P.attention_reference(M, s.q_rot[:n], s.kp, s.vp)
            assert ((s.att[:n].double() - ref).abs() <= tol).all()
        assert (s.att[n:] == -3).all()
        for b in range(n_req):
            at, c, x = M.cu_list[b], ctx[b], new[b]
            rows = lambda p0, p1: (torch.tensor([s.rows[b][p // page] for p in range(p0, p1)], dtype=torch.long),
                                   torch.tensor([p % page for p in range(p0, p1)], dtype=torch.long))
            if c:                                  # what was accepted before is as it was stored
                i = rows(0, c)
                assert torch.equal(s.kp[i], torch.stack([k for k, _ in kept[b]]))
                assert torch.equal(s.vp[i], torch.stack([v for _, v in kept[b]]))
            if x:
                i = rows(c, c + x)
                assert torch.equal(s.vp[i], s.qkv[at:at + x, s.Hq + s.Hkv:])
                accepted = x if c == 0 else r(min(1, x), x)
                rejected += x - accepted
                kept[b] += [(s.kp[i[0][j], i[1][j]].clone(), s.vp[i[0][j], i[1][j]].clone())
                            for j in range(accepted)]
                ctx[b] = c + accepted
    assert refused and rejected > 50


def test_a_short_list_and_bad_starts_leave_an_empty_step():
    s = Replayed(2, 8, 4, 6, 40, 32)
    assert s.replay([0, 0], [9, 30]) == OK and s.model([0, 0], [9, 30])       # 2 + 4 pages, all of them
    s.check_books()
    before = s.table.clone()
    assert s.replay([9, 30], [8, 0]) == WORKSPACE          # a third page for the first
    assert torch.equal(s.table, before) and not s.out[0].any() and s.out[4].item() == 0
    s.check_books()
    assert s.replay([9, 30], [7, 2]) == OK                 # fits in what they hold
    s.check_books()
    for bad in (-1, 7, 2 ** 31 - 1, -2 ** 31):
        s.free_start.fill_(bad)
        assert s.replay([9, 30], [1, 1]) == INVALID and s.free_start.item() == bad
        assert torch.equal(s.table, before) and not s.out[0].any()


def test_the_place_alone_and_no_requests():
    """free_start without n_held; a batch of none moves nothing."""
    st, start = _i32([0]), _i32([2])
    table = torch.full((2, 4), -1, dtype=I32, device="cuda")
    o = [_i32([0] * n) for n in (3, 2, 12, 12, 1)]
    B.page_plan(_i32([0, 0]), _i32([3, 9]), _i32([9, 8, 7, 6, 5, 4]), table, 8, 10, *o, st, free_start=start)
    assert table.tolist() == [[7, -1, -1, -1], [6, 5, -1, -1]] and start.item() == 5 and st.item() == 0
    none = [_i32([0] * n) for n in (1, 0, 4, 4, 1)]
    B.page_plan(_i32([]), _i32([]), _i32([1, 2]), table[:0], 8, 10, *none, st, n_held=_i32([]), free_start=start.fill_(1))
    assert start.item() == 1 and st.item() == 0 and none[2].tolist() == [-1] * 4
