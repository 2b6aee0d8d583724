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
