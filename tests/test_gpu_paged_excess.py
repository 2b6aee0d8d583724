"""ks_paged_attention_bf16 where a request's lengths break max_new, n_tokens or
its table row: the excess is dropped and reported, and what is left is computed
at its own positions (fp64 reference below, tolerance as tests/_paged.py derives
it)."""
import math

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


@pytest.fixture(scope="module")
def ws(lib):
    return B.paged_attention_workspace()


def _queries(n, Hq, hd, seed=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(n, Hq, hd, generator=g, device="cuda") * 1.3).to(P.BF16)


def _attend(q, kp, vp, table, cu, kv, max_new, ws, window=0, sinks=0):
    out = torch.full_like(q, -3.0)
    st = torch.zeros(1, dtype=I32, device="cuda")
    B.paged_attention_bf16(q, kp, vp, table, cu, kv, max_new, out, ws, window=window, sinks=sinks,
                           status=st)
    return out, st.item()


def _within(out, ref, tol):
    err = (out.double() - ref).abs()
    assert not out.isnan().any() and (err <= tol).all(), \
        f"worst error / tolerance {(err / tol).max().item():.3f}"


@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 3)])
@pytest.mark.parametrize("lens,max_new", [([(300, 2), (40, 1), (500, 5)], 3), ([(200, 11), (0, 9), (64, 1)], 4),
                                          ([(130, 300), (20, 90), (700, 2)], 33), ([(0, 7)], 1)])
def test_tokens_past_max_new_leave_the_others_in_place(lens, max_new, window, sinks, ws):
    L = P.Layout(lens, 16)
    kp, vp = L.pool(2, 64), L.pool(2, 64, seed=2)
    q = _queries(L.n_tokens, 8, 64)
    ref, tol = P.attention_reference(L, q, kp, vp, window, sinks)
    out, st = _attend(q, kp, vp, L.table, L.cu, L.kv_len, max_new, ws, window, sinks)
    assert st == 1
    kept = torch.zeros(L.n_tokens, dtype=torch.bool)
    for at, n in zip(L.cu_list, L.new):
        kept[at: at + min(n, max_new)] = True
    kept = kept.cuda()
    _within(out[kept], ref[kept], tol[kept])
    assert (out[~kept] == -3).all()


@pytest.mark.parametrize("n,max_new", [(301, 400), (24, 24)])
def test_tokens_past_the_query_rows_leave_the_others_in_place(n, max_new, ws):
    lens = [(90, n // 2), (33, n - n // 2)]
    L = P.Layout(lens, 32)
    kp, vp = L.pool(2, 128), L.pool(2, 128, seed=2)
    q = _queries(n, 4, 128)
    ref, tol = P.attention_reference(L, q, kp, vp)
    for rows in (n - 1, n - n // 4):
        out, st = _attend(q[:rows], kp, vp, L.table, L.cu, L.kv_len, max_new, ws)
        assert st == 1
        _within(out, ref[:rows], tol[:rows])


def _reference_row(q, k, v, pos, cap, window, sinks):
    """One token at position pos over the keys 0 .. cap-1: (out, tolerance) [Hq][hd]."""
    Hq, hd = q.shape
    j = torch.arange(cap, device=q.device)
    seen = j <= pos
    if window:
        seen = seen & ((j > pos - window) | (j < sinks))
    if not seen.any():
        z = torch.zeros(Hq, hd, dtype=torch.float64, device=q.device)
        return z, z
    grp = Hq // k.shape[1]
    k, v = (x[seen].double().repeat_interleave(grp, 1) for x in (k, v))
    s = torch.einsum("hd,jhd->hj", q.double(), k) / math.sqrt(hd)
    w = torch.softmax(s, -1)
    o = torch.einsum("hj,jhd->hd", w, v)
    big = torch.einsum("hd,jhd->hj", q.double().abs(), k.abs()).amax(-1, keepdim=True)
    e = P.HALF_STEP + 2.0 ** -18 + hd * 2.0 ** -23 * big / math.sqrt(hd)
    tol = (P.HALF_STEP * o.abs() * (1 + 2 * P.HALF_STEP)
           + e / (1 - e) * (torch.einsum("hj,jhd->hd", w, v.abs()) + o.abs()) + 1e-30)
    return o, tol


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("size", [20, 29, 30])
def test_scores_up_to_two_to_the_thirty(size, new, ws):
    """Equal scores of 1 and -1 times 2^size: every key weighs the same (fp32 sums of at most 240 values, one
    rounding of the weights and one of the result)."""
    L = P.Layout([(200, new)], 16)
    kp, vp = L.pool(1, 64, fill=0.0), L.pool(1, 64, seed=2)
    q = torch.zeros(L.n_tokens, 2, 64, dtype=P.BF16, device="cuda")
    q[..., 0] = 2.0 ** 10
    v = vp[torch.tensor(L.rows[0][: P.ceil(L.kv[0], 16)], device="cuda")].flatten(0, 1)[:, 0].double()
    seen = torch.arange(L.kv[0], device="cuda")[None] <= torch.arange(200, L.kv[0], device="cuda")[:, None]
    w = seen.double() / seen.sum(-1, keepdim=True)
    ref, size_of_v = w @ v[: L.kv[0]], w @ v[: L.kv[0]].abs()
    e = P.HALF_STEP + 2.0 ** -16
    tol = P.HALF_STEP * ref.abs() * (1 + 2 * P.HALF_STEP) + e / (1 - e) * (size_of_v + ref.abs()) + 1e-30
    for sign in (1, -1):
        kp[..., 0] = sign * 2.0 ** (size - 10) * 8     # sqrt(head_dim) = 8
        out, st = _attend(q, kp, vp, L.table, L.cu, L.kv_len, new, ws)
        assert st == 0
        for h in range(2):
            _within(out[:, h], ref, tol)


# (page, columns of the table, cached tokens, new tokens, window, sinks): the table's row ends inside a
# block of 128 keys, at its border, before the first new token, inside the window, before it
PAST = [(16, 5, 70, 6, 0, 0), (16, 5, 70, 40, 0, 0), (128, 1, 100, 60, 0, 0), (64, 2, 128, 3, 0, 0),
        (64, 2, 128, 90, 0, 0), (48, 3, 500, 5, 0, 0), (48, 3, 500, 150, 0, 0), (16, 9, 150, 7, 20, 0),
        (16, 9, 150, 70, 20, 3), (128, 2, 1000, 4, 64, 130), (64, 3, 1000, 90, 64, 190), (8, 40, 300, 65, 30, 5),
        (64, 2, 2 ** 31 - 8, 7, 100, 0), (64, 2, 2 ** 31 - 80, 79, 0, 0), (64, 3, 2 ** 31 - 8, 7, 100, 500)]


@pytest.mark.parametrize("page,cols,ctx,new,window,sinks", PAST)
def test_keys_past_the_table_row_are_dropped(page, cols, ctx, new, window, sinks, ws):
    """The tokens keep their positions, so a window counts from them; they see the keys that the table holds."""
    Hq, Hkv, hd, cap = 4, 2, 64, page * cols
    L = P.Layout([(cap, 0), (cap, 0)], page, extra_blocks=0, seed=new)
    kp, vp = L.pool(Hkv, hd), L.pool(Hkv, hd, seed=2)
    i32 = lambda x: torch.tensor(x, dtype=I32, device="cuda")
    q = _queries(new + 1, Hq, hd)
    # the second request's one token is a good one
    out, st = _attend(q, kp, vp, L.table, i32([0, new, new + 1]), i32([ctx + new, cap]), new, ws, window, sinks)
    assert st == int(ctx + new > cap)              # the first case still fits: 76 of 80
    for b, rows in ((0, range(new)), (1, [new])):
        ids = torch.tensor(L.rows[b], device="cuda")
        k, v = (x[ids].flatten(0, 1) for x in (kp, vp))
        for r in rows:
            pos = ctx + r if b == 0 else cap - 1
            _within(out[r], *_reference_row(q[r], k, v, pos, cap, window, sinks))
