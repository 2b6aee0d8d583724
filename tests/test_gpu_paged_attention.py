"""ks_paged_attention_bf16 against fp64 (tests/_paged.py derives the tolerance):
lengths from one token up, odd pages and groups, windows and first tokens,
masks that leave a row or a page empty, garbage where nobody looks, padding,
bad pages, streams, captured calls; and the three paged calls together."""
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


def _queries(L, Hq, hd, pad=0, seed=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(L.n_tokens + pad, Hq, hd, generator=g, device="cuda") * 1.3).to(P.BF16)


def _attend(L, q, kp, vp, ws, window=0, sinks=0, out=None, max_new=None, kv_len=None, table=None):
    out = torch.full_like(q, -3.0) if out is None else out
    st = torch.zeros(1, dtype=I32, device="cuda")
    B.paged_attention_bf16(q, kp, vp, L.table if table is None else table, L.cu,
                           L.kv_len if kv_len is None else kv_len,
                           L.max_new if max_new is None else max_new, out, ws, window=window,
                           sinks=sinks, status=st)
    return out, st


def _within(out, ref, tol):
    err = (out.double() - ref).abs()
    worst = (err / tol).max().item() if err.numel() else 0.0
    assert not out.isnan().any() and (err <= tol).all(), f"worst error / tolerance {worst:.3f}"


def _ragged(n, ctx, new, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda lo, hi: torch.randint(lo, hi + 1, (n,), generator=g).tolist()
    return list(zip(r(*ctx), r(*new)))


# (lens, heads, page)
PLAIN = [
    ([(0, 1)], (4, 4, 64), 8),
    ([(0, 1)], (32, 8, 128), 16),
    ([(126, 1), (127, 1), (128, 1), (129, 1), (255, 1), (0, 1)], (16, 4, 64), 16),
    ([(0, 5), (7, 0), (0, 0), (250, 9), (1, 2)], (32, 8, 128), 48),
    ([(0, 31), (1, 32), (0, 33), (5, 43), (300, 64)], (12, 4, 128), 24),
    ([(0, 128)], (1, 1, 128), 128),
    ([(0, 127), (1, 129), (200, 300)], (4, 4, 64), 256),
    ([(100, 77)], (8, 1, 128), 64),
    ([(100, 3), (40, 1)], (128, 1, 64), 32),
    ([(20000, 1)], (8, 1, 128), 16),
    ([(3000, 3), (9000, 2)], (16, 2, 128), 64),
    ([(5000, 700)], (4, 2, 128), 64),
    (_ragged(300, (0, 200), (0, 3), 1), (8, 2, 64), 16),
    (_ragged(1200, (0, 40), (0, 1), 2), (2, 1, 64), 8),
    (_ragged(37, (0, 900), (1, 11), 3), (32, 8, 128), 32),
]


@pytest.mark.parametrize("i", range(len(PLAIN)))
def test_causal_attention_over_pages(i, ws):
    lens, (Hq, Hkv, hd), page = PLAIN[i]
    L = P.Layout(lens, page, seed=i)
    kp, vp = L.pool(Hkv, hd, seed=10 + i), L.pool(Hkv, hd, seed=20 + i)
    q = _queries(L, Hq, hd)
    out, st = _attend(L, q, kp, vp, ws)
    _within(out, *P.attention_reference(L, q, kp, vp))
    assert st.item() == 0
    # the same call again: the same bits
    assert torch.equal(_attend(L, q, kp, vp, ws)[0], out)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("heads,new", [((8, 2), n) for n in (2, 4, 5, 8, 9, 12, 16, 17, 32, 33)]
                         + [((10, 2), 13), ((10, 2), 26), ((7, 1), 10), ((6, 2), 43), ((31, 1), 2),
                            ((33, 1), 2), ((100, 1), 1), ((65, 1), 1)])
def test_row_counts_around_the_tile_sizes(heads, new, hd, ws):
    """Query rows per kv head on both sides of 16, 32, 64 and 128, of full and of
    short chunks in one step; the pages divide neither a block nor each other."""
    Hq, Hkv = heads
    L = P.Layout([(333, new), (0, max(1, new - 1)), (1500, 1), (127, new), (640, 0), (129, 1)], 40,
                 seed=new)
    kp, vp = L.pool(Hkv, hd), L.pool(Hkv, hd, seed=2)
    q = _queries(L, Hq, hd)
    for window, sinks in ((0, 0), (150, 3)):
        out, st = _attend(L, q, kp, vp, ws, window, sinks)
        _within(out, *P.attention_reference(L, q, kp, vp, window, sinks))
        assert st.item() == 0


@pytest.mark.parametrize("hd,grp,hi,window", [(64, 4, 11, 769), (64, 4, 14, 0), (128, 4, 11, 0), (64, 1, 60, 300),
                                              (128, 7, 9, 0)])
def test_many_short_requests_of_different_row_counts(hd, grp, hi, window, ws):
    """Units of 1 to 64 rows that follow one another on the same SM: nothing of one
    unit's rows may reach the next one's, however far its warps have run ahead."""
    for seed in range(6):
        g = torch.Generator().manual_seed(seed)
        r = lambda lo, h, n: torch.randint(lo, h + 1, (n,), generator=g).tolist()
        lens = [(c if c > 60 else 0, n) for c, n in zip(r(0, 1300, 110), r(0, hi, 110))]
        L = P.Layout(lens, 32, seed=seed)
        kp, vp = L.pool(2, hd, seed=seed), L.pool(2, hd, seed=seed + 50)
        q = _queries(L, 2 * grp, hd, seed=seed)
        ref = P.attention_reference(L, q, kp, vp, window, 4)
        first = None
        for _ in range(3):
            out, st = _attend(L, q, kp, vp, ws, window, 4, max_new=64 // grp)
            _within(out, *ref)
            assert st.item() == 0 and (first is None or torch.equal(out, first))
            first = out


@pytest.mark.parametrize("page", [8, 40, 56, 96, 128, 384, 1024])
@pytest.mark.parametrize("new", [3, 70])
def test_page_sizes(page, new, ws):
    L = P.Layout([(1000, new), (page, 1), (page - 1, 2), (3 * page + 5, new)], page, seed=page)
    kp, vp = L.pool(2, 128), L.pool(2, 128, seed=2)
    q = _queries(L, 8, 128)
    out, st = _attend(L, q, kp, vp, ws)
    _within(out, *P.attention_reference(L, q, kp, vp))
    assert st.item() == 0


def test_many_requests_mostly_idle(ws):
    g = torch.Generator().manual_seed(7)
    n = (torch.rand(5000, generator=g) < 0.1).long().tolist()
    c = torch.randint(0, 300, (5000,), generator=g).tolist()
    lens = [(ci if ni else 0, ni) for ci, ni in zip(c, n)]
    lens[-1] = (4000, 1)
    L = P.Layout(lens, 16)
    kp, vp = L.pool(1, 64), L.pool(1, 64, seed=2)
    q = _queries(L, 2, 64)
    out, st = _attend(L, q, kp, vp, ws)
    _within(out, *P.attention_reference(L, q, kp, vp))
    assert st.item() == 0


@pytest.mark.parametrize("new", [1, 40])
def test_a_pool_past_32_bit_offsets(new, ws):
    """Pages behind the 2^31st element of a pool (4.3 GB each of K and V)."""
    Hkv, hd, page = 8, 128, 64
    L = P.Layout([(700, new), (130, 1)], page)
    n_pages = (1 << 31) // (page * Hkv * hd) + L.n_pages
    kp, vp = (torch.empty(n_pages, page, Hkv, hd, dtype=P.BF16, device="cuda") for _ in range(2))
    first = n_pages - L.n_pages
    kp[first:], vp[first:] = L.pool(Hkv, hd), L.pool(Hkv, hd, seed=2)
    q = _queries(L, 32, hd)
    table = torch.where(L.table >= 0, L.table + first, L.table)
    out, st = _attend(L, q, kp, vp, ws, table=table)
    _within(out, *P.attention_reference(L, q, kp[first:], vp[first:]))
    assert st.item() == 0


# (lens, heads, page, window, sinks)
WINDOWED = [
    ([(0, 1), (5, 1), (400, 1)], (4, 4, 64), 16, 1, 0),
    ([(0, 9), (300, 9), (128, 3)], (32, 8, 128), 16, 1, 1),
    ([(0, 200), (511, 3)], (16, 4, 64), 32, 17, 4),
    ([(1000, 5), (90, 2), (4000, 1)], (32, 8, 128), 48, 128, 130),
    ([(1000, 300)], (8, 1, 128), 64, 100, 63),
    ([(10000, 2), (128, 1), (129, 1)], (8, 2, 128), 128, 1000, 4),
    ([(700, 1), (60, 40)], (12, 4, 128), 24, 5000, 4),       # a window wider than the context
    ([(700, 2), (300, 1)], (8, 2, 64), 16, 64, 5000),        # every token a first token
    ([(2047, 64)], (16, 4, 64), 8, 257, 0),
]


def _invisible(L, window, sinks, shape, kv=None):
    """Mask [n_pages][page] of the positions that no token of any request sees,
    and the table with the entries of wholly unseen pages overwritten."""
    dead = torch.ones(shape[:2], dtype=torch.bool)
    table = torch.full_like(L.table, 1 << 29)
    for b in range(L.B):
        S = L.kv[b]
        for t in range(L.new[b]):
            p = S - L.new[b] + t
            lo = max(0, p - window + 1) if window else 0
            for j in list(range(min(sinks, lo))) + list(range(lo, p + 1)):
                dead[L.rows[b][j // L.page], j % L.page] = False
                table[b, j // L.page] = L.rows[b][j // L.page]
    return dead.cuda(), table


@pytest.mark.parametrize("i", range(len(WINDOWED)))
def test_window_and_first_tokens(i, ws):
    lens, (Hq, Hkv, hd), page, window, sinks = WINDOWED[i]
    L = P.Layout(lens, page, seed=i)
    kp, vp = L.pool(Hkv, hd, seed=10 + i), L.pool(Hkv, hd, seed=20 + i)
    q = _queries(L, Hq, hd)
    ref = P.attention_reference(L, q, kp, vp, window, sinks)
    out, st = _attend(L, q, kp, vp, ws, window, sinks)
    _within(out, *ref)
    assert st.item() == 0
    # garbage at every position that nobody sees, in the table's entries of pages
    # without a visible key, and in the pages of nobody
    dead, table = _invisible(L, window, sinks, kp.shape)
    for bad in (math.nan, math.inf):
        kp[dead], vp[dead] = bad, -bad
        again, st = _attend(L, q, kp, vp, ws, window, sinks, table=table)
        assert torch.equal(again, out) and st.item() == 0


@pytest.mark.parametrize("i", [2, 3, 4, 6, 9, 11])
def test_garbage_behind_the_sequences_is_not_seen(i, ws):
    lens, (Hq, Hkv, hd), page = PLAIN[i]
    L = P.Layout(lens, page, seed=i)
    kp, vp = L.pool(Hkv, hd, seed=10 + i), L.pool(Hkv, hd, seed=20 + i)
    q = _queries(L, Hq, hd)
    out, _ = _attend(L, q, kp, vp, ws)
    dead, table = _invisible(L, 0, 0, kp.shape)
    for bad in (math.nan, math.inf):
        kp[dead], vp[dead] = bad, bad
        again, st = _attend(L, q, kp, vp, ws, table=table)
        assert torch.equal(again, out) and st.item() == 0


def test_infinite_keys_in_masked_places_of_the_chunk(ws):
    """A later token's key is masked for an earlier one by position, not by
    arithmetic on its score."""
    L = P.Layout([(100, 6)], 16)
    kp, vp = L.pool(2, 64), L.pool(2, 64, seed=2)
    q = _queries(L, 4, 64).abs()
    out, _ = _attend(L, q, kp, vp, ws)
    last = L.kv[0] - 1
    kp[L.rows[0][last // 16], last % 16] = math.inf
    again, _ = _attend(L, q, kp, vp, ws)
    assert torch.equal(again[:5], out[:5])


@pytest.mark.parametrize("heads,page", [((8, 2, 128), 16), ((4, 4, 64), 64)])
def test_tokens_without_a_key_get_zeros_and_padding_is_left(heads, page, ws):
    Hq, Hkv, hd = heads
    L = P.Layout([(0, 5), (3, 130), (0, 1), (64, 2)], page)
    kp, vp = L.pool(Hkv, hd), L.pool(Hkv, hd, seed=2)
    q = _queries(L, Hq, hd, pad=13)
    q[L.n_tokens:] = math.nan
    kv = [2, 100, 0, 66]                       # shorter than the chunk: the first tokens see nothing
    out, st = _attend(L, q, kp, vp, ws, kv_len=torch.tensor(kv, dtype=I32, device="cuda"))
    ref, tol = P.attention_reference(L, q, kp, vp, kv=kv)
    n = L.n_tokens
    _within(out[:n], ref, tol)
    assert (out[:3] == 0).all() and (out[5:35] == 0).all() and (out[135] == 0).all()
    assert (out[n:] == -3).all() and st.item() == 0


def test_large_scores_and_a_late_maximum(ws):
    """Scores up to about 60 whose maximum comes last: the running reference
    moves, earlier sums shrink to nothing."""
    L = P.Layout([(2000, 3), (700, 1)], 32)
    kp, vp = L.pool(2, 128), L.pool(2, 128, seed=2)
    q = _queries(L, 8, 128)
    ids = [L.rows[0][j // 32] * 32 + j % 32 for j in range(0, 2003, 97)]
    rise = torch.linspace(0.2, 4.0, len(ids), device="cuda")[:, None, None].to(P.BF16)
    kp.view(-1, 2, 128)[ids] = rise * q[0, ::4]
    out, _ = _attend(L, q, kp, vp, ws)
    _within(out, *P.attention_reference(L, q, kp, vp))


def test_bad_pages_and_lengths_are_reported(ws):
    L = P.Layout([(300, 2), (40, 1), (500, 3)], 16)
    kp, vp = L.pool(2, 64), L.pool(2, 64, seed=2)
    q = _queries(L, 8, 64)
    good, st = _attend(L, q, kp, vp, ws)
    assert st.item() == 0
    for page in (-1, L.n_pages, 2 ** 31 - 1, -2 ** 31):
        table = L.table.clone()
        table[0, 5] = page
        out, st = _attend(L, q, kp, vp, ws, table=table)
        assert st.item() == 1
        z = P.Layout([(300, 2), (40, 1), (500, 3)], 16)     # a page of zeros in its place
        z.rows[0][5] = z.n_pages
        k0, v0 = (torch.cat((x, torch.zeros_like(x[:1]))) for x in (kp, vp))
        ref, tol = P.attention_reference(z, q, k0, v0)
        _within(out, ref, tol)
    # a request longer than its table row, and one with more tokens than max_new
    kv = L.kv_len.clone()
    kv[1] = L.max_blocks * 16 + 5
    assert _attend(L, q, kp, vp, ws, kv_len=kv)[1].item() == 1
    out, st = _attend(L, q, kp, vp, ws, max_new=2)
    assert st.item() == 1 and torch.equal(out[:3], good[:3]) and (out[5] == -3).all()
    # and the next call is a good one again
    out, st = _attend(L, q, kp, vp, ws)
    assert st.item() == 0 and torch.equal(out, good)


def test_a_table_without_columns(ws):
    """No position fits: every token sees nothing, and the lengths are reported."""
    q = torch.randn(3, 8, 64, device="cuda").to(P.BF16)
    out = torch.full_like(q, -3.0)
    kp = torch.randn(2, 16, 2, 64, device="cuda").to(P.BF16)
    i32 = lambda x: torch.tensor(x, dtype=I32, device="cuda")
    st = i32([0])
    B.paged_attention_bf16(q, kp, kp.clone(), torch.zeros(2, 0, dtype=I32, device="cuda"), i32([0, 1, 3]),
                           i32([1, 2]), 2, out, ws, status=st)
    assert (out == 0).all() and st.item() == 1


@pytest.mark.parametrize("new,fill", [(1, 0x7F), (1, 0xFF), (60, 0x7F)])
def test_a_workspace_that_does_not_start_out_zero_is_reported(new, fill):
    L = P.Layout([(9000, new)], 64)            # long enough to be cut into pieces
    kp, vp = L.pool(2, 128), L.pool(2, 128, seed=2)
    q = _queries(L, 8, 128)
    w = B.paged_attention_workspace().fill_(fill)
    assert _attend(L, q, kp, vp, w)[1].item() == 3
    w.zero_()
    out, st = _attend(L, q, kp, vp, w)
    _within(out, *P.attention_reference(L, q, kp, vp))
    assert st.item() == 0


def test_one_workspace_serves_calls_of_every_shape(ws):
    """Large, small, cut and uncut steps one after the other, without clearing."""
    for i in (9, 0, 11, 14, 6, 12, 10):
        lens, (Hq, Hkv, hd), page = PLAIN[i]
        L = P.Layout(lens, page, seed=i)
        kp, vp = L.pool(Hkv, hd, seed=10 + i), L.pool(Hkv, hd, seed=20 + i)
        q = _queries(L, Hq, hd)
        fresh = _attend(L, q, kp, vp, B.paged_attention_workspace())[0]
        assert torch.equal(_attend(L, q, kp, vp, ws)[0], fresh)


def test_scores_that_jump_past_every_reference(ws):
    """A key whose score exceeds all before it by hundreds takes the whole row, at
    the piece's start, in its middle and at its end; before it the row is even."""
    for new, Hq in ((1, 4), (5, 8), (40, 8)):
        for at in (3, 130, 1000, 1999):
            L = P.Layout([(2000, new)], 32)
            kp, vp = L.pool(2, 128, fill=0.0), L.pool(2, 128, seed=2)
            q = _queries(L, Hq, 128).abs()
            row = L.rows[0][at // 32]
            kp[row, at % 32] = 60.0
            out, st = _attend(L, q, kp, vp, ws)
            v = vp[row, at % 32].repeat_interleave(Hq // 2, 0)
            assert st.item() == 0 and torch.equal(out, v.expand_as(out))


@pytest.mark.parametrize("cu", [[0, -4, 3, 6], [0, 5, 2, 6], [0, 2, 3, 900], [-3, 2, 3, 6],
                                [0, 2, 3, 2 ** 31 - 1], [2 ** 31 - 1, -2 ** 31, 0, 6]])
def test_broken_offsets_stay_in_bounds(cu, ws):
    L = P.Layout([(300, 2), (40, 1), (500, 3)], 16)
    kp, vp = L.pool(2, 64), L.pool(2, 64, seed=2)
    q = _queries(L, 8, 64, pad=4)
    buf = torch.full((3 * q.shape[0], 8, 64), -3.0, dtype=P.BF16, device="cuda")
    out = buf[q.shape[0]: 2 * q.shape[0]]
    L.cu = torch.tensor(cu, dtype=I32, device="cuda")
    _, st = _attend(L, q, kp, vp, ws, out=out)
    assert st.item() == 1
    assert (buf[: q.shape[0]] == -3).all() and (buf[2 * q.shape[0]:] == -3).all()


def test_equals_the_contiguous_attention(ws):
    """One state of T evaluation tokens over one request: what ks_attention_bf16
    computes from a contiguous cache."""
    T, ctx, Hq, Hkv, hd = 16, 1000, 32, 8, 128
    L = P.Layout([(ctx, T)], 16)
    kp, vp = L.pool(Hkv, hd), L.pool(Hkv, hd, seed=2)
    q = _queries(L, Hq, hd)
    ids = torch.tensor(L.rows[0][: P.ceil(ctx + T, 16)], device="cuda")
    kc, vc = (x[ids].flatten(0, 1).contiguous() for x in (kp, vp))
    dense = torch.empty_like(q)
    B.attention_bf16(q, kc, vc, T, ctx, dense)
    out, _ = _attend(L, q, kp, vp, ws)
    ref, tol = P.attention_reference(L, q, kp, vp)
    _within(dense, ref, tol)
    _within(out, ref, tol)


def test_two_streams_with_a_workspace_each(ws):
    work = []
    for i in (9, 11, 14):
        lens, (Hq, Hkv, hd), page = PLAIN[i]
        L = P.Layout(lens, page, seed=i)
        kp, vp = L.pool(Hkv, hd), L.pool(Hkv, hd, seed=2)
        q = _queries(L, Hq, hd)
        alone = _attend(L, q, kp, vp, ws)[0]
        work.append((L, q, kp, vp, alone, torch.cuda.Stream(), B.paged_attention_workspace()))
    torch.cuda.synchronize()
    outs = []
    for rep in range(5):
        for L, q, kp, vp, _, s, w in work:
            with torch.cuda.stream(s):
                outs.append(_attend(L, q, kp, vp, w)[0])
    torch.cuda.synchronize()
    for k, o in enumerate(outs):
        assert torch.equal(o, work[k % 3][4])


def test_captured_step_follows_new_lengths(ws):
    """Plan, append and attention captured once, replayed with other lengths
    (an idle request, a shrunk batch) and other values; two graphs share a
    workspace, one after the other."""
    Hq, Hkv, hd, page, cap, max_new = 8, 2, 128, 16, 24, 6
    first = [(100, 3), (0, 6), (47, 1), (15, 2)]
    L = P.Layout(first, page, full=False, extra_blocks=8, spare=40)
    g = torch.Generator(device="cuda").manual_seed(0)
    qkv = torch.randn(cap, Hq + 2 * Hkv, hd, generator=g, device="cuda").to(P.BF16)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    kp, vp = L.pool(Hkv, hd), L.pool(Hkv, hd, seed=2)
    z = lambda n: torch.zeros(n, dtype=I32, device="cuda")
    ctx, new, free, table = L.ctx_len, L.new_len, L.free, L.table
    cu, kv, pos, slots, taken, st = z(5), z(4), z(cap), z(cap), z(1), z(1)
    q_out = torch.zeros(cap, Hq, hd, dtype=P.BF16, device="cuda")
    out, wout = torch.zeros_like(q_out), torch.zeros_like(q_out)

    def step():
        B.page_plan(ctx, new, free, table, page, L.n_pages, cu, kv, pos, slots, taken, st)
        B.rope_append_bf16(q, k, v, pos, slots, kp, vp, 1e4, q_out, st)
        B.paged_attention_bf16(q_out, kp, vp, table, cu, kv, max_new, out, ws, status=st)

    def windowed():
        B.paged_attention_bf16(q_out, kp, vp, table, cu, kv, max_new, wout, ws, window=20, sinks=2,
                               status=st)

    step()
    windowed()
    torch.cuda.synchronize()
    graphs = []
    for f in (step, windowed):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            f()
        graphs.append(graph)
    for lens in (first, [(100, 1), (30, 5), (20, 0), (9, 6)], [(0, 0), (1, 1), (80, 0), (0, 0)],
                 [(112, 6), (16, 6), (48, 6), (15, 6)]):
        M = P.Layout(lens, page, full=False, extra_blocks=8, spare=40, seed=sum(map(sum, lens)))
        blocks = table.shape[1]
        rows = [(r + [-1] * blocks)[:blocks] for r in M.rows]
        n_free = min(free.numel(), len(M.free_list))
        qkv.normal_(generator=g)
        table.copy_(torch.tensor(rows, dtype=I32))
        free.fill_(-1)
        M.free_list = [x for x in M.free_list if x < L.n_pages]
        rows_ok = all(x < L.n_pages for r in rows for x in r)
        if not rows_ok or n_free == 0:         # keep every page inside the captured pool
            order = torch.randperm(L.n_pages, generator=torch.Generator().manual_seed(1)).tolist()
            for b, r in enumerate(rows):
                n = sum(x >= 0 for x in r)
                rows[b], order = order[:n] + [-1] * (blocks - n), order[n:]
            M.free_list = order
            table.copy_(torch.tensor(rows, dtype=I32))
        n = min(free.numel(), len(M.free_list))
        free[:n] = torch.tensor(M.free_list[:n], dtype=I32)
        ctx.copy_(M.ctx_len)
        new.copy_(M.new_len)
        out.fill_(-3)
        wout.fill_(-3)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert st.item() == 0
        M.rows = rows
        M.rows = P.plan_reference(M, cap)[0]
        assert table.tolist() == M.rows and slots.tolist() == P.plan_reference(M, cap)[4]
        n = M.n_tokens
        p = pos[:n].long()
        ref = P.rope_reference(q[:n], p, 1e4)
        assert ((q_out[:n].double() - ref).abs() <= P.rope_tolerance(q[:n], ref, p)).all()
        if n:
            _within(out[:n], *P.attention_reference(M, q_out[:n], kp, vp))
            _within(wout[:n], *P.attention_reference(M, q_out[:n], kp, vp, 20, 2))
        assert (out[n:] == -3).all() and (wout[n:] == -3).all()


def test_a_run_of_steps_equals_one_contiguous_cache(ws):
    """Prompt, drafts of one token, a verification: the three calls step by step
    over a growing paged cache, against fp64 attention over the whole history."""
    Hq, Hkv, hd, page, base, n_req = 16, 4, 64, 16, 1e4, 3
    g = torch.Generator(device="cuda").manual_seed(5)
    steps = [(70, 33, 1), (1, 1, 1), (1, 0, 1), (1, 1, 1), (5, 4, 0), (1, 1, 130)]
    blocks = 20
    i32 = lambda x: torch.tensor(x, dtype=I32, device="cuda")
    table = torch.full((n_req, blocks), -1, dtype=I32, device="cuda")
    order = torch.randperm(60, generator=torch.Generator().manual_seed(1)).tolist()
    kp = torch.full((60, page, Hkv, hd), math.nan, dtype=P.BF16, device="cuda")
    vp = torch.full_like(kp, math.nan)
    hist = [[] for _ in range(n_req)]          # per request: (q, k, v) rows as given
    ctx = [0] * n_req
    for new in steps:
        n = sum(new)
        qkv = torch.randn(n, Hq + 2 * Hkv, hd, generator=g, device="cuda").to(P.BF16)
        cu, kv = i32([0] * (n_req + 1)), i32([0] * n_req)
        pos, slots, taken, st = i32([0] * n), i32([0] * n), i32([0]), i32([0])
        q_out = torch.empty(n, Hq, hd, dtype=P.BF16, device="cuda")
        out = torch.empty_like(q_out)
        B.page_plan(i32(ctx), i32(list(new)), i32(order), table, page, 60, cu, kv, pos, slots, taken, st)
        B.rope_append_bf16(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], pos, slots, kp, vp,
                           base, q_out, st)
        B.paged_attention_bf16(q_out, kp, vp, table, cu, kv, max(new), out, ws, status=st)
        assert st.item() == 0
        order = order[taken.item():]
        at = 0
        for b in range(n_req):
            hist[b].append(qkv[at:at + new[b]])
            allr = torch.cat(hist[b]).double()
            S, m = allr.shape[0], new[b]
            p = torch.arange(S, device="cuda")
            k = P.rope_reference(allr[:, Hq:Hq + Hkv], p, base).to(P.BF16)
            if m:
                D = P.Layout([(S - m, m)], page, extra_blocks=0)
                ids = torch.tensor(D.rows[0], device="cuda")
                dk, dv = D.pool(Hkv, hd, fill=0.0), D.pool(Hkv, hd, fill=0.0)
                pad = lambda x: torch.cat((x, x.new_zeros(len(ids) * page - S, Hkv, hd)))
                dk[ids] = pad(k).view(-1, page, Hkv, hd)
                dv[ids] = pad(allr[:, Hq + Hkv:].to(P.BF16)).view(-1, page, Hkv, hd)
                ref, tol = P.attention_reference(D, q_out[at:at + m], dk, dv)
                # a rotated key may fall on the other side of a rounding: one step of bf16 in
                # each of a row's keys moves a score by up to 2^-7 sum|q k| / sqrt(hd), twice that
                # the probabilities' relative error
                rows = q_out[at:at + m].double().abs().amax()
                wide = 2 * 2.0 ** -7 * hd * rows * 2.0 ** -12 * dk.double().abs().amax() / math.sqrt(hd)
                _within(out[at:at + m], ref, tol + wide)
            at += m
            ctx[b] += m
