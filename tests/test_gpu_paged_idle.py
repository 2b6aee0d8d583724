"""ks_paged_attention_bf16 over batches of mostly idle requests: they change
neither the result nor, much, the time."""
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


def _call(L, at, total, q, kp, vp, ws):
    """The requests of L at the places `at` of a batch of `total`, the others idle: (call, out, status)."""
    i32 = lambda x: torch.tensor(x, dtype=I32, device="cuda")
    new = torch.zeros(total, dtype=torch.long)
    new[at] = torch.tensor(L.new)
    cu = torch.zeros(total + 1, dtype=I32, device="cuda")
    cu[1:] = torch.cumsum(new, 0).cuda()
    kv = torch.zeros(total, dtype=I32, device="cuda")
    kv[at] = L.kv_len
    table = torch.full((total, L.max_blocks), -1, dtype=I32, device="cuda")
    table[at] = L.table
    out, st = torch.full_like(q, -3.0), i32([0])
    return lambda: B.paged_attention_bf16(q, kp, vp, table, cu, kv, L.max_new, out, ws, status=st), out, st


def _setup(lens, heads=(8, 2, 128), page=64):
    L = P.Layout(lens, page)
    Hq, Hkv, hd = heads
    g = torch.Generator(device="cuda").manual_seed(3)
    q = (torch.randn(L.n_tokens, Hq, hd, generator=g, device="cuda") * 1.3).to(P.BF16)
    return L, q, L.pool(Hkv, hd), L.pool(Hkv, hd, seed=2)


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("total", [33, 300, 5000, 16384])
def test_idle_requests_between_the_others_change_nothing(total, new, ws):
    n = min(30, total - 1)
    g = torch.Generator().manual_seed(total)
    L, q, kp, vp = _setup([(int(c), new) for c in torch.randint(0, 900, (n,), generator=g)])
    first, out0, st = _call(L, list(range(n)), n, q, kp, vp, ws)
    first()
    ref, tol = P.attention_reference(L, q, kp, vp)
    assert st.item() == 0 and ((out0.double() - ref).abs() <= tol).all()
    for seed in range(4):
        g = torch.Generator().manual_seed(seed)
        at = sorted(torch.randperm(total, generator=g)[:n].tolist())
        if seed == 1:                              # in two bunches at the ends
            at = list(range(n // 2)) + list(range(total - (n - n // 2), total))
        f, out, st = _call(L, at, total, q, kp, vp, ws)
        f()
        assert st.item() == 0 and torch.equal(out, out0)      # the same cuts, so the same bits


def _time(f):
    """us a call: ten calls in a graph, the best of five replays."""
    f()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(10):
            f()
    graph.replay()
    best = float("inf")
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        graph.replay()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) * 100)
    return best


def test_idle_requests_do_not_hold_the_others_up(ws):
    """Eight live requests of 16,384.  At the batch's end nobody looks past them: that is the measure.  In
    front of the idle ones, and on both sides of them (where the SMs' shares meet at a border of the two
    sides, and inside a request), the step took 29 times as long when the idle ones were walked over 32 at
    a time, past a share's end too."""
    total, n = 16384, 8
    L, q, kp, vp = _setup([(2000, 1)] * n)
    last = _time(_call(L, list(range(total - n, total)), total, q, kp, vp, ws)[0])
    for front in (n, n // 2, n // 2 - 1):
        at = list(range(front)) + list(range(total - n + front, total))
        f, _, st = _call(L, at, total, q, kp, vp, ws)
        assert _time(f) < 4 * last and st.item() == 0
