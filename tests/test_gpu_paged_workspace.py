"""A workspace of ks_paged_attention_bf16 that does not start out zero is reported,
whatever its arrival counters hold."""
import pytest
import torch

from knapsack_layer_selection_b200 import binding as B
from knapsack_layer_selection_b200 import build as BUILD
from tests import _paged as P

pytestmark = pytest.mark.gpu
I32 = torch.int32
WORKSPACE = 3


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    BUILD.build()
    return B.load()


@pytest.mark.parametrize("new", [1, 40])
def test_small_counts_left_in_the_workspace_are_reported(new):
    """9,000 keys of two heads: units cut over many SMs.  A leftover count from 1 to a unit's pieces less one
    would make an early piece pass for the last one."""
    L = P.Layout([(9000, new)], 64)
    kp, vp = L.pool(2, 128), L.pool(2, 128, seed=2)
    g = torch.Generator(device="cuda").manual_seed(3)
    q = (torch.randn(L.n_tokens, 8, 128, generator=g, device="cuda") * 1.3).to(P.BF16)
    ref, tol = P.attention_reference(L, q, kp, vp)
    ws = B.paged_attention_workspace()
    words = ws.view(I32)
    for count in list(range(1, 148)) + [-1, -2, 255, 1 << 16, 1 << 24, 0x01010101, 0x3F800000]:
        words[:256] = count
        st = torch.zeros(1, dtype=I32, device="cuda")
        B.paged_attention_bf16(q, kp, vp, L.table, L.cu, L.kv_len, L.max_new, torch.empty_like(q), ws, status=st)
        assert st.item() == WORKSPACE, count
    ws.zero_()
    for _ in range(3):
        st = torch.zeros(1, dtype=I32, device="cuda")
        out = torch.empty_like(q)
        B.paged_attention_bf16(q, kp, vp, L.table, L.cu, L.kv_len, L.max_new, out, ws, status=st)
        assert st.item() == 0 and ((out.double() - ref).abs() <= tol).all()
        assert not words[:256].any()               # ready for the next call
