"""ks_page_plan_carried's refusals, in the binding and at the C ABI, before
anything is enqueued.  No GPU needed."""
import pytest
import torch

from knapsack_layer_selection_b200 import binding as B
from knapsack_layer_selection_b200 import build as BUILD

FAKE = 4096                                    # an aligned address that no refused call reads
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    BUILD.build()
    return B.load()


def _i(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def _plan(**kw):
    B.page_plan(_i(3), _i(3), _i(9), _i(3, 5), 16, 20, _i(4), _i(3), _i(8), _i(8), _i(1), **kw)


def test_shapes():
    for bad in (_i(4), _i(2), _i(3, 1)):
        with pytest.raises(B.KnapSpecError, match="n_held must have shape"):
            _plan(n_held=bad)
    with pytest.raises(B.KnapSpecError, match="must be a CUDA tensor"):
        _plan(n_held=_i(3))
    for bad in (_i(0), _i(2), _i(1, 1)):
        with pytest.raises(B.KnapSpecError, match="free_start must have shape"):
            _plan(free_start=bad)


def test_refusals(lib):
    def call(B_=2, n_free=4, n_pages=10, page=16, max_blocks=4, cap=8, ctx=FAKE, cu=FAKE, table=FAKE,
             free=FAKE, pos=FAKE, held=FAKE, start=FAKE):
        return lib.ks_page_plan_carried(ctx, FAKE, B_, free, n_free, n_pages, page, table, max_blocks, cap,
                                        cu, FAKE, pos, FAKE, FAKE, held, start, None, None)
    for kw, code in (({"B_": -1}, INVALID), ({"B_": 16385}, UNSUPPORTED), ({"n_free": -1}, INVALID),
                     ({"n_pages": 0}, INVALID), ({"page": 20}, UNSUPPORTED), ({"max_blocks": -1}, INVALID),
                     ({"cap": -1}, INVALID), ({"ctx": None}, INVALID), ({"cu": None}, INVALID),
                     ({"table": None}, INVALID), ({"free": None}, INVALID), ({"pos": None}, INVALID),
                     ({"n_pages": 1 << 28}, UNSUPPORTED), ({"max_blocks": 1 << 27}, UNSUPPORTED)):
        assert call(**kw) == code, kw
        assert call(held=None, start=None, **kw) == code, kw
        assert b"page plan" in lib.ks_last_error()
