"""The paged cache's refusals: the binding's shape checks and the C ABI's
argument checks, all before anything is enqueued.  No GPU needed."""
import ctypes

import pytest
import torch

from knapsack_layer_selection_b200 import binding as B
from knapsack_layer_selection_b200 import build as BUILD

NOT_CUDA = "must be a CUDA tensor"
FAKE = 4096                                    # an aligned address that no refused call reads


@pytest.fixture(scope="module")
def lib():
    BUILD.build()
    return B.load()


def _i(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def _bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def test_plan_shapes():
    def call(**kw):
        a = dict(ctx=_i(3), new=_i(3), free=_i(9), table=_i(3, 5), cu=_i(4), kv=_i(3), pos=_i(8),
                 slots=_i(8), taken=_i(1))
        a.update(kw)
        B.page_plan(a["ctx"], a["new"], a["free"], a["table"], 16, 20, a["cu"], a["kv"], a["pos"],
                    a["slots"], a["taken"])
    with pytest.raises(B.KnapSpecError, match=NOT_CUDA):
        call()
    for kw, text in (({"new": _i(4)}, "new_len must have shape"), ({"cu": _i(3)}, "cu_new must have shape"),
                     ({"kv": _i(2)}, "kv_len must"), ({"table": _i(2, 5)}, r"block_table must be \[3\]"),
                     ({"slots": _i(7)}, "slots must"), ({"taken": _i(2)}, "n_taken must"),
                     ({"free": _i(3, 3)}, "free_pages must"), ({"ctx": _i(3, 1)}, "ctx_len must")):
        with pytest.raises(B.KnapSpecError, match=text):
            call(**kw)


def test_append_shapes():
    def call(**kw):
        a = dict(q=_bf(6, 8, 64), k=_bf(6, 2, 64), v=_bf(6, 2, 64), pos=_i(6), slots=_i(6),
                 kp=_bf(9, 16, 2, 64), vp=_bf(9, 16, 2, 64), qo=_bf(6, 8, 64))
        a.update(kw)
        B.rope_append_bf16(a["q"], a["k"], a["v"], a["pos"], a["slots"], a["kp"], a["vp"], 1e4, a["qo"])
    with pytest.raises(B.KnapSpecError, match=NOT_CUDA):
        call()
    for kw, text in (({"v": _bf(6, 2, 32)}, "v must have shape"), ({"qo": _bf(6, 8, 32)}, "q_out must"),
                     ({"q": None}, "q and q_out go together"), ({"pos": _i(5)}, "positions must"),
                     ({"kp": _bf(9, 16, 2, 32)}, "k_pages must"), ({"vp": _bf(8, 16, 2, 64)}, "v_pages must"),
                     ({"k": _bf(6, 128)}, r"k must be \[n\]"), ({"q": _bf(5, 8, 64)}, "q must have shape")):
        with pytest.raises(B.KnapSpecError, match=text):
            call(**kw)
    wide = _bf(6, 16, 64)[:, ::2]              # heads that do not lie side by side
    with pytest.raises(B.KnapSpecError, match="side by side"):
        call(q=wide)


def test_attention_shapes():
    def call(**kw):
        a = dict(q=_bf(6, 8, 64), kp=_bf(9, 16, 2, 64), vp=_bf(9, 16, 2, 64), table=_i(3, 4), cu=_i(4),
                 kv=_i(3), out=_bf(6, 8, 64), ws=torch.zeros(1 << 20, dtype=torch.uint8))
        a.update(kw)
        B.paged_attention_bf16(a["q"], a["kp"], a["vp"], a["table"], a["cu"], a["kv"], 2, a["out"], a["ws"])
    with pytest.raises(B.KnapSpecError, match=NOT_CUDA):
        call()
    for kw, text in (({"out": _bf(6, 8, 32)}, "out must"), ({"kp": _bf(9, 16, 2, 32)}, "k_pages must"),
                     ({"vp": _bf(9, 16, 1, 64)}, "v_pages must"), ({"cu": _i(3)}, "cu_new must"),
                     ({"kv": _i(4)}, "kv_len must"), ({"table": _i(12)}, "block_table must be"),
                     ({"q": _bf(6, 512)}, r"q must be \[n\]"), ({"kp": _bf(144, 2, 64)}, "k_pages must")):
        with pytest.raises(B.KnapSpecError, match=text):
            call(**kw)


def _pool(n_pages=10, page_size=16, Hkv=2, hd=64, k=FAKE, v=FAKE):
    return B.PagePool(k, v, n_pages, page_size, Hkv, hd)


INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
POOLS = [(dict(k=None), INVALID), (dict(v=FAKE + 2), INVALID), (dict(n_pages=0), INVALID),
         (dict(page_size=0), INVALID), (dict(Hkv=0), INVALID), (dict(hd=96), UNSUPPORTED),
         (dict(page_size=12), UNSUPPORTED), (dict(n_pages=1 << 27, page_size=16), UNSUPPORTED),
         (dict(Hkv=1 << 20), UNSUPPORTED)]


def test_plan_refusals(lib):
    def call(B_=2, n_free=4, n_pages=10, page=16, max_blocks=4, cap=8, ctx=FAKE, cu=FAKE, table=FAKE,
             free=FAKE, pos=FAKE):
        return lib.ks_page_plan(ctx, FAKE, B_, free, n_free, n_pages, page, table, max_blocks, cap, cu,
                                FAKE, pos, FAKE, FAKE, None, None)
    for kw, code in (({"B_": -1}, INVALID), ({"B_": 16385}, UNSUPPORTED), ({"n_free": -1}, INVALID),
                     ({"n_pages": 0}, INVALID), ({"page": 0}, INVALID), ({"page": 20}, UNSUPPORTED),
                     ({"max_blocks": -1}, INVALID), ({"cap": -1}, INVALID), ({"ctx": None}, INVALID),
                     ({"cu": None}, INVALID), ({"table": None}, INVALID), ({"free": None}, INVALID),
                     ({"pos": None}, INVALID), ({"n_pages": 1 << 28}, UNSUPPORTED),
                     ({"max_blocks": 1 << 27}, UNSUPPORTED)):
        assert call(**kw) == code, kw
        assert b"page plan" in lib.ks_last_error()


def test_append_refusals(lib):
    def call(pool=None, q=FAKE, qs=512, k=FAKE, ks=128, v=FAKE, vs=128, n=3, Hq=8, pos=FAKE, base=1e4,
             qo=FAKE):
        return lib.ks_rope_append_bf16(q, qs, k, ks, v, vs, n, Hq, ctypes.byref(pool or _pool()), pos,
                                       FAKE, base, qo, None, None)
    for kw, code in POOLS:
        assert call(pool=_pool(**kw)) == code, kw
    for kw in ({"n": -1}, {"Hq": 0}, {"q": None}, {"qo": None}, {"k": None}, {"v": None}, {"pos": None},
               {"base": 0.0}, {"base": float("nan")}, {"base": float("inf")}, {"qs": 511}, {"qs": 504},
               {"ks": 120}, {"vs": 0}, {"vs": -128}, {"q": FAKE + 8}, {"k": FAKE + 2}, {"qo": FAKE + 4}):
        assert call(**kw) == INVALID, kw
        assert b"rope append" in lib.ks_last_error()
    assert call(Hq=1 << 20, qs=1 << 26) == UNSUPPORTED
    assert call(n=0) == 0                      # nothing to do: no launch
    assert lib.ks_rope_append_bf16(FAKE, 512, FAKE, 128, FAKE, 128, 3, 8, None, FAKE, FAKE, 1e4, FAKE,
                                   None, None) == INVALID


def test_attention_refusals(lib):
    size = B.paged_attention_workspace_size()
    assert size > 0 and lib.ks_paged_attention_workspace_size(None) == INVALID

    def call(pool=None, q=FAKE, table=FAKE, max_blocks=4, cu=FAKE, kv=FAKE, B_=2, n=3, max_new=2, Hq=8,
             window=0, sinks=0, out=FAKE, ws=FAKE, nbytes=size):
        return lib.ks_paged_attention_bf16(q, ctypes.byref(pool or _pool()), table, max_blocks, cu, kv,
                                           B_, n, max_new, Hq, window, sinks, out, ws, nbytes, None, None)
    for kw, code in POOLS:
        assert call(pool=_pool(**kw)) == code, kw
    for kw, code in (({"B_": -1}, INVALID), ({"B_": 16385}, UNSUPPORTED), ({"n": -1}, INVALID),
                     ({"max_new": -1}, INVALID), ({"Hq": 0}, INVALID), ({"Hq": 7}, INVALID),
                     ({"Hq": 258}, UNSUPPORTED), ({"window": -1}, INVALID), ({"sinks": -1}, INVALID),
                     ({"q": None}, INVALID), ({"out": None}, INVALID), ({"cu": None}, INVALID),
                     ({"kv": None}, INVALID), ({"table": None}, INVALID), ({"ws": None}, INVALID),
                     ({"q": FAKE + 8}, INVALID), ({"out": FAKE + 2}, INVALID), ({"ws": FAKE + 16}, INVALID),
                     ({"nbytes": size - 1}, WORKSPACE), ({"max_blocks": 1 << 27}, UNSUPPORTED),
                     ({"max_blocks": -1}, INVALID)):
        assert call(**kw) == code, kw
        assert b"paged attention" in lib.ks_last_error()
    for kw in ({"B_": 0}, {"n": 0}, {"max_new": 0}):      # nothing to do: no launch
        assert call(**kw) == 0, kw
