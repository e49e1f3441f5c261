"""Sinks, trees, pages and slots refuse what they cannot take before any launch (no GPU needed), and their oracle is pinned."""
import ctypes

import numpy as np
import pytest

from oracle import kv as OK
from tests.test_kv_abi import BAD_CACHE, FAKE, cache, heads, wq  # noqa: F401


@pytest.mark.parametrize("change,status", BAD_CACHE)
def test_bad_caches(wq, change, status):  # noqa: F811
    c, h, want, L, r = cache(wq, **change), heads(wq), getattr(wq, status), wq.lib, ctypes.byref
    assert L.wq_attend_ex(r(c), r(h), r(h), None, 2, 3, 32, FAKE, None, 0, 0.1, 5, 2, None, 8, None, 0, None) == want
    assert L.wq_kv_append_slots(r(c), r(h), r(h), 3, FAKE, None) == want
    assert L.wq_kv_reserve(r(c), FAKE, 9, FAKE, FAKE, 2, FAKE, FAKE, None, 5, FAKE, None, None, None) == want
    assert L.wq_kv_release(r(c), FAKE, 9, FAKE, FAKE, 2, FAKE, None, None) == want
    assert L.wq_kv_keep(r(c), FAKE, 2, FAKE, 3, None, None) == want


def test_bad_attend_arguments(wq):  # noqa: F811
    c, h, L, r = cache(wq), heads(wq), wq.lib, ctypes.byref

    def call(tokens=3, window=5, sinks=2, tree=None, flags=8, **kw):
        t = None if tree is None else r(wq.wq_tree(*tree))
        return L.wq_attend_ex(r(c), r(h), r(h), None, kw.get("batch", 2), tokens, 32, kw.get("lens", FAKE), None, 0, 0.1, window, sinks, t,
                              flags, None, 0, None)

    assert call(sinks=-1) == wq.WQ_ERR_ARG
    assert call(window=0, flags=0) == wq.WQ_ERR_ARG                      # sinks are causal
    assert call(window=0, sinks=0, tree=(FAKE, FAKE, 3, 3), flags=0) == wq.WQ_ERR_ARG   # and so are trees
    assert call(tree=(None, FAKE, 3, 3)) == wq.WQ_ERR_ARG
    assert call(tree=(FAKE, FAKE, -1, 3)) == wq.WQ_ERR_ARG and call(tree=(FAKE, FAKE, 3, -1)) == wq.WQ_ERR_ARG
    assert call(tree=(FAKE + 2, FAKE, 3, 3)) == wq.WQ_ERR_ALIGN and call(tree=(FAKE, FAKE + 1, 3, 3)) == wq.WQ_ERR_ALIGN
    assert call(tokens=1025, tree=(FAKE, None, 0, 0)) == wq.WQ_ERR_SHAPE
    assert call(lens=None) == wq.WQ_ERR_ARG and call(flags=2) == wq.WQ_ERR_ARG and call(window=-1) == wq.WQ_ERR_ARG
    assert call(batch=0) == wq.WQ_OK and call(tokens=0) == wq.WQ_OK


def test_bad_page_arguments(wq):  # noqa: F811
    c, L, r = cache(wq), wq.lib, ctypes.byref

    def reserve(c=c, free=FAKE, size=9, top=FAKE, out=FAKE, batch=2, lens=FAKE, counts=FAKE, granted=None, tokens=5, slots=FAKE, pos=None,
                starts=None):
        return L.wq_kv_reserve(r(c), free, size, top, out, batch, lens, counts, granted, tokens, slots, pos, starts, None)

    def release(c=c, free=FAKE, size=9, top=FAKE, out=FAKE, batch=2, lens=FAKE, keep=None):
        return L.wq_kv_release(r(c), free, size, top, out, batch, lens, keep, None)

    for f in (reserve, release):
        assert f(c=cache(wq, table=None)) == wq.WQ_ERR_ARG
        for name in ("free", "top", "out", "lens"):
            assert f(**{name: None}) == wq.WQ_ERR_ARG
            assert f(**{name: FAKE + 2}) == wq.WQ_ERR_ALIGN
        assert f(size=-1) == wq.WQ_ERR_ARG and f(batch=-1) == wq.WQ_ERR_ARG
        assert f(batch=65537) == wq.WQ_ERR_SHAPE and f(size=2 ** 31) == wq.WQ_ERR_SHAPE
    assert reserve(counts=None) == wq.WQ_ERR_ARG and reserve(tokens=-1) == wq.WQ_ERR_ARG and reserve(granted=FAKE) == wq.WQ_ERR_ARG
    assert reserve(tokens=2 ** 31) == wq.WQ_ERR_SHAPE
    assert reserve(slots=FAKE + 4) == wq.WQ_ERR_ALIGN and reserve(granted=FAKE + 6) == wq.WQ_ERR_ALIGN
    assert reserve(pos=FAKE + 2) == wq.WQ_ERR_ALIGN and reserve(starts=FAKE + 1) == wq.WQ_ERR_ALIGN and reserve(counts=FAKE + 2) == wq.WQ_ERR_ALIGN
    assert release(keep=FAKE + 2) == wq.WQ_ERR_ALIGN


def test_bad_slot_path_and_tree_arguments(wq):  # noqa: F811
    c, h, L, r = cache(wq), heads(wq), wq.lib, ctypes.byref
    assert L.wq_kv_append_slots(r(c), r(h), r(h), -1, FAKE, None) == wq.WQ_ERR_ARG
    assert L.wq_kv_append_slots(r(c), r(h), r(h), 2 ** 31, FAKE, None) == wq.WQ_ERR_SHAPE
    assert L.wq_kv_append_slots(r(c), r(h), r(h), 3, None, None) == wq.WQ_ERR_ARG
    assert L.wq_kv_append_slots(r(c), r(h), r(h), 3, FAKE + 4, None) == wq.WQ_ERR_ALIGN
    assert L.wq_kv_append_slots(r(c), None, r(h), 3, FAKE, None) == wq.WQ_ERR_ARG
    assert L.wq_kv_append_slots(r(c), r(heads(wq, token=1020)), r(h), 3, FAKE, None) == wq.WQ_ERR_ALIGN
    assert L.wq_kv_append_slots(r(c), None, None, 0, None, None) == wq.WQ_OK
    assert L.wq_kv_keep(r(c), None, 2, FAKE, 3, None, None) == wq.WQ_ERR_ARG
    assert L.wq_kv_keep(r(c), FAKE, 2, None, 3, None, None) == wq.WQ_ERR_ARG
    assert L.wq_kv_keep(r(c), FAKE, -2, FAKE, 3, None, None) == wq.WQ_ERR_ARG
    assert L.wq_kv_keep(r(c), FAKE, 2, FAKE, 513, None, None) == wq.WQ_ERR_SHAPE
    assert L.wq_kv_keep(r(cache(wq, table=None)), FAKE, 17, FAKE, 3, None, None) == wq.WQ_ERR_SHAPE
    assert L.wq_kv_keep(r(c), FAKE, 2, FAKE + 2, 3, None, None) == wq.WQ_ERR_ALIGN
    assert L.wq_kv_keep(r(c), None, 0, None, 3, None, None) == wq.WQ_OK and L.wq_kv_keep(r(c), None, 2, None, 0, None, None) == wq.WQ_OK
    assert L.wq_tree_mask(FAKE, 2, 1025, None, 0, FAKE, FAKE, None) == wq.WQ_ERR_SHAPE
    assert L.wq_tree_mask(FAKE, 2, 5, None, -1, FAKE, FAKE, None) == wq.WQ_ERR_ARG
    assert L.wq_tree_mask(None, 2, 5, None, 0, FAKE, FAKE, None) == wq.WQ_ERR_ARG
    assert L.wq_tree_mask(FAKE, 2, 5, None, 0, None, FAKE, None) == wq.WQ_ERR_ARG
    assert L.wq_tree_mask(FAKE, 2, 5, FAKE + 2, 0, FAKE, FAKE, None) == wq.WQ_ERR_ALIGN
    assert L.wq_tree_mask(None, 0, 5, None, 0, None, None, None) == wq.WQ_OK


# ------------------------------------------------------------------ the oracle
def test_oracle_of_trees_by_hand():
    #  0 - 1 - 3
    #    \ 2       4 - 5
    seen, depth = OK.ancestors([-1, 0, 0, 1, -1, 4, 5], 6)
    assert depth.tolist() == [0, 1, 1, 2, 0, 1, 0]
    assert [np.flatnonzero(r).tolist() for r in seen] == [[0], [0, 1], [0, 2], [0, 1, 3], [4], [4, 5], []]
    assert OK.mask_words(seen).tolist() == [[1], [3], [5], [11], [16], [48], [0]]
    near, _ = OK.ancestors([-1, 0, 0, 1, -1, 4, 5], 6, window=2)
    assert np.flatnonzero(near[3]).tolist() == [1, 3]
    wide = np.zeros((1, 40), bool)
    wide[0, [31, 32]] = True
    assert OK.mask_words(wide).tolist() == [[-2 ** 31, 1]]


def test_oracle_of_what_is_visible():
    assert [np.flatnonzero(r).tolist() for r in OK.visible(3, 2, 7, window=2, sinks=1)] == [[0, 4, 5], [0, 5, 6], []]
    nodes, depth = OK.ancestors([-1, 0, 0], 3)
    got = OK.visible(3, 3, 8, window=3, sinks=1, nodes=nodes, depth=depth)
    assert [np.flatnonzero(r).tolist() for r in got] == [[0, 3, 4, 5], [0, 4, 5, 6], [0, 4, 5, 7]]
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((4, 2, 8)), rng.standard_normal((9, 1, 8)), rng.standard_normal((9, 1, 8))
    a, b = OK.attend(q, k, v, 4, 0.3, True, 5), OK.attend_seen(q, k, v, OK.visible(4, 4, 9, window=5), 0.3)
    assert all(np.allclose(x, y) for x, y in zip(a, b))


# ------------------------------------------------------------------ the binding
def test_the_binding_refuses_host_memory_and_wrong_arguments(wq):  # noqa: F811
    torch = pytest.importorskip("torch")
    c = cache(wq)
    lead = (ctypes.addressof(c), c.heads, c.dim, 2, 0, 0)
    ints, rows, k = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 3, 8, 128).bfloat16(), torch.zeros(3, 8, 128).bfloat16()
    calls = wq._calls
    for call in (lambda: calls.attend(*lead, rows, ints, None, True, 0, None, 0, None, False, False, None, 1, None, None),
                 lambda: calls.append(*lead, rows, rows, None, None), lambda: calls.append_slots(*lead, k, k, torch.zeros(3, dtype=torch.int64)),
                 lambda: calls.read(*lead, 5, ints, None, False, 2), lambda: calls.reserve(*lead, ints, ints[:1], ints, ints, 5, None, None),
                 lambda: calls.release(*lead, ints, ints[:1], ints, None, None), lambda: calls.keep(*lead, ints, torch.zeros(2, 3, dtype=torch.int32), None),
                 lambda: calls.tree_mask(0, 0, 0, 0, 0, 0, torch.zeros(2, 3, dtype=torch.int32), None, 0),
                 lambda: calls.attend(*lead, rows[0], ints, None, True, 0, None, 0, None, False, False, None, 1, None, None),
                 lambda: calls.append(*lead, rows[..., :64], rows[..., :64], None, None), lambda: calls.append(*lead, "k", rows, None, None),
                 lambda: calls.append(*lead, rows.expand(2, 3, 8, 128), rows[:1], None, None)):
        with pytest.raises(AssertionError):
            call()
    for call in (lambda: calls.append(*lead, rows, rows, None), lambda: calls.tree_mask(), lambda: calls.bind(1, 2)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(TypeError):
        calls.tree_mask(0, 0, 0, 0, 0, 0, torch.zeros(2, 3, dtype=torch.int32), None, "wide")
