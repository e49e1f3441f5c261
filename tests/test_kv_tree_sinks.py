"""Trees behind a window with sinks: the oracle against decoding every path token by token, and the entry point's refusals
(no GPU needed)."""
import numpy as np
import pytest

from oracle import kv as OK
from tests.test_kv_abi import FAKE, wq  # noqa: F401


def token_by_token(path, base, window, sinks):
    """Positions (context) and nodes that the last token of `path` sees when the path is decoded behind `base` tokens."""
    row = np.flatnonzero(OK.visible(1, 1, base + len(path), window, sinks)[0])
    return set(row[row < base].tolist()), {path[t - base] for t in row if t >= base}


def test_a_chain_behind_a_short_context_by_hand():
    nodes, depth = OK.ancestors(np.arange(8) - 1, 8, 3, 4, 2)
    assert np.flatnonzero(OK.visible(8, 8, 10, 3, 4, nodes, depth)[7]).tolist() == [0, 1, 2, 3, 7, 8, 9]


@pytest.mark.parametrize("seed", range(20))
def test_the_mask_of_a_tree_is_decoding_its_paths(seed):
    rng = np.random.default_rng(seed)
    for _ in range(10):
        n, base = int(rng.integers(1, 20)), int(rng.integers(0, 12))
        window, sinks = int(rng.integers(0, 8)), int(rng.integers(0, 16))
        parents = np.array([rng.integers(max(-1, i - 3), i) for i in range(n)], np.int32)
        nodes, depth = OK.ancestors(parents, n, window, sinks, base)
        seen = OK.visible(n, n, base + n, window, sinks, nodes, depth)
        for i in range(n):
            path = [i]
            while parents[path[0]] >= 0:
                path.insert(0, int(parents[path[0]]))
            row = np.flatnonzero(seen[i])
            assert (set(row[row < base].tolist()), set((row[row >= base] - base).tolist())) == token_by_token(path, base, window, sinks)


def test_bad_arguments(wq):  # noqa: F811
    def mask(parents=FAKE, batch=2, tokens=5, counts=None, window=3, sinks=2, lens=FAKE, mask=FAKE, depth=FAKE):
        return wq.lib.wq_tree_mask_ex(parents, batch, tokens, counts, window, sinks, lens, mask, depth, None)

    assert mask(sinks=-1) == wq.WQ_ERR_ARG and mask(window=-1) == wq.WQ_ERR_ARG and mask(lens=None) == wq.WQ_ERR_ARG
    assert mask(parents=None) == wq.WQ_ERR_ARG and mask(mask=None) == wq.WQ_ERR_ARG and mask(batch=-1) == wq.WQ_ERR_ARG
    assert mask(tokens=1025) == wq.WQ_ERR_SHAPE and mask(batch=2 ** 31) == wq.WQ_ERR_SHAPE
    for name in ("parents", "counts", "lens", "mask", "depth"):
        assert mask(**{name: FAKE + 2}) == wq.WQ_ERR_ALIGN
    assert mask(batch=0, lens=None, sinks=0) == wq.WQ_OK and mask(tokens=0) == wq.WQ_OK
