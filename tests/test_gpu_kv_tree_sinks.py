"""Drafted trees behind a window with sinks see what decoding their paths token by token would, also where the context is
shorter than the sinks, so that drafted tokens are sinks themselves."""
import numpy as np
import pytest
import torch

from oracle import kv as OK
from tests.gpu_common import need_gpu, wq
from tests.helpers import rel_l2
from tests.test_gpu_kv_cache import F32_REL_L2, Case, bf16, ints
from tests.test_gpu_kv_select import check, cuda, random_trees

pytestmark = pytest.mark.gpu
FMTS = pytest.mark.parametrize("fmt", ["q4_0", "nvfp4"])


@pytest.mark.parametrize("tokens", [1, 2, 8, 31, 32, 33, 100, 1024])
@pytest.mark.parametrize("window,sinks", [(0, 9), (1, 0), (1, 1), (3, 4), (3, 40), (40, 41), (16, 10 ** 12), (10 ** 12, 5)])
def test_tree_mask_with_sinks(tokens, window, sinks):
    need_gpu()
    m, rng = wq(), np.random.default_rng(tokens)
    parents = random_trees(rng, 8, tokens, int(rng.integers(1, 5)))
    parents[:4] = np.arange(tokens) - 1                                  # chains
    counts = [tokens, tokens, max(1, tokens // 2), tokens, tokens, 0, tokens + 9, tokens]
    n = [min(max(c, 0), tokens) for c in counts]
    bases = [0, 2, 1, 38, 3, 7, 30, 2 ** 31 - 1 - tokens]
    lens = [x + y for x, y in zip(bases, n)]
    mask, depth = m.tree_mask(cuda(parents), ints(counts), window=window, sinks=sinks, lens=ints(lens))
    for b in range(8):
        seen, d = OK.ancestors(parents[b], n[b], window, sinks, bases[b])
        assert np.array_equal(mask[b].cpu().numpy(), OK.mask_words(seen)) and np.array_equal(depth[b].cpu().numpy(), d)
    assert m.last_device_status() == 0


def test_lengths_below_the_draft():
    """A length of less than the draft, or below zero, puts its first nodes before the first position."""
    need_gpu()
    m, chain = wq(), torch.arange(-1, 7, dtype=torch.int32, device="cuda").expand(2, -1).contiguous()
    mask, _ = m.tree_mask(chain, window=2, sinks=1, lens=ints([5, -3]))
    for b, base in ((0, -3), (1, -8)):
        assert np.array_equal(mask[b].cpu().numpy(), OK.mask_words(OK.ancestors(np.arange(8) - 1, 8, 2, 1, base)[0]))
    assert m.last_device_status() == 0


@pytest.mark.parametrize("window,sinks", [(3, 0), (0, 4), (0, 0)])
def test_a_window_or_sinks_alone_look_at_no_length(window, sinks):
    need_gpu()
    m, parents = wq(), cuda(random_trees(np.random.default_rng(7), 3, 40, 2))
    want = m.tree_mask(parents, window=window)
    for lens in (None, ints([40, 3, -9]), ints([45, 2 ** 31 - 1, 0])):
        got = m.tree_mask(parents, window=window, sinks=sinks, lens=lens)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        if lens is not None and sinks == 0:
            for b, n in enumerate(lens.tolist()):
                seen, depth = OK.ancestors(parents[b].tolist(), 40, window, sinks, max(n, 0) - 40)
                assert np.array_equal(got[0][b].cpu().numpy(), OK.mask_words(seen)) and np.array_equal(got[1][b].cpu().numpy(), depth)
    assert m.last_device_status() == 0


@FMTS
@pytest.mark.parametrize("D,hq", [(64, 4), (128, 8)])
@pytest.mark.parametrize("tokens", [5, 8, 40, 150])
@pytest.mark.parametrize("window,sinks", [(3, 4), (3, 30), (33, 60), (16, 200)])
def test_a_chain_is_causal_attention_with_sinks(fmt, D, hq, tokens, window, sinks):
    """Node i below node i - 1 behind contexts of 2, 25 and 250 tokens: what attention without a tree gives."""
    need_gpu()
    m, case = wq(), Case(110, fmt, 2, D, 3, 400, 16)
    contexts = [2, 25, 250]
    cache, lens = case.upload(), ints([c + tokens for c in contexts])
    q = bf16(case.rng, 3, tokens, hq, D).cuda()
    chain = torch.arange(-1, tokens - 1, dtype=torch.int32, device="cuda").expand(3, -1).contiguous()
    tree = m.tree_mask(chain, window=window, sinks=sinks, lens=lens)
    args = dict(window=window, sinks=sinks, return_lse=True, out_f32=True)
    got, lse = m.attend(cache, q, lens, tree=tree, **args)
    want, wlse = m.attend(cache, q, lens, **args)
    # both calls have the same rows, so they take the same kernel: equal sums, whose running maximum may be another one
    assert torch.allclose(lse, wlse, rtol=0, atol=2e-5)
    assert rel_l2(got.cpu().numpy(), want.cpu().numpy()) <= F32_REL_L2 and m.last_device_status() == 0


@FMTS
@pytest.mark.parametrize("tokens,hq,h,D", [(7, 8, 2, 128), (20, 4, 4, 64), (40, 8, 2, 128), (100, 4, 1, 64)])
@pytest.mark.parametrize("window,sinks", [(2, 6), (5, 40), (40, 130)])
def test_trees_whose_nodes_are_sinks(fmt, tokens, hq, h, D, window, sinks):
    need_gpu()
    m, contexts = wq(), [0, 3, 33, 120]
    case = Case(111, fmt, h, D, 4, 120 + tokens, 16)
    parents = random_trees(case.rng, 4, tokens, 2)
    counts, lens = [tokens, tokens - 1, tokens, tokens], [c + tokens for c in contexts]
    lens[1] -= 1
    nodes, depth = zip(*(OK.ancestors(p, n, window, sinks, c) for p, n, c in zip(parents, counts, contexts)))
    check(case, tokens, hq, lens, counts, window=window, sinks=sinks, nodes=np.stack(nodes), depth=np.stack(depth))
    mask, _ = m.tree_mask(cuda(parents), ints(counts), window=window, sinks=sinks, lens=ints(lens))
    assert np.array_equal(mask.cpu().numpy(), OK.mask_words(np.stack(nodes)))


def test_replayed_with_other_lengths_and_refusals():
    need_gpu()
    m, rng = wq(), np.random.default_rng(6)
    parents, lens = cuda(random_trees(rng, 2, 40, 2)), ints([40, 45])
    m.tree_mask(parents, window=3, sinks=8, lens=lens)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mask, depth = m.tree_mask(parents, window=3, sinks=8, lens=lens)
    for base in ([0, 5], [4, 60]):
        lens.copy_(ints([40 + x for x in base]))
        g.replay()
        for b in range(2):
            seen, d = OK.ancestors(parents[b].tolist(), 40, 3, 8, base[b])
            assert np.array_equal(mask[b].cpu().numpy(), OK.mask_words(seen)) and np.array_equal(depth[b].cpu().numpy(), d)
    launches = m.lib.wq_kernel_launches()
    for bad in (dict(window=3, sinks=8), dict(window=3, sinks=-1, lens=lens)):
        with pytest.raises(m.WQError):
            m.tree_mask(parents, **bad)
    for bad in (lens.cpu(), lens[:1], lens.long()):
        with pytest.raises(AssertionError):
            m.tree_mask(parents, window=3, sinks=8, lens=bad)
    assert m.lib.wq_kernel_launches() == launches and m.last_device_status() == 0
