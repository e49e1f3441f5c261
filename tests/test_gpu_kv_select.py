"""Attention over the 4-bit KV cache with sinks behind a window, and of trees of drafted tokens, against fp64.

The arithmetic is wq_attend's, so are the bounds (tests/test_gpu_kv_cache.py): with A the largest sum of |scale q k| that a row
sees, |out - ref| <= (2^-11 (2 A + 4) + 2^-20) sum p |v| and |lse - ref| <= 2^-11 A + 2^-20 |ref| + 2^-20 for the fp32 output, and
the bf16 output is that one rounded."""
import numpy as np
import pytest
import torch

from oracle import kv as OK
from tests.gpu_common import need_gpu, wq
from tests.helpers import rel_l2
from tests.test_gpu_kv_cache import Case, F32_REL_L2, bf16, ints

pytestmark = pytest.mark.gpu
FMTS = pytest.mark.parametrize("fmt", ["q4_0", "nvfp4"])


def random_trees(rng, batch, tokens, reach=4):
    """Parents [batch, tokens]: below one of the last few nodes, now and then a root."""
    out = np.full((batch, tokens), -1, np.int32)
    for i in range(1, tokens):
        out[:, i] = np.where(rng.random(batch) < 0.1, -1, rng.integers(max(0, i - reach), i, batch))
    return out


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def check(case, tokens, q_heads, lens, counts=None, window=0, sinks=0, nodes=None, depth=None, q_std=1.0, max_len=0, exact=True):
    """nodes: bool [batch or 1, tokens, tokens] and depth int [batch or 1, tokens] or None."""
    m, B, D = wq(), case.batch, case.D
    cache = case.upload()
    q = bf16(case.rng, B, tokens, q_heads, D, std=q_std)
    tree = None if nodes is None else (cuda(OK.mask_words(nodes)), None if depth is None else cuda(depth.astype(np.int32)))
    args = dict(counts=None if counts is None else ints(counts), window=window, sinks=sinks, tree=tree, return_lse=True, max_len=max_len)
    got, lse = m.attend(cache, q.cuda(), ints(lens), out_f32=True, **args)
    got16, lse16 = m.attend(cache, q.cuda(), ints(lens), **args)
    assert m.last_device_status() == 0
    assert torch.equal(lse, lse16) and torch.equal(got.bfloat16(), got16)
    got, lse = got.cpu().double().numpy(), lse.cpu().double().numpy()
    refs = []
    for b in range(B):
        n = tokens if counts is None else min(max(counts[b], 0), tokens)
        T = max(0, lens[b])
        at = lambda x: None if x is None else x[b if len(x) == B else 0]  # noqa: E731
        seen = OK.visible(tokens, n, T, window, sinks, at(nodes), at(depth))
        k, v = case.values(b, T)
        ref, rlse, mean, top = OK.attend_seen(q[b].float().numpy(), k, v, seen, D ** -0.5)
        refs.append(ref)
        empty = np.isneginf(rlse)
        assert np.array_equal(np.isneginf(lse[b]), empty) and not got[b][empty].any()
        bound = (2.0 ** -11 * (2 * top[..., None] + 4) + 2.0 ** -20) * mean
        assert np.all(np.abs(got[b] - ref) <= bound + 1e-30), np.max(np.abs(got[b] - ref) / (bound + 1e-30))
        ok = ~empty
        assert np.all(np.abs(lse[b][ok] - rlse[ok]) <= 2.0 ** -11 * top[ok] + 2.0 ** -20 * np.abs(rlse[ok]) + 2.0 ** -20)
    if exact and np.linalg.norm(np.stack(refs)) > 0:
        assert rel_l2(got, np.stack(refs)) <= F32_REL_L2


# ------------------------------------------------------------------ sinks
@FMTS
@pytest.mark.parametrize("hq,h,D,page", [(8, 2, 128, 16), (4, 4, 64, 0), (6, 1, 128, 48), (33, 3, 64, 32)])
@pytest.mark.parametrize("window,sinks", [(1, 1), (15, 4), (64, 33), (100, 200), (40, 10 ** 12), (7, 128)])
def test_one_token(fmt, hq, h, D, page, window, sinks):
    need_gpu()
    lens = [333, 1, 2, 16, 65, 0, 129, 200]
    check(Case(60, fmt, h, D, len(lens), 333, page), 1, hq, lens, window=window, sinks=sinks)


@FMTS
@pytest.mark.parametrize("window,sinks", [(1, 3), (20, 1), (64, 64), (130, 150), (10 ** 6, 5)])
@pytest.mark.parametrize("tokens,hq,h,D", [(6, 8, 2, 128), (12, 3, 3, 64), (20, 3, 3, 128), (150, 4, 2, 64), (140, 2, 1, 128), (300, 1, 1, 64)])
def test_several_tokens_ragged(fmt, window, sinks, tokens, hq, h, D):
    need_gpu()
    lens, counts = [433, max(90, tokens), 40, 0, tokens], [tokens, tokens // 2, tokens, tokens, 0]
    check(Case(61, fmt, h, D, 5, 433, 16), tokens, hq, lens, counts, window=window, sinks=sinks)


@FMTS
def test_no_window_or_no_sinks_is_plain_attention(fmt):
    """The same bits as without the arguments."""
    need_gpu()
    m, case = wq(), Case(62, fmt, 2, 128, 2, 300, 16)
    cache, lens = case.upload(), ints([300, 77])
    for tokens in (1, 40):
        q = bf16(case.rng, 2, tokens, 8, 128).cuda()
        for window in (0, 50):
            want = m.attend(cache, q, lens, window=window, return_lse=True)
            got = m.attend(cache, q, lens, window=window, sinks=9 if window == 0 else 0, return_lse=True)
            assert all(torch.equal(a, b) for a, b in zip(want, got))


@FMTS
def test_long_sequences_and_shared_tokens(fmt):
    """Windows that are split over blocks and joined, sinks of several tiles, a plan from a bound."""
    need_gpu()
    check(Case(63, fmt, 1, 128, 1, 30011, 64), 1, 4, [30011], window=9001, sinks=130)
    check(Case(64, fmt, 2, 64, 2, 9000, 16), 3, 8, [9000, 513], window=6000, sinks=77)
    check(Case(65, fmt, 1, 64, 2, 6000, 0), 1, 1, [6000, 3], window=900, sinks=4, max_len=6000)
    check(Case(66, fmt, 1, 128, 1, 5000, 32), 130, 2, [5000], window=2100, sinks=300)
    check(Case(67, fmt, 3, 128, 1, 5000, 32), 70, 3, [4990], window=64, sinks=1)


@FMTS
@pytest.mark.parametrize("tokens,hq,h,D,batch", [(1, 8, 8, 64, 31), (1, 32, 8, 128, 40), (3, 16, 4, 128, 40), (7, 12, 3, 64, 60), (2, 7, 7, 128, 129)])
@pytest.mark.parametrize("longest", [20, 150, 700])
def test_many_sequences_of_very_unequal_lengths(fmt, tokens, hq, h, D, batch, longest):
    """More items than places: runs that begin and end inside items, items of many runs, sequences of nothing between them."""
    need_gpu()
    rng = np.random.default_rng(batch)
    lens = [int(x) for x in rng.integers(0, 1 + longest // 8, batch)]
    lens[batch // 3], lens[-1], lens[batch // 2] = longest, longest - 3, 0
    counts = [int(x) for x in rng.integers(0, tokens + 1, batch)]
    check(Case(78, fmt, h, D, batch, longest, 16), tokens, hq, lens, window=longest // 2, sinks=5)
    case = Case(79, fmt, h, D, batch, longest, 32)
    nodes, depth = zip(*(OK.ancestors(p, tokens) for p in random_trees(case.rng, batch, tokens)))
    lens = [max(x, tokens) for x in lens]
    check(case, tokens, hq, lens, counts, nodes=np.stack(nodes), depth=np.stack(depth))
    check(case, tokens, hq, lens, counts, window=max(3, longest // 3), sinks=70, nodes=np.stack(nodes), depth=np.stack(depth))


@FMTS
@pytest.mark.parametrize("tokens", [1, 5, 140])
def test_tokens_between_sinks_and_window_are_not_read(fmt, tokens):
    """Their pages hold NaN, or are not there at all: nothing changes, nothing is reported."""
    need_gpu()
    m, case = wq(), Case(68, fmt, 2, 128, 2, 800, 128)
    cache, lens = case.upload(), ints([800, 790])
    q = bf16(case.rng, 2, tokens, 8, 128).cuda()
    want = m.attend(cache, q, lens, window=90, sinks=5, return_lse=True)
    cache.tensors[4][:, 1:4] = ints([10 ** 6, -1, 2 ** 31 - 1])     # positions 128 .. 511
    got = m.attend(cache, q, lens, window=90, sinks=5, return_lse=True)
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and m.last_device_status() == 0


def test_sinks_where_the_length_passes_the_capacity():
    """Query rows keep their positions: windows past the capacity see nothing, sinks stay."""
    need_gpu()
    m, case = wq(), Case(69, "q4_0", 1, 64, 1, 96, 16)
    cache = case.upload()
    for tokens in (1, 40):
        q = bf16(case.rng, 1, tokens, 1, 64)
        out, lse = m.attend(cache, q.cuda(), ints([500]), window=20, sinks=90, return_lse=True, out_f32=True)
        assert m.last_device_status() == m.WQ_ERR_ARG
        k, v = case.values(0, 96)
        seen = np.zeros((tokens, 96), bool)
        seen[:, :90] = True
        ref, rlse, *_ = OK.attend_seen(q[0].float().numpy(), k, v, seen, 0.125)
        assert rel_l2(out[0].cpu().numpy(), ref) <= F32_REL_L2 and np.allclose(lse[0].cpu().numpy(), rlse, atol=1e-2)


# ------------------------------------------------------------------ trees
@FMTS
@pytest.mark.parametrize("hq,h,D,page", [(8, 2, 128, 16), (4, 4, 64, 0), (6, 1, 128, 48), (16, 1, 64, 32)])
@pytest.mark.parametrize("tokens", [1, 2, 7, 16, 31, 33, 64])
def test_trees(fmt, hq, h, D, page, tokens):
    need_gpu()
    case = Case(70, fmt, h, D, 5, 333, page)
    nodes, depth = zip(*(OK.ancestors(p, tokens) for p in random_trees(case.rng, 5, tokens)))
    lens = [333, tokens, 200, 64 + tokens // 2, max(tokens - 3, 0)]     # the last: some nodes lie before the first position
    check(case, tokens, hq, lens, [tokens, tokens, max(1, tokens // 2), tokens, tokens], nodes=np.stack(nodes), depth=np.stack(depth))


@FMTS
@pytest.mark.parametrize("tokens,hq,h,D", [(5, 8, 2, 128), (24, 4, 4, 64), (40, 8, 2, 128), (100, 4, 1, 64), (300, 2, 2, 64)])
@pytest.mark.parametrize("window,sinks", [(5, 0), (40, 3), (130, 140), (10 ** 9, 1)])
def test_trees_behind_a_window(fmt, tokens, hq, h, D, window, sinks):
    need_gpu()
    case = Case(71, fmt, h, D, 3, 520, 16)
    nodes, depth = zip(*(OK.ancestors(p, tokens, window) for p in random_trees(case.rng, 3, tokens, 2)))
    check(case, tokens, hq, [520, tokens, max(300, tokens)], [tokens, tokens, tokens - 1], window=window, sinks=sinks,
          nodes=np.stack(nodes), depth=np.stack(depth))
    check(case, tokens, hq, [520, tokens, max(300, tokens)], window=window, sinks=sinks, nodes=np.stack(nodes))   # depths in order


@FMTS
@pytest.mark.parametrize("tokens", [9, 45])
def test_any_bits_and_rows_that_see_nothing(fmt, tokens):
    """Masks that are no tree's: random bits, later nodes too, rows without a bit behind an empty context."""
    need_gpu()
    case = Case(72, fmt, 2, 64, 3, 300, 16)
    nodes = case.rng.random((3, tokens, tokens)) < 0.3
    nodes[:, 2] = False
    nodes[1, 4] = True
    check(case, tokens, 4, [tokens, tokens, 200], nodes=nodes)
    check(case, tokens, 4, [tokens, tokens - 1, 200], nodes=nodes[:1])          # one tree for all
    check(case, tokens, 4, [tokens, 100, 200], nodes=nodes[:1], window=3, sinks=1)


@FMTS
def test_a_chain_is_causal_attention(fmt):
    """Node i below node i - 1: the bits of causal attention, with a window too."""
    need_gpu()
    m, case = wq(), Case(73, fmt, 2, 128, 2, 400, 16)
    cache, lens = case.upload(), ints([400, 150])
    for tokens in (1, 5, 70, 150):
        q = bf16(case.rng, 2, tokens, 8, 128).cuda()
        for window in (0, 33, 140):
            parents = torch.arange(-1, tokens - 1, dtype=torch.int32, device="cuda").expand(2, -1).contiguous()
            tree = m.tree_mask(parents, window=window)
            got = m.attend(cache, q, lens, window=window, tree=tree, return_lse=True, out_f32=True)
            want = m.attend(cache, q, lens, window=window, return_lse=True, out_f32=True)
            # The same sums; tiles that one of the two masks and the other leaves out may order the running maximum otherwise.
            # q4_0 trees of 17 to 32 rows go to the kernel that rounds (c - 8) d to 11 bits, the tokens to the one that does
            # not: each score then moves by 2^-12 of sum |scale q k| at most, and a log-sum-exp by no more than its scores.
            off = 0.0
            if fmt == "q4_0" and 16 < tokens * 4 <= 32:
                off = 2.0 ** -12 * max(OK.attend_seen(q[b].float().cpu().numpy(), *case.values(b, n), np.ones((tokens, n), bool), 128 ** -0.5)[3].max()
                                       for b, n in ((0, 400), (1, 150)))
            assert torch.allclose(got[1], want[1], rtol=0, atol=2e-5 + off)
            assert rel_l2(got[0].cpu().numpy(), want[0].cpu().numpy()) <= F32_REL_L2
    assert m.last_device_status() == 0


@FMTS
def test_long_contexts_of_trees(fmt):
    need_gpu()
    case = Case(74, fmt, 1, 128, 1, 20011, 64)
    nodes, depth = OK.ancestors(random_trees(case.rng, 1, 7)[0], 7)
    check(case, 7, 4, [20011], nodes=nodes[None], depth=depth[None])
    case = Case(75, fmt, 2, 64, 2, 7000, 16)
    nodes, depth = zip(*(OK.ancestors(p, 50) for p in random_trees(case.rng, 2, 50)))
    check(case, 50, 8, [7000, 4099], [50, 41], nodes=np.stack(nodes), depth=np.stack(depth))
    check(case, 50, 8, [7000, 4099], [50, 41], nodes=np.stack(nodes), depth=np.stack(depth), window=1000, sinks=100)


@FMTS
@pytest.mark.parametrize("tokens,hq,n", [(5, 4, 9000), (30, 8, 700)])
def test_other_streams_graphs_and_workspaces(fmt, tokens, hq, n):
    """Equal bits from call to call, on another stream, and replayed with other trees, lengths and counts."""
    need_gpu()
    m, case = wq(), Case(76, fmt, 2, 128, 2, n, 16)
    cache, lens, counts = case.upload(), ints([n, n - 100]), ints([tokens, tokens - 1])
    q = bf16(case.rng, 2, tokens, hq, 128).cuda()
    parents = cuda(random_trees(case.rng, 2, tokens))
    args = dict(counts=counts, window=n // 2, sinks=40)
    ws = torch.full((max(16, m.attend_workspace_bytes(cache, 2, tokens, hq, select=True)),), 0xFF, dtype=torch.uint8, device="cuda")
    step = lambda **kw: m.attend(cache, q, lens, tree=m.tree_mask(parents, counts, window=n // 2), **args, **kw)  # noqa: E731
    want = step().clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert torch.equal(step(workspace=ws), want)
    torch.cuda.current_stream().wait_stream(side)
    out, g = torch.empty_like(q), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(out=out, workspace=ws)
    g.replay()
    assert torch.equal(out, want)
    parents.copy_(cuda(random_trees(case.rng, 2, tokens, 2)))
    lens.sub_(61)
    counts.sub_(1)
    g.replay()
    assert torch.equal(out, step()) and m.last_device_status() == 0


def test_a_bad_scale_of_v_reaches_only_rows_that_see_it():
    """A drafted node whose V scale is NaN, in both kernels: siblings' rows keep their bits."""
    need_gpu()
    for fmt, bits in (("q4_0", 0x7E00), ("nvfp4", 0x7F)):
        for tokens, group in ((6, 2), (40, 2)):
            m, case = wq(), Case(77, fmt, 2, 64, 1, 200, 16)
            nodes, depth = OK.ancestors(random_trees(case.rng, 1, tokens)[0], tokens)
            cache, q = case.upload(), bf16(case.rng, 1, tokens, 2 * group, 64).cuda()
            tree = (cuda(OK.mask_words(nodes[None])), None)
            args = dict(tree=tree, out_f32=True, return_lse=True)
            clean, clse = m.attend(cache, q, ints([190]), **args)
            page, off = case.at(0, 190 - tokens + 3)                       # node 3, head 1
            t = case.t[3].view(torch.int16) if fmt == "q4_0" else case.t[3]
            t[int(page), 1, int(off), 1] = bits
            got, lse = m.attend(cache, q, ints([190]), **args)
            hit = torch.zeros(1, tokens, 2 * group, dtype=torch.bool, device="cuda")
            hit[0, :, group:] = cuda(nodes[:, 3])[:, None]
            assert hit.any() and not hit.all()
            assert torch.equal(got[~hit], clean[~hit]) and torch.equal(lse[~hit], clse[~hit])
            assert not torch.isfinite(got[hit]).all(-1).any()


def test_offsets_past_32_bits():
    """Code arrays of more than 2^32 bytes each, sinks and drafted nodes at both ends."""
    need_gpu()
    m = wq()
    pages, H, D, size = 70000, 8, 128, 128
    table = torch.tensor([[pages - 3, 0, pages - 1, 33]], dtype=torch.int32, device="cuda")
    cache = m.kv_alloc("q4_0", pages, size, H, D, table)
    x = bf16(np.random.default_rng(50), 1, 400, H, D)
    m.kv_append(cache, x.cuda(), x.cuda())
    rows = OK.decode_rows("q4_0", *OK.encode_rows("q4_0", x[0].float().numpy()))
    for tokens in (3, 40):
        nodes, depth = OK.ancestors(random_trees(np.random.default_rng(1), 1, tokens)[0], tokens)
        q = bf16(np.random.default_rng(51), 1, tokens, H, D)
        out = m.attend(cache, q.cuda(), ints([400]), window=100, sinks=5, tree=(cuda(OK.mask_words(nodes[None])), cuda(depth[None])),
                       out_f32=True)
        ref, *_ = OK.attend_seen(q[0].float().numpy(), rows, rows, OK.visible(tokens, tokens, 400, 100, 5, nodes, depth), D ** -0.5)
        assert rel_l2(out[0].cpu().numpy(), ref) <= F32_REL_L2
    assert m.last_device_status() == 0


# ------------------------------------------------------------------ more blocks than places, and what the plans do with them
class Shared(Case):
    """`batch` sequences over the same pages, in orders of their own (only read)."""

    def __init__(self, seed, fmt, heads, D, batch, capacity, page):
        super().__init__(seed, fmt, heads, D, 1, capacity, page)
        self.batch, per = batch, self.table.shape[1]
        self.table = np.stack([self.rng.permutation(self.pages)[:per] for _ in range(batch)]).astype(np.int32)


@FMTS
@pytest.mark.parametrize("batch", [255, 256, 257])
def test_as_many_sequences_as_are_sorted_and_one_more(fmt, batch):
    need_gpu()
    rng = np.random.default_rng(batch)
    lens = [int(x) for x in rng.integers(0, 130, batch)]
    check(Shared(90, fmt, 2, 64, batch, 160, 16), 1, 2, lens, window=50, sinks=3)
    lens[7] = lens[100] = 160
    check(Shared(91, fmt, 2, 64, batch, 160, 16), 1, 4, lens, [int(x) for x in rng.integers(0, 2, batch)], window=70, sinks=20)


@FMTS
@pytest.mark.parametrize("batch,tokens,hq,h,D", [(80, 40, 8, 4, 64), (45, 40, 16, 4, 128), (160, 9, 8, 2, 128)])
def test_many_trees_of_many_rows(fmt, batch, tokens, hq, h, D):
    """One and two groups of rows a block, sequences of few nodes among those of many."""
    need_gpu()
    case = Shared(92, fmt, h, D, batch, 300, 32)
    nodes, depth = zip(*(OK.ancestors(p, tokens) for p in random_trees(case.rng, batch, tokens)))
    lens = [int(x) for x in case.rng.integers(tokens, 300, batch)]
    counts = [int(x) for x in case.rng.integers(0, tokens + 1, batch)]
    check(case, tokens, hq, lens, counts, nodes=np.stack(nodes), depth=np.stack(depth))
    check(case, tokens, hq, lens, counts, window=60, sinks=9, nodes=np.stack(nodes))


@FMTS
@pytest.mark.parametrize("tokens,hq,h", [(1, 16, 4), (2, 8, 4), (4, 8, 2)])
def test_long_sequences_in_two_parts(fmt, tokens, hq, h):
    """More items than half of the places, and a cache for more than 4096 tokens a sequence: parts that some sequences fill
    and others leave empty."""
    need_gpu()
    batch = 116 if h == 2 else 58
    case = Shared(93, fmt, h, 128, batch, 4300, 64)
    lens = [int(x) for x in case.rng.integers(tokens, 90, batch)]
    lens[3], lens[20], lens[21] = 4300, 4177, 0
    check(case, tokens, hq, lens, window=4200, sinks=5)
    nodes, depth = zip(*(OK.ancestors(p, tokens) for p in random_trees(case.rng, batch, tokens)))
    lens[21] = tokens
    check(case, tokens, hq, lens, nodes=np.stack(nodes), depth=np.stack(depth))


@FMTS
@pytest.mark.parametrize("D,heads,batch,tokens,q_heads", [(64, 1, 1, 1, 1), (128, 2, 1, 3, 8), (64, 38, 4, 1, 38), (128, 1, 3, 20, 1), (128, 2, 1, 40, 4),
                                                          (64, 1, 2, 150, 2), (128, 4, 60, 1, 8), (128, 2, 40, 70, 2)])
def test_nothing_is_written_past_the_workspace(fmt, D, heads, batch, tokens, q_heads):
    """attend_workspace_bytes(select=True) is enough for every window, number of sinks and tree."""
    need_gpu()
    m, n = wq(), 6400
    case = Shared(94, fmt, heads, D, batch, n, 64)
    cache, q = case.upload(), bf16(case.rng, batch, tokens, q_heads, D).cuda()
    lens = ints([n - 17 * b for b in range(batch)])
    nodes, depth = OK.ancestors(random_trees(case.rng, 1, tokens)[0], tokens)
    tree = (cuda(OK.mask_words(nodes[None])), cuda(depth[None]))
    need = m.attend_workspace_bytes(cache, batch, tokens, q_heads, select=True)
    assert need >= m.attend_workspace_bytes(cache, batch, tokens, q_heads)
    guarded = torch.full((need + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
    for window, sinks, t in ((0, 0, tree), (1, 1, None), (300, 5000, None), (1500, 4, tree), (4000, 100, None), (4095, 1, None), (5000, 64, tree),
                             (10 ** 9, 3, None)):
        args = dict(window=window, sinks=sinks, tree=t)
        want = m.attend(cache, q, lens, **args)
        got = m.attend(cache, q, lens, workspace=guarded[4096:4096 + need], **args)
        assert torch.equal(got, want)
        assert (guarded[:4096] == 0xA5).all() and (guarded[4096 + need:] == 0xA5).all()
    assert m.last_device_status() == 0


# ------------------------------------------------------------------ what buffers may hold, and how calls may be made
@FMTS
@pytest.mark.parametrize("tokens", [5, 40])
def test_depths_of_any_value(fmt, tokens):
    """Depths outside the draft are clamped to it."""
    need_gpu()
    case = Case(95, fmt, 2, 64, 2, 300, 16)
    nodes, _ = zip(*(OK.ancestors(p, tokens) for p in random_trees(case.rng, 2, tokens)))
    depth = case.rng.integers(-3, tokens + 5, (2, tokens)).astype(np.int64)
    depth[:, 1], depth[:, 3] = 2 ** 31 - 1, -2 ** 31
    check(case, tokens, 4, [300, 100], window=37, sinks=2, nodes=np.stack(nodes), depth=depth)


def test_lengths_of_any_value():
    """Lengths up to 2^31 - 1 and below zero from old buffers: reported or empty, and nothing else."""
    need_gpu()
    m, case = wq(), Case(96, "q4_0", 1, 64, 3, 96, 16)
    cache = case.upload()
    for tokens in (1, 40):
        q = bf16(case.rng, 3, tokens, 1, 64).cuda()
        tree = m.tree_mask(cuda(random_trees(case.rng, 3, tokens)))
        assert m.last_device_status() == 0
        for args in (dict(window=20, sinks=90), dict(tree=tree), dict(tree=tree, window=30, sinks=7)):
            out, lse = m.attend(cache, q, ints([2 ** 31 - 1, -5, 96]), return_lse=True, **args)
            assert m.last_device_status() == m.WQ_ERR_ARG
            assert not out[1].any() and (lse[1] == -float("inf")).all()
            alone, alse = m.attend(cache, q, ints([0, 0, 96]), return_lse=True, **args)
            assert torch.equal(out[2], alone[2]) and torch.equal(lse[2], alse[2]) and m.last_device_status() == 0
            assert torch.isfinite(out[0]).all()


def test_strided_views_and_other_streams():
    """q a column range of a wider buffer, out a view, the call on a stream given by stream=."""
    need_gpu()
    m, case = wq(), Case(97, "nvfp4", 2, 128, 2, 200, 32)
    cache, lens = case.upload(), ints([200, 133])
    side = torch.cuda.Stream()
    for tokens in (3, 60):
        wide = bf16(case.rng, 2, tokens, 14 * 128).cuda()
        q = wide[..., 128:9 * 128].unflatten(-1, (8, 128))
        tree = m.tree_mask(cuda(random_trees(case.rng, 2, tokens)))
        args = dict(window=64, sinks=3, tree=tree)
        want, wlse = m.attend(cache, q.contiguous(), lens, return_lse=True, **args)
        full = torch.full((2, tokens + 2, 9, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        out = full[:, 1:-1, :8]
        side.wait_stream(torch.cuda.current_stream())
        got, lse = m.attend(cache, q, lens, out=out, return_lse=True, stream=side, **args)
        torch.cuda.current_stream().wait_stream(side)
        assert got.data_ptr() == out.data_ptr() and torch.equal(out, want) and torch.equal(lse, wlse)
        assert (full[:, 0] == 7).all() and (full[:, -1] == 7).all() and (full[:, :, 8] == 7).all()
        assert lse.is_contiguous() and lse.shape == (2, tokens, 8) and want.is_contiguous() and want.untyped_storage().data_ptr() % 16 == 0


def test_refusals_from_python():
    need_gpu()
    m, case = wq(), Case(98, "q4_0", 2, 64, 2, 200, 32)
    cache, lens, q = case.upload(), ints([200, 133]), bf16(case.rng, 2, 5, 4, 64).cuda()
    mask, depth = m.tree_mask(cuda(random_trees(case.rng, 2, 5)))
    launches = m.lib.wq_kernel_launches()
    for bad in (dict(tree=(mask.cpu(), depth)), dict(tree=(mask, depth.cpu())), dict(tree=(mask[:, :4], depth)), dict(tree=(mask.long(), depth)),
                dict(tree=(mask, depth[:, ::2])), dict(tree=(mask[:, :, None], depth)), dict(tree=(None, depth), sinks=1, window=1, out=q[:1])):
        with pytest.raises(AssertionError):
            m.attend(cache, q, lens, **bad)
    for bad in (dict(sinks=-1), dict(sinks=1, causal=False), dict(tree=(mask, depth), causal=False), dict(window=-1, sinks=2)):
        with pytest.raises(m.WQError):
            m.attend(cache, q, lens, **bad)
    for bad in (dict(counts=ints([1])), dict(counts=ints([1, 1]).cpu()), dict(window=-1)):
        with pytest.raises((AssertionError, m.WQError)):
            m.tree_mask(cuda(random_trees(case.rng, 2, 5)), **bad)
    for bad in (torch.zeros(2, 5, device="cuda"), torch.zeros(2, 5, dtype=torch.int32), torch.zeros(5, dtype=torch.int32, device="cuda"), "parents"):
        with pytest.raises(AssertionError):
            m.tree_mask(bad)
    with pytest.raises(TypeError):
        m.attend(cache, q, lens, window="wide", sinks=1)
    with pytest.raises(OverflowError):
        m.attend(cache, q, lens, window=2 ** 63, sinks=1)
    assert m.lib.wq_kernel_launches() == launches and m.last_device_status() == 0
