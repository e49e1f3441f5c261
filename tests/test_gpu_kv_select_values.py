"""Attention with sinks and of trees over values that drive the kernels' special ways: V and K scales that are no finite numbers,
blocks whose scale is 8192 or more, scores that leave one weight or make all equal.

A block of V whose scale is infinite or NaN makes its own elements of the rows that see the token non-finite (in the many-row
kernel the whole of those rows NaN); every other output is the same bits as over the clean cache.  A NaN scale of K makes
the rows that see it NaN.

Finite values keep the bounds of tests/test_gpu_kv_select.py, which are relative to sum p |v|, and a floor where that sum is small
beside the row's largest weight times V's size.  The weights go to fp16 as 2^k p, p relative to the row's largest: below 2^-14
a rounding is off by 2^-25 at most, not by a part of the value, so that p is off by 2^-25 2^-k.  k is 12 (q4_0) or 15 (NVFP4)
in the few-row kernel; in the many-row one 11, and the maximum that p is relative to may lie 3 (base 2) above the row's, for weights
that are still to be taken eightfold: 8 at least.  The sum of weights is 1 or more, so
|out - ref| <= ... + 2^-33 sum |v| over the tokens seen.  There, a row of V beside a block whose scale is 8192 or more holds an
eighth of its values, off by 2^-25 at most where they are small: 2^-22 of the value, times weights that add up to one."""
import numpy as np
import pytest
import torch

from oracle import kv as OK
from tests.gpu_common import need_gpu, wq
from tests.helpers import rel_l2
from tests.test_gpu_kv_cache import F32_REL_L2, Case, bf16, ints
from tests.test_gpu_kv_nonfinite import BAD
from tests.test_gpu_kv_select import FMTS, Shared, cuda, random_trees

pytestmark = pytest.mark.gpu


def many_rows(fmt, D, rows):
    """Whether rows go to the many-row kernel (wq.h: more than 32, with sinks or trees more than 16 of q4_0 heads of 128)."""
    return rows > (16 if fmt == "q4_0" and D == 128 else 32)


def check_bad(case, which, bits, bad, tokens, hq, lens, counts=None, window=0, sinks=0, nodes=None, depth=None, q_std=1.0):
    """bad: (page, head, offset, block of 16 or 32 elements) of K's (which 0) or V's (1) scales that become `bits`."""
    m, B, D, H = wq(), len(lens), case.D, case.H
    group, size = hq // H, 32 if case.fmt == "q4_0" else 16
    cache, q = case.upload(), bf16(case.rng, B, tokens, hq, D, std=q_std).cuda()
    tree = None if nodes is None else (cuda(OK.mask_words(nodes)), None if depth is None else cuda(depth.astype(np.int32)))
    args = dict(counts=None if counts is None else ints(counts), window=window, sinks=sinks, tree=tree, out_f32=True, return_lse=True)
    clean, clse = (x.cpu() for x in m.attend(cache, q, ints(lens), **args))
    t = case.t[2 * which + 1]
    t = t.view(torch.int16) if t.dtype == torch.float16 else t
    own = torch.zeros(B, tokens, hq, D, dtype=torch.bool)
    for page, head, off, block in bad:
        t[page, head, off, block] = bits - 65536 if t.dtype == torch.int16 and bits >= 32768 else bits
    for b in range(B):
        seen = OK.visible(tokens, tokens if counts is None else counts[b], lens[b], window, sinks,
                          *(None if x is None else x[b] for x in (nodes, depth)))
        pages, offs = case.at(b, np.arange(lens[b]))
        for page, head, off, block in bad:
            rows = torch.from_numpy(seen[:, (pages == page) & (offs == off)].any(1))
            own[b, :, head * group:(head + 1) * group, block * size:(block + 1) * size] |= rows[:, None, None]
    hit = own.any(-1)
    got, lse = (x.cpu() for x in m.attend(cache, q, ints(lens), **args))
    assert m.last_device_status() == 0
    if which == 0:
        assert torch.isnan(got[hit]).all() and torch.isnan(lse[hit]).all()
    elif many_rows(case.fmt, D, tokens * group):
        assert torch.isnan(got[hit]).all()
    else:
        assert not torch.isfinite(got[own]).any() and torch.equal(lse, clse)
        hit = torch.zeros_like(hit)
        got, clean = got[~own], clean[~own]
        assert torch.equal(got, clean)
        return own
    assert torch.equal(got[~hit], clean[~hit]) and torch.equal(lse[~hit], clse[~hit])
    return own


# position of the bad token: a sink; in the sinks' tile and no sink; between; before the window and where it begins; near the end
PLACES = [2, 7, 150, 255, 262, 291, 299]


@pytest.mark.parametrize("fmt,bits", BAD)
@pytest.mark.parametrize("D,q_std", [(64, 1.0), (128, 1.0), (128, 300.0)])
@pytest.mark.parametrize("tokens", [1, 5, 12, 40, 140])
def test_a_bad_scale_of_v_behind_a_window_with_sinks(fmt, bits, D, q_std, tokens):
    need_gpu()
    hits = 0
    for pos in PLACES:
        case = Case(130, fmt, 2, D, 2, 320, 16)
        page, off = (int(x) for x in case.at(0, pos))
        own = check_bad(case, 1, bits, [(page, 1, off, 1)], tokens, 4, [300, 131], window=40, sinks=5, q_std=q_std)
        hits += bool(own.any())
    assert hits >= 3 + (tokens > 5)


@pytest.mark.parametrize("fmt,bits", BAD)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("tokens", [5, 12, 40, 140])
@pytest.mark.parametrize("window,sinks", [(0, 0), (30, 9)])
def test_bad_scales_in_a_tree_and_its_context(fmt, bits, D, tokens, window, sinks):
    """One node, one sink, one token of the context: K's and V's."""
    need_gpu()
    for which in (0, 1):
        if which == 0 and fmt == "q4_0" and bits != 0x7E00:
            continue                                                   # an infinite d times a code of zero score: not all NaN
        for pos in (300 - tokens + 3, 4, 11, 300 - tokens - 6):
            case = Case(131, fmt, 2, D, 2, 320, 16)
            nodes, depth = (np.stack(x) for x in zip(*(OK.ancestors(p, tokens, window) for p in random_trees(case.rng, 2, tokens, 2))))
            page, off = (int(x) for x in case.at(0, pos))
            check_bad(case, which, bits, [(page, 1, off, 1)], tokens, 4, [300, 160], window=window, sinks=sinks, nodes=nodes, depth=depth)


@pytest.mark.parametrize("fmt,bits", BAD)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("tokens", [3, 12, 40, 200])
def test_many_bad_scales_of_v_over_several_tiles(fmt, bits, D, tokens):
    """A long sequence shared by blocks of several tiles each, bad scales all over it, hidden and seen."""
    need_gpu()
    case, n = Case(132, fmt, 1, D, 1, 9000, 64), 9000
    blocks = D // (32 if fmt == "q4_0" else 16)
    where = list(range(3, n, 397)) + [n - 1 - tokens // 3, n - tokens - 2]
    bad = [(int(p), 0, int(o), k % (blocks - 1)) for k, (p, o) in enumerate(zip(*case.at(0, np.array(where))))]
    own = check_bad(case, 1, bits, bad, tokens, 2, [n], window=4000, sinks=700)
    assert own.any()
    case = Case(132, fmt, 1, D, 1, 9000, 64)
    nodes, depth = (x[None] for x in OK.ancestors(random_trees(case.rng, 1, tokens, 2)[0], tokens))
    bad = [(int(p), 0, int(o), 0) for p, o in zip(*case.at(0, n - tokens + np.array([1, tokens - 2])))]
    check_bad(case, 1, bits, bad, tokens, 2, [n], nodes=nodes, depth=depth)


@pytest.mark.parametrize("fmt,bits", BAD)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("which", [0, 1])
def test_bad_scales_where_blocks_hold_two_groups_of_rows(fmt, bits, D, which):
    need_gpu()
    if which == 0 and fmt == "q4_0" and bits != 0x7E00:
        return
    case, tokens, batch = Shared(133, fmt, 4, D, 45, 300, 32), 40, 45
    nodes, depth = (np.stack(x) for x in zip(*(OK.ancestors(p, tokens) for p in random_trees(case.rng, batch, tokens, 2))))
    lens = [int(x) for x in case.rng.integers(tokens, 300, batch)]
    counts = [int(x) for x in case.rng.integers(1, tokens + 1, batch)]
    own = check_bad(case, which, bits, [(int(case.table[0, 1]), 2, 7, 1), (int(case.table[1, 0]), 0, 30, 0)], tokens, 16, lens, counts,
                    window=90, sinks=20, nodes=nodes, depth=depth)
    assert own.any() and not own.any(-1).all()


# ------------------------------------------------------------------ finite values of every size
def check_values(case, tokens, hq, lens, counts=None, window=0, sinks=0, nodes=None, depth=None, q_std=1.0, exact=True):
    m, B, D = wq(), len(lens), case.D
    cache, q = case.upload(), bf16(case.rng, B, tokens, hq, D, std=q_std)
    tree = None if nodes is None else (cuda(OK.mask_words(nodes)), None if depth is None else cuda(depth.astype(np.int32)))
    got, lse = m.attend(cache, q.cuda(), ints(lens), counts=None if counts is None else ints(counts), window=window, sinks=sinks, tree=tree,
                        return_lse=True, out_f32=True)
    assert m.last_device_status() == 0
    got, lse, refs = got.cpu().double().numpy(), lse.cpu().double().numpy(), []
    for b in range(B):
        seen = OK.visible(tokens, tokens if counts is None else counts[b], lens[b], window, sinks,
                          *(None if x is None else x[b] for x in (nodes, depth)))
        k, v = case.values(b, lens[b])
        ref, rlse, mean, top = OK.attend_seen(q[b].float().numpy(), k, v, seen, D ** -0.5)
        refs.append(ref)
        empty = np.isneginf(rlse)
        assert np.array_equal(np.isneginf(lse[b]), empty) and not got[b][empty].any()
        size = np.einsum("lt,thd->lhd", seen.astype(np.float64), np.abs(v.astype(np.float64))).repeat(hq // case.H, 1)
        bound = (2.0 ** -11 * (2 * top[..., None] + 4) + 2.0 ** -20) * mean + 2.0 ** -33 * size + 2.0 ** -22
        assert np.all(np.abs(got[b] - ref) <= bound), np.max(np.abs(got[b] - ref) / bound)
        assert np.all(np.abs(lse[b][~empty] - rlse[~empty]) <= 2.0 ** -11 * top[~empty] + 2.0 ** -20 * np.abs(rlse[~empty]) + 2.0 ** -20)
    if exact and np.linalg.norm(np.stack(refs)) > 0:
        assert rel_l2(got, np.stack(refs)) <= F32_REL_L2


VALUES = [dict(q_std=300.0, exact=False), dict(q_std=0.0), dict(q_std=2e-3, k_std=3000.0, v_std=20000.0),
          dict(q_std=2e-4, k_std=25000.0, v_std=25000.0), dict(q_std=100.0, k_std=0.01, v_std=0.01)]


@FMTS
@pytest.mark.parametrize("values", VALUES, ids=["one weight", "equal weights", "large V", "large K and V", "small"])
@pytest.mark.parametrize("tokens,hq,h,D", [(1, 8, 2, 128), (4, 8, 2, 64), (5, 8, 2, 128), (8, 8, 2, 64), (40, 8, 2, 128), (40, 8, 2, 64), (140, 2, 1, 128)])
def test_values_of_any_size(fmt, values, tokens, hq, h, D):
    need_gpu()
    values = dict(values)
    std = {x: values.pop(x) for x in ("k_std", "v_std") if x in values}
    case = Case(134, fmt, h, D, 3, 700, 16, **std)
    if fmt == "q4_0" and std.get("v_std", 0) > 1e4:
        assert (np.abs(case.rows[1][1].astype(np.float32)) >= 8192).any()
    if fmt == "q4_0" and std.get("k_std", 0) > 1e4:
        assert (np.abs(case.rows[0][1].astype(np.float32)) >= 8192).any()
    lens, counts = [700, 200, max(3, tokens)], [tokens, max(1, tokens - 1), tokens]
    check_values(case, tokens, hq, lens, counts, window=90, sinks=30, **values)
    nodes, depth = (np.stack(x) for x in zip(*(OK.ancestors(p, tokens, 60) for p in random_trees(case.rng, 3, tokens, 3))))
    check_values(case, tokens, hq, lens, counts, window=60, sinks=30, nodes=nodes, depth=depth, **values)
    check_values(case, tokens, hq, lens, counts, nodes=nodes, **values)


@FMTS
@pytest.mark.parametrize("v_std", [1.0, 25000.0])
@pytest.mark.parametrize("D", [64, 128])
def test_values_of_any_size_where_blocks_hold_two_groups_of_rows(fmt, v_std, D):
    need_gpu()
    case = Shared(135, fmt, 4, D, 45, 300, 32)
    if v_std > 1:
        case.rows = [OK.encode_rows(fmt, (case.rng.standard_normal((case.pages, 4, 32, D)) * v_std).astype(np.float32), g) for g in case.g]
    lens = [int(x) for x in case.rng.integers(40, 300, 45)]
    nodes, depth = (np.stack(x) for x in zip(*(OK.ancestors(p, 40, 70) for p in random_trees(case.rng, 45, 40, 3))))
    for q_std, exact in ((1.0 / v_std, True), (300.0 / v_std, False)):
        check_values(case, 40, 16, lens, window=70, sinks=20, nodes=nodes, depth=depth, q_std=q_std, exact=exact)
