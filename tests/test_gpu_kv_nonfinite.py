"""Scales in the cache that are no finite numbers: what they touch, and that they touch nothing else.

A block of V whose scale is infinite or NaN makes its own elements of the rows that see the token non-finite (with more than
32 query rows per cached head: the whole of those rows NaN); every other output is the same bits as over the clean cache.
A NaN scale of K makes the rows that see the token NaN, any other such scale at least leaves the rows that do not see it."""
import numpy as np
import pytest
import torch

from tests.gpu_common import need_gpu, wq
from tests.test_gpu_kv_cache import Case, bf16, ints

pytestmark = pytest.mark.gpu

BAD = [("q4_0", 0x7E00), ("q4_0", 0x7C00), ("q4_0", 0xFC00), ("nvfp4", 0x7F), ("nvfp4", 0xFF)]   # NaN, +-inf; the two NaNs
LENS = [300, 131]


def seen_by(tokens, group, heads, window, b, h, pos):
    """bool [2, tokens, heads * group]: the rows that see position pos of sequence b, cached head h (causal)."""
    hit = torch.zeros(2, tokens, heads * group, dtype=torch.bool)
    p = LENS[b] - tokens + torch.arange(tokens)
    hit[b, :, h * group:(h + 1) * group] = ((p >= pos) & ((window == 0) | (pos > p - window)))[:, None]
    return hit


def corrupt(case, which, b, h, pos, block, bits):
    """Sets one scale of K (0) or V (1) and returns what was there."""
    page, off = (int(x) for x in case.at(b, pos))
    t = case.t[2 * which + 1]
    t = t.view(torch.int16) if t.dtype == torch.float16 else t
    old = t[page, h, off, block].clone()
    t[page, h, off, block] = bits - 65536 if t.dtype == torch.int16 and bits >= 32768 else bits
    return t, (page, h, off, block), old


# (query tokens, position of the bad token behind which some rows lie, window): the token is seen by no row (just before the
# window, in a tile that is read), by some, by all
PLACES = [(1, 299, 0), (1, 298, 1), (1, 259, 40), (1, 260, 40), (5, 299, 0), (5, 297, 0), (5, 297, 2), (5, 293, 3), (12, 290, 0),
          (12, 294, 3), (12, 200, 0), (140, 299, 0), (140, 230, 0), (140, 170, 20), (140, 130, 17), (140, 139, 21)]


@pytest.mark.parametrize("fmt,bits", BAD)
@pytest.mark.parametrize("tokens,pos,window", PLACES)
@pytest.mark.parametrize("D,q_std", [(64, 1.0), (128, 1.0), (128, 300.0)])
def test_a_bad_scale_of_v_reaches_only_rows_that_see_it(fmt, bits, tokens, pos, window, D, q_std):
    """q_std 300: nearly every row gives the token a weight of zero, and sees it all the same."""
    need_gpu()
    m, case = wq(), Case(80, fmt, 2, D, 2, 320, 16)
    cache, q = case.upload(), bf16(case.rng, 2, tokens, 4, D, std=q_std).cuda()
    args = dict(window=window, out_f32=True, return_lse=True)
    clean, clse = (x.cpu() for x in m.attend(cache, q, ints(LENS), **args))
    size, block = (32, 1) if fmt == "q4_0" else (16, 3)
    corrupt(case, 1, 0, 1, pos, block, bits)
    got, lse = (x.cpu() for x in m.attend(cache, q, ints(LENS), **args))
    hit = seen_by(tokens, 2, 2, window, 0, 1, pos)
    own = torch.zeros(2, tokens, 4, D, dtype=torch.bool)
    own[..., block * size:(block + 1) * size] = hit[..., None]
    rest = ~own if tokens * 2 <= 32 else (~hit)[..., None].expand_as(own)
    assert torch.equal(got[rest], clean[rest]) and torch.equal(lse[~hit], clse[~hit])
    assert not torch.isfinite(got[own]).any()
    if tokens * 2 > 32:
        assert torch.isnan(got[hit]).all()
    else:
        assert torch.equal(lse, clse)
    assert m.last_device_status() == 0


@pytest.mark.parametrize("fmt,bits", BAD)
@pytest.mark.parametrize("tokens,pos,window", PLACES)
def test_a_bad_scale_of_k_reaches_only_rows_that_see_it(fmt, bits, tokens, pos, window):
    need_gpu()
    m, case = wq(), Case(81, fmt, 2, 64, 2, 320, 16)
    cache, q = case.upload(), bf16(case.rng, 2, tokens, 4, 64).cuda()
    args = dict(window=window, out_f32=True, return_lse=True)
    clean, clse = (x.cpu() for x in m.attend(cache, q, ints(LENS), **args))
    corrupt(case, 0, 0, 1, pos, 1, bits)
    got, lse = (x.cpu() for x in m.attend(cache, q, ints(LENS), **args))
    hit = seen_by(tokens, 2, 2, window, 0, 1, pos)
    assert torch.equal(got[~hit], clean[~hit]) and torch.equal(lse[~hit], clse[~hit])
    if fmt == "nvfp4" or bits == 0x7E00:
        assert torch.isnan(got[hit]).all() and torch.isnan(lse[hit]).all()


@pytest.mark.parametrize("fmt,bits", BAD)
@pytest.mark.parametrize("tokens", [1, 5, 12, 140])
def test_many_bad_scales_of_v_over_split_tokens(fmt, bits, tokens):
    """A long sequence shared by many blocks, bad scales all over it, hidden and seen: the elements that see one are non-finite,
    all others are the clean bits."""
    need_gpu()
    m, n, window = wq(), 9000, 4000
    case = Case(82, fmt, 1, 64, 1, n, 64)
    cache, q = case.upload(), bf16(case.rng, 1, tokens, 2, 64).cuda()
    args = dict(window=window, out_f32=True)
    clean = m.attend(cache, q, ints([n]), **args).cpu()
    size, blocks = (32, 2) if fmt == "q4_0" else (16, 4)
    p = n - tokens + torch.arange(tokens)
    bad = torch.zeros(tokens, 64, dtype=torch.bool)
    for k, pos in enumerate(list(range(17, n - window - tokens, 611)) + [n - window - tokens // 2, n - 1 - tokens // 3]):
        block = k % (blocks - 1)                # the last block stays clean
        corrupt(case, 1, 0, 0, pos, block, bits)
        sees = (p >= pos) & (pos > p - window)
        bad[:, block * size:(block + 1) * size] |= sees[:, None]
    got = m.attend(cache, q, ints([n]), **args).cpu()
    own = bad[None, :, None].expand_as(got)
    rest = ~own if tokens * 2 <= 32 else ~bad.any(1)[None, :, None, None].expand_as(got)
    assert torch.equal(got[rest], clean[rest]) and not torch.isfinite(got[own]).any()
    assert m.last_device_status() == 0
