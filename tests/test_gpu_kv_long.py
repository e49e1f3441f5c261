"""Appending and reading back many tokens a call, where whole blocks of tokens share a look-up of their page:
bit for bit against the oracle over page sizes and starts that cut the blocks anywhere, and positions or table
entries outside the cache in the middle and at the end of such a call."""
import numpy as np
import pytest
import torch

from oracle import kv as OK
from tests.gpu_common import need_gpu, wq
from tests.test_gpu_kv_cache import Case, bf16, check_append, ints, raw

pytestmark = pytest.mark.gpu
FMTS = pytest.mark.parametrize("fmt", ["q4_0", "nvfp4"])


@FMTS
@pytest.mark.parametrize("D,page", [(64, 0), (128, 0), (64, 16), (128, 16), (64, 48), (128, 48), (64, 64), (128, 128), (64, 256)])
def test_append_many_tokens(fmt, D, page):
    need_gpu()
    check_append(Case(70, fmt, 2, D, 4, 512, page), 300, [0, 61, 212, 64], [300, 257, 300, 129])


@FMTS
@pytest.mark.parametrize("D,page", [(64, 0), (128, 0), (64, 16), (128, 16), (64, 48), (128, 48), (64, 64), (128, 128), (64, 256)])
@pytest.mark.parametrize("f32", [False, True])
def test_read_many_tokens(fmt, D, page, f32):
    need_gpu()
    m, case = wq(), Case(71, fmt, 2, D, 4, 512, page)
    start, counts, n = [0, 61, 212, 64], [300, 257, 300, 0], 300
    got = m.kv_read(case.upload(), n, ints(start), ints(counts), out_f32=f32)
    for j in range(2):
        want = np.zeros((4, n, 2, D), np.float32)
        for b in range(4):
            want[b, :counts[b]] = case.values(b, counts[b], start[b])[j]
        want = torch.from_numpy(want)
        assert torch.equal(got[j].cpu(), want if f32 else want.bfloat16())
    assert m.last_device_status() == 0


@FMTS
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [0, 16, 64])
@pytest.mark.parametrize("first", [150, 147, -70])
def test_long_calls_that_leave_the_cache(fmt, D, page, first):
    """Sequence 0 runs over an end of its 320 positions, sequence 1 (paged) over a bad table entry: those tokens are
    dropped, or read as zero, every other one is served, and nothing else changes."""
    need_gpu()
    m, case = wq(), Case(72, fmt, 2, D, 3, 320, page)
    tokens, start = 250, [first, 13, 40]
    if page:
        case.table[1, 128 // page] = -1
        case.table[1, 192 // page] = case.pages
    cache = case.upload()
    before = [raw(t).copy() for t in case.t]
    k, v = (bf16(case.rng, 3, tokens, 2, D) for _ in range(2))
    assert m.last_device_status() == 0
    m.kv_append(cache, k.cuda(), v.cuda(), ints(start))
    assert m.last_device_status() == m.WQ_ERR_ARG
    want = [torch.zeros(3, tokens, 2, D) for _ in range(2)]
    for b in range(3):
        pos = start[b] + np.arange(tokens)
        ok = (pos >= 0) & (pos < 320)
        if page:
            there = case.table[b, np.clip(pos, 0, 319) // page]
            ok &= (there >= 0) & (there < case.pages)
        where, off = case.at(b, pos[ok])
        for j, x in enumerate((k, v)):
            codes, scales = OK.encode_rows(fmt, x[b, ok].float().numpy(), case.g[j])
            before[2 * j][where, :, off] = codes
            before[2 * j + 1][where, :, off] = np.ascontiguousarray(scales).view(np.uint8)
            want[j][b, ok] = torch.from_numpy(OK.decode_rows(fmt, codes, scales, case.g[j]))
    assert all(np.array_equal(raw(t), x) for t, x in zip(case.t, before))
    got = m.kv_read(cache, tokens, ints(start), out_f32=True)
    assert m.last_device_status() == m.WQ_ERR_ARG
    assert all(torch.equal(a.cpu(), b) for a, b in zip(got, want))
