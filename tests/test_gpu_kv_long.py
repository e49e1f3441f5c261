"""Appending and reading back many tokens a call, where whole blocks of tokens share a look-up of their page:
bit for bit against the oracle over page sizes and starts that cut the blocks anywhere, and positions or table
entries outside the cache in the middle and at the end of such a call."""
import numpy as np
import pytest
import torch

from oracle import kv as OK
from tests.gpu_common import need_gpu, wq
from tests.test_gpu_kv_cache import Case, bf16, check_append, check_attend, ints, raw

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


@FMTS
@pytest.mark.parametrize("tokens", [1, 40])
def test_calls_on_another_stream(fmt, tokens):
    """stream=: append, attend (with a workspace) and read run there and give what the current stream gives; results and
    workspace come from memory that the current stream's pending work does not use."""
    need_gpu()
    m, case = wq(), Case(73, fmt, 2, 128, 2, 4000, 16)
    cache = case.upload()
    k, v, q = (bf16(case.rng, 2, tokens, h, 128).cuda() for h in (2, 2, 8))
    lens = ints([4000, 3001])
    start = lens - tokens
    m.kv_append(cache, k, v, start)
    want, want_lse = m.attend(cache, q, lens, return_lse=True)
    wk, wv = m.kv_read(cache, 4000, counts=lens)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        busy = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
        for _ in range(20):
            busy.fill_(1)              # the current stream still writes this memory when it is given back
        del busy
        m.kv_append(cache, k, v, start, stream=other)
        out, lse = m.attend(cache, q, lens, return_lse=True, stream=other)
        gk, gv = m.kv_read(cache, 4000, counts=lens, stream=other)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse) and torch.equal(gk, wk) and torch.equal(gv, wv)
    assert m.last_device_status() == 0


@pytest.mark.parametrize("fmt,window", [("q4_0", 0), ("nvfp4", 0), ("q4_0", 300), ("nvfp4", 6300)])
def test_attend_over_an_uneven_number_of_parts(fmt, window):
    """152 heads of long sequences: three parts each, joined from the workspace."""
    need_gpu()
    check_attend(Case(74, fmt, 38, 64, 4, 6400, 64), 1, 38, [6400, 1, 100, 4001], window=window)


@FMTS
@pytest.mark.parametrize("D,q_heads,tokens", [(64, 4, 1), (128, 16, 3), (64, 2, 40), (128, 16, 150)])
def test_attend_leaves_out_pages_that_are_not_there(fmt, D, q_heads, tokens):
    """Bad table entries in the middle of a sequence: its tokens are not there, the other sequence is untouched, the status
    tells.  Bounds as for any attention."""
    need_gpu()
    m, case = wq(), Case(75, fmt, 2, D, 2, 640, 16)
    lens = [633, 500]
    kv = [case.values(b, lens[b]) for b in range(2)]
    case.table[1, 3], case.table[1, 17] = -1, case.pages
    there = np.ones(lens[1], bool)
    there[48:64] = there[272:288] = False
    kv[1] = [x[there] for x in kv[1]]
    q = bf16(case.rng, 2, tokens, q_heads, D)
    assert m.last_device_status() == 0
    out, lse = m.attend(case.upload(), q.cuda(), ints(lens), out_f32=True, return_lse=True)
    assert m.last_device_status() == m.WQ_ERR_ARG
    for b in range(2):
        ref, rlse, mean, top = OK.attend(q[b].float().numpy(), kv[b][0], kv[b][1], tokens, D ** -0.5, True)
        assert np.all(np.abs(out[b].cpu().double().numpy() - ref) <= (2.0 ** -11 * (2 * top[..., None] + 4) + 2.0 ** -20) * mean + 1e-30)
        assert np.all(np.abs(lse[b].cpu().double().numpy() - rlse) <= 2.0 ** -11 * top + 2.0 ** -20 * np.abs(rlse) + 2.0 ** -20)
