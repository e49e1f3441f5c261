"""The 4-bit KV cache on the GPU against the oracle: appended codes and scales bit for bit, values read
back exactly, attention against fp64.

Tolerances of the attention tests (fixed before the first run).  Scores, softmax statistics and sums are
fp32; where an operand enters a matrix instruction it may be rounded once to 11 significant bits (K, V,
the weights p, and p times a block's scale), each a relative 2^-11 at most.  With A the largest sum of
|scale q k| of the row, rounding K moves a score by 2^-11 A at most, a weight by 2 * 2^-11 A, so that
  |out - ref| <= 2^-11 (2 A + 4) sum p |v| + 2^-20 sum p |v|     and     |lse - ref| <= 2^-11 A + 2^-20 |ref| + 2^-20,
plus half a bf16 ulp, 2^-9 |ref| (1 + 2^-8), where out is bf16.  These roundings are independent, so for random
data the relative L2 error is far smaller: sqrt(4) * 2^-11 = 1e-3 bounds it for the fp32 output.
"""
import numpy as np
import pytest
import torch

from oracle import kv as OK
from tests.gpu_common import wq, need_gpu, REL_L2_TOL
from tests.helpers import rel_l2

pytestmark = pytest.mark.gpu

F32_REL_L2 = 1e-3
KG, VG = np.float32(0.0074), np.float32(0.0021)


class Case:
    """A cache of random rows on the host and the GPU, paged in a random order (page > 0) or contiguous."""

    def __init__(self, seed, fmt, heads, D, batch, capacity, page=0, k_std=1.0, v_std=1.0, use_g=True):
        rng = np.random.default_rng(seed)
        self.rng, self.fmt, self.H, self.D, self.batch = rng, fmt, heads, D, batch
        self.size = page or -(-capacity // 16) * 16
        per = -(-capacity // self.size)
        self.pages = batch * per + (2 if page else 0)
        self.table = rng.permutation(self.pages)[:batch * per].reshape(batch, per).astype(np.int32) if page else None
        self.g = ((KG, VG) if use_g else (None, None)) if fmt == "nvfp4" else (None, None)
        shape = (self.pages, heads, self.size, D)
        self.rows = [OK.encode_rows(fmt, (rng.standard_normal(shape) * s).astype(np.float32), g)
                     for s, g in zip((k_std, v_std), self.g)]

    def upload(self):
        m = wq()
        t = [torch.from_numpy(np.ascontiguousarray(a)).cuda() for pair in self.rows for a in pair]
        self.t = t
        table = None if self.table is None else torch.from_numpy(self.table).cuda()
        g = [None if x is None else torch.tensor([x], device="cuda") for x in self.g]
        return m.KVCache(self.fmt, t[0], t[1], t[2], t[3], table, g[0], g[1])

    def at(self, b, pos):
        """(page, offset) of positions pos of sequence b."""
        pos = np.asarray(pos)
        return (np.full(pos.shape, b), pos) if self.table is None else (self.table[b, pos // self.size], pos % self.size)

    def values(self, b, n, start=0):
        """K and V [n, H, D] of the sequence's positions from start on, as fp32."""
        page, off = self.at(b, np.arange(start, start + n))
        return [OK.decode_rows(self.fmt, c[page, :, off], s[page, :, off], g) for (c, s), g in zip(self.rows, self.g)]


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def bf16(rng, *shape, std=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32)).bfloat16()


def raw(t):
    return t.cpu().view(torch.uint8).numpy() if t.dtype != torch.uint8 else t.cpu().numpy()


# ------------------------------------------------------------------ append
def check_append(case, tokens, start, counts, std=1.0, special=None):
    m, B, H, D = wq(), case.batch, case.H, case.D
    cache = case.upload()
    before = [a.copy() for pair in case.rows for a in pair]
    k, v = bf16(case.rng, B, tokens, H, D, std=std), bf16(case.rng, B, tokens, H, D, std=std)
    if special is not None:
        special(k)
        special(v)
    m.kv_append(cache, k.cuda(), v.cuda(), None if start is None else ints(start), None if counts is None else ints(counts))
    torch.cuda.synchronize()
    for j, x in enumerate((k, v)):
        for b in range(B):
            n = tokens if counts is None else min(max(counts[b], 0), tokens)
            if n == 0:
                continue
            page, off = case.at(b, (0 if start is None else start[b]) + np.arange(n))
            codes, scales = OK.encode_rows(case.fmt, x[b, :n].float().numpy(), case.g[j])
            before[2 * j][page, :, off] = codes
            before[2 * j + 1][page, :, off] = scales
    for j in range(4):
        assert np.array_equal(raw(case.t[j]), before[j].view(np.uint8)), ("k codes", "k scales", "v codes", "v scales")[j]
    assert m.last_device_status() == 0


@pytest.mark.parametrize("fmt", ["q4_0", "nvfp4"])
@pytest.mark.parametrize("H,D,page", [(20, 64, 0), (8, 128, 16), (1, 64, 48), (3, 128, 0), (6, 64, 64)])
def test_append_bits_and_nothing_else(fmt, H, D, page):
    need_gpu()
    check_append(Case(1, fmt, H, D, 3, 150, page), 37, [0, 61, 113], [37, 20, 1])


@pytest.mark.parametrize("fmt", ["q4_0", "nvfp4"])
def test_append_defaults_and_clamped_counts(fmt):
    need_gpu()
    check_append(Case(2, fmt, 2, 64, 2, 40, 0), 9, None, None)
    check_append(Case(3, fmt, 2, 128, 3, 64, 32), 9, [50, 3, 7], [-4, 100, 0])
    check_append(Case(4, fmt, 5, 64, 1, 64, 16, use_g=False), 1, [63], None)


@pytest.mark.parametrize("fmt", ["q4_0", "nvfp4"])
@pytest.mark.parametrize("D", [64, 128])
def test_append_ties_zeros_and_extremes(fmt, D):
    need_gpu()

    def special(x):
        x[0, 0] = 0.0
        x[0, 1] = -0.0
        x[0, 2, :, 0], x[0, 2, :, 1] = 7.0, -7.0        # the first of two equal magnitudes sets the sign of d
        x[0, 3, :, 5], x[0, 3, :, 31] = -9.0, 9.0
        x[0, 4, :, 17], x[0, 4, :, 16] = 9.0, -9.0
        x[0, 5] = torch.linspace(-4, 4, D).bfloat16()    # many half-way quotients
        x[0, 6] = (torch.arange(D) % 17 - 8).bfloat16() * 0.5
        x[0, 7] = 1e-30                                  # d underflows to zero
        x[0, 8] *= 1e-6                                  # d is a subnormal fp16
        x[0, 9] *= 300.0
        x[0, 10] *= 60000.0
    check_append(Case(5, fmt, 2, D, 1, 32, 0), 11, [3], None, special=special)


def test_append_nan_stays_in_its_block():
    need_gpu()
    m, case = wq(), Case(6, "q4_0", 2, 64, 1, 32)
    cache = case.upload()
    k = torch.ones(1, 4, 2, 64, dtype=torch.bfloat16)
    k[0, 1, 0, 40] = float("nan")
    k[0, 2, 1, 3] = float("inf")
    m.kv_append(cache, k.cuda(), k.cuda())
    got = m.kv_read(cache, 4, out_f32=True)[0].cpu()
    bad = torch.zeros(1, 4, 2, 64, dtype=torch.bool)
    bad[0, 1, 0, 32:] = True
    bad[0, 2, 1, :32] = True
    assert torch.isnan(got[0, 1, 0, 32:]).all() and not torch.isfinite(got[bad]).any()
    assert torch.equal(got[~bad], torch.ones_like(got[~bad]))


def test_append_from_column_ranges_of_a_fused_projection():
    need_gpu()
    m, case = wq(), Case(7, "q4_0", 4, 64, 2, 48, 16)
    cache, T = case.upload(), 13
    qkv = bf16(case.rng, 2, T, 3 * 4 * 64).cuda()
    k, v = (qkv[..., i * 256:(i + 1) * 256].unflatten(-1, (4, 64)) for i in (1, 2))
    m.kv_append(cache, k, v, ints([5, 30]))
    gk, gv = m.kv_read(cache, T, ints([5, 30]), out_f32=True)
    for got, x in ((gk, k), (gv, v)):
        c, s = OK.encode_rows("q4_0", x.float().cpu().numpy())
        assert np.array_equal(got.cpu().numpy(), OK.decode_rows("q4_0", c, s))
    # head-major K (a transposed view) too
    kt = k.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    m.kv_append(cache, kt, v, ints([5, 30]))
    assert torch.equal(m.kv_read(cache, T, ints([5, 30]), out_f32=True)[0], gk)


# ------------------------------------------------------------------ read
@pytest.mark.parametrize("fmt", ["q4_0", "nvfp4"])
@pytest.mark.parametrize("H,D,page", [(20, 64, 0), (8, 128, 16), (1, 64, 48), (3, 128, 64)])
@pytest.mark.parametrize("f32", [False, True])
def test_read_values(fmt, H, D, page, f32):
    need_gpu()
    m, case = wq(), Case(11, fmt, H, D, 3, 150, page)
    cache, start, counts, n = case.upload(), [0, 61, 113], [50, 0, 37], 50
    got = m.kv_read(cache, n, ints(start), ints(counts), out_f32=f32)
    for j in range(2):
        want = np.zeros((3, n, H, D), np.float32)
        for b in range(3):
            want[b, :counts[b]] = case.values(b, counts[b], start[b])[j]
        want = torch.from_numpy(want)
        assert torch.equal(got[j].cpu(), want if f32 else want.bfloat16())
    assert m.last_device_status() == 0


def test_read_one_side_into_strided_rows_and_every_code():
    """Each of the 16 codes under every kind of scale (q4_0: negative, zero, subnormal; NVFP4: all 256 bytes but NaN)."""
    need_gpu()
    m, L = wq(), wq().lib
    import ctypes
    for fmt in ("q4_0", "nvfp4"):
        case = Case(12, fmt, 2, 64, 1, 256)
        case.rows[0][0][:] = case.rng.integers(0, 256, case.rows[0][0].shape)
        if fmt == "q4_0":
            d = np.array([0.0, -0.0, 1.0, -1.0, 6e-8, -6e-8, 65504.0, 0.3334], np.float16)
            case.rows[0][1][:] = d[case.rng.integers(0, 8, case.rows[0][1].shape)]
        else:
            b = case.rng.permutation(256 * 8) % 256
            case.rows[0][1][:] = np.where(b & 127 == 127, 0, b).reshape(1, 2, 256, 4)
        cache = case.upload()
        full = torch.full((256, 3, 2, 64), 7.0, device="cuda")
        h = m.wq_heads(full[:, 1].data_ptr(), 0, full.stride(0), 64)
        rc = L.wq_kv_read(cache.ref, ctypes.byref(h), None, 1, 256, None, None, 1,
                          ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        assert rc == 0
        got = full.cpu().numpy()
        assert np.array_equal(got[:, 1], case.values(0, 256)[0])
        assert (got[:, 0] == 7).all() and (got[:, 2] == 7).all()


def test_positions_outside_the_cache_are_reported_and_touch_nothing():
    need_gpu()
    m, case = wq(), Case(13, "q4_0", 2, 64, 3, 64, 16)
    case.table[1, 1] = 10 ** 6                    # not a page
    case.table[2, 0] = -1
    cache = case.upload()
    before = [raw(t).copy() for t in case.t]
    k = bf16(case.rng, 3, 4, 2, 64).cuda()
    assert m.last_device_status() == 0
    m.kv_append(cache, k, k, ints([62, 16, 3]))   # two past the capacity, four on a bad page, four on a bad page
    assert m.last_device_status() == m.WQ_ERR_ARG and m.last_device_status() == 0
    page, off = case.at(0, np.array([62, 63]))
    for j in range(2):
        codes, scales = OK.encode_rows("q4_0", k[0, :2].float().cpu().numpy())
        before[2 * j][page, :, off] = codes
        before[2 * j + 1].reshape(-1, 2, 16, 4)[page, :, off] = scales.view(np.uint8).reshape(2, 2, 4)
    assert all(np.array_equal(raw(t), b) for t, b in zip(case.t, before))
    got, _ = m.kv_read(cache, 2, ints([-1, 15, 15]))
    assert m.last_device_status() == m.WQ_ERR_ARG
    assert not got[0, 0].any() and got[0, 1].any() and got[1, 0].any() and not got[1, 1].any() and not got[2, 0].any()
    out, lse = m.attend(cache, bf16(case.rng, 3, 1, 2, 64).cuda(), ints([70, 20, 16]), return_lse=True)
    assert m.last_device_status() == m.WQ_ERR_ARG
    assert torch.isfinite(out).all() and torch.isfinite(lse[:2]).all() and (lse[2] == -float("inf")).all()


# ------------------------------------------------------------------ attention
def check_attend(case, tokens, q_heads, lens, counts=None, causal=True, window=0, scale=None, q_std=1.0, max_len=0,
                 random_data=True):
    m, B, D = wq(), case.batch, case.D
    cache = case.upload()
    q = bf16(case.rng, B, tokens, q_heads, D, std=q_std)
    sc = D ** -0.5 if scale is None else scale
    args = dict(counts=None if counts is None else ints(counts), causal=causal, window=window, scale=scale, max_len=max_len,
                return_lse=True)
    got32, lse = m.attend(cache, q.cuda(), ints(lens), out_f32=True, **args)
    got16, lse16 = m.attend(cache, q.cuda(), ints(lens), **args)
    assert m.last_device_status() == 0
    assert torch.equal(lse, lse16) and torch.equal(got32.bfloat16(), got16)
    got32, lse = got32.cpu().double().numpy(), lse.cpu().double().numpy()
    refs = []
    for b in range(B):
        n = max(0, lens[b])
        k, v = case.values(b, n)
        nq = tokens if counts is None else min(max(counts[b], 0), tokens)
        ref, rlse, mean, top = OK.attend(q[b].float().numpy(), k, v, nq, sc, causal, window)
        refs.append(ref)
        empty = np.isneginf(rlse)
        assert np.array_equal(np.isneginf(lse[b]), empty) and not got32[b][empty].any()
        bound = (2.0 ** -11 * (2 * top[..., None] + 4) + 2.0 ** -20) * mean
        assert np.all(np.abs(got32[b] - ref) <= bound + 1e-30), np.max(np.abs(got32[b] - ref) / (bound + 1e-30))
        ok = ~empty
        assert np.all(np.abs(lse[b][ok] - rlse[ok]) <= 2.0 ** -11 * top[ok] + 2.0 ** -20 * np.abs(rlse[ok]) + 2.0 ** -20)
    if random_data and np.linalg.norm(np.stack(refs)) > 0:
        assert rel_l2(got32, np.stack(refs)) <= F32_REL_L2
        assert rel_l2(got16.float().cpu().numpy(), np.stack(refs)) <= REL_L2_TOL


LAYOUTS = [(20, 20, 64, 0), (6, 6, 64, 16), (32, 8, 128, 16), (32, 4, 128, 48), (16, 1, 128, 64), (8, 1, 64, 32), (40, 8, 128, 0),
           (33, 3, 64, 16), (3, 3, 128, 16)]


@pytest.mark.parametrize("fmt", ["q4_0", "nvfp4"])
@pytest.mark.parametrize("hq,h,D,page", LAYOUTS)
def test_attend_one_token(fmt, hq, h, D, page):
    need_gpu()
    lens = [1, 2, 15, 16, 17, 31, 33, 64, 97, 0, 300]
    check_attend(Case(21, fmt, h, D, len(lens), 300, page), 1, hq, lens)


@pytest.mark.parametrize("fmt", ["q4_0", "nvfp4"])
@pytest.mark.parametrize("hq,h,D,page", LAYOUTS)
@pytest.mark.parametrize("tokens", [2, 7, 19])
def test_attend_several_tokens_ragged(fmt, hq, h, D, page, tokens):
    need_gpu()
    lens, counts = [0, 1, 5, 33, 130, 257], [tokens, 1, tokens, 0, tokens, tokens - 1]
    check_attend(Case(22, fmt, h, D, 6, 257, page), tokens, hq, lens, counts)
    check_attend(Case(23, fmt, h, D, 6, 257, page), tokens, hq, lens, counts, causal=False)


@pytest.mark.parametrize("fmt", ["q4_0", "nvfp4"])
@pytest.mark.parametrize("hq,h,D,page", [(4, 4, 64, 0), (8, 2, 128, 16), (6, 1, 128, 32), (5, 1, 64, 48)])
@pytest.mark.parametrize("causal", [True, False])
def test_attend_many_tokens(fmt, hq, h, D, page, causal):
    need_gpu()
    check_attend(Case(24, fmt, h, D, 2, 420, page), 161, hq, [420, 163], [161, 150], causal=causal)


@pytest.mark.parametrize("fmt", ["q4_0", "nvfp4"])
@pytest.mark.parametrize("window", [1, 15, 64, 100, 10 ** 6])
@pytest.mark.parametrize("tokens,hq,h,D", [(1, 8, 2, 128), (6, 8, 2, 128), (150, 4, 2, 64), (140, 2, 1, 128)])
def test_attend_window(fmt, window, tokens, hq, h, D):
    need_gpu()
    check_attend(Case(25, fmt, h, D, 3, 333, 16), tokens, hq, [333, max(90, tokens), 40], window=window)


@pytest.mark.parametrize("fmt", ["q4_0", "nvfp4"])
@pytest.mark.parametrize("tokens", [1, 3, 40])
def test_attend_rows_before_the_first_token_see_nothing(fmt, tokens):
    """More query tokens than cached ones: the first rows are before position 0."""
    need_gpu()
    check_attend(Case(26, fmt, 2, 128, 4, 48, 16), tokens, 4, [0, 1, 2, 39])


@pytest.mark.parametrize("fmt,D", [("q4_0", 128), ("nvfp4", 64)])
def test_attend_long_and_split(fmt, D):
    """Few rows over long sequences: the tokens are split over many blocks and joined."""
    need_gpu()
    check_attend(Case(27, fmt, 1, D, 1, 20011, 64), 1, 4, [20011])
    check_attend(Case(28, fmt, 2, D, 2, 9000, 16), 3, 8, [9000, 513])
    check_attend(Case(29, fmt, 1, D, 2, 6000, 0), 1, 1, [6000, 3], max_len=6000)
    check_attend(Case(29, fmt, 1, D, 2, 6000, 0), 1, 1, [6000, 3], max_len=5)   # a wrong plan is only slower
    check_attend(Case(30, fmt, 1, D, 1, 5000, 32), 130, 2, [5000])


@pytest.mark.parametrize("fmt", ["q4_0", "nvfp4"])
@pytest.mark.parametrize("tokens", [1, 140])
def test_attend_peaked_and_extreme_scores(fmt, tokens):
    """Scores up to some thousands (one token takes all), no scores at all, tiny and huge values."""
    need_gpu()
    T = 200 if tokens == 1 else 300
    check_attend(Case(31, fmt, 2, 128, 2, T, 16), tokens, 4, [T, T - 50], q_std=300.0, random_data=False)
    check_attend(Case(32, fmt, 2, 64, 2, T, 16), tokens, 4, [T, T - 50], q_std=0.0)
    check_attend(Case(33, fmt, 2, 64, 2, T, 16), tokens, 4, [T, T - 50], scale=-0.3)
    check_attend(Case(34, fmt, 2, 64, 2, T, 16), tokens, 4, [T, T - 50], scale=0.0)
    if fmt == "q4_0":   # values far from 1: the scales carry them (fp16 d)
        check_attend(Case(35, fmt, 2, 128, 2, T, 16, k_std=3000.0, v_std=20000.0), tokens, 4, [T, 150], q_std=2e-3)
        check_attend(Case(36, fmt, 2, 128, 2, T, 16, k_std=0.01, v_std=0.01), tokens, 4, [T, 150], q_std=100.0)
    else:
        check_attend(Case(37, fmt, 2, 128, 2, T, 16, k_std=4.0, use_g=False, v_std=4.0), tokens, 4, [T, 150])


@pytest.mark.parametrize("fmt", ["q4_0", "nvfp4"])
@pytest.mark.parametrize("tokens", [1, 5, 140])
@pytest.mark.parametrize("page", [0, 16])
def test_attend_ignores_what_lies_past_the_length(fmt, tokens, page):
    """NaN and infinite scales in the unused part of the cache and of the last page, table entries past the end that
    are no pages: the outputs are the same bits as over a clean cache, and nothing is reported."""
    need_gpu()
    m, lens = wq(), [141, 150, 177]
    case = Case(38, fmt, 2, 128, 3, 240, page)
    q = bf16(case.rng, 3, tokens, 4, 128).cuda()
    clean = m.attend(case.upload(), q, ints(lens), return_lse=True)
    used = np.zeros((case.pages, case.size), bool)
    for b, n in enumerate(lens):
        used[case.at(b, np.arange(n))] = True
    for j in range(2):
        bad = np.array([np.nan, np.inf, -np.inf], np.float16) if fmt == "q4_0" else np.array([0x7F, 0xFF, 0x7E], np.uint8)
        s = case.rows[j][1].transpose(0, 2, 1, 3)
        s[~used] = bad[np.arange(s[~used].size) % 3].reshape(s[~used].shape)
        c = case.rows[j][0].transpose(0, 2, 1, 3)
        c[~used] = case.rng.integers(0, 256, c[~used].shape)
    if page:
        for b, n in enumerate(lens):
            case.table[b, -(-n // page):] = [-1, 2 ** 30, 10 ** 9][b]
    dirty = m.attend(case.upload(), q, ints(lens), return_lse=True)
    assert torch.equal(clean[0], dirty[0]) and torch.equal(clean[1], dirty[1]) and torch.isfinite(dirty[1]).all()
    assert m.last_device_status() == 0


@pytest.mark.parametrize("tokens", [1, 140])
def test_attend_nan_and_inf_reach_only_their_rows(tokens):
    """A NaN key or query spoils the rows that see it and no other; an infinite V only its own elements."""
    need_gpu()
    m, case = wq(), Case(39, "q4_0", 2, 64, 2, 300)
    cache, q = case.upload(), bf16(case.rng, 2, tokens, 4, 64)
    clean, clse = m.attend(cache, q.cuda(), ints([290, 280]), return_lse=True)
    case.t[1][0, 1, 285] = float("nan")                    # K of sequence 0, head 1, position 285
    got, lse = m.attend(cache, q.cuda(), ints([290, 280]), return_lse=True)
    pos = 290 - tokens + torch.arange(tokens)
    hit = torch.zeros(2, tokens, 4, dtype=torch.bool)
    hit[0, :, 2:] = (pos >= 285)[:, None]
    assert torch.isnan(lse.cpu()[hit]).all() and torch.isnan(got.cpu()[hit]).all()
    assert torch.equal(lse.cpu()[~hit], clse.cpu()[~hit]) and torch.equal(got.cpu()[~hit], clean.cpu()[~hit])
    cache = Case(39, "q4_0", 2, 64, 2, 300)
    c2 = cache.upload()
    q[1, tokens - 1, 3, 7] = float("nan")
    got, lse = m.attend(c2, q.cuda(), ints([290, 280]), return_lse=True)
    hit[:] = False
    hit[1, tokens - 1, 3] = True
    assert torch.isnan(lse.cpu()[hit]).all() and torch.isnan(got.cpu()[hit]).all()
    assert torch.equal(lse.cpu()[~hit], clse.cpu()[~hit]) and torch.equal(got.cpu()[~hit], clean.cpu()[~hit])


@pytest.mark.parametrize("tokens,hq,h,D", [(3, 8, 2, 128), (90, 4, 2, 64)])
def test_attend_strided_q_and_out(tokens, hq, h, D):
    need_gpu()
    m, case = wq(), Case(40, "nvfp4", h, D, 2, 200, 32)
    cache, lens = case.upload(), ints([200, 133])
    fused = bf16(case.rng, 2, tokens, (hq + 2 * h) * D).cuda()
    q = fused[..., :hq * D].unflatten(-1, (hq, D))
    want = m.attend(cache, q.contiguous(), lens)
    full = torch.full((2, tokens + 2, hq + 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
    out = full[:, 1:tokens + 1, :hq]
    assert m.attend(cache, q, lens, out=out).data_ptr() == out.data_ptr()
    assert torch.equal(out, want)
    assert (full[:, 0] == 7).all() and (full[:, -1] == 7).all() and (full[:, :, hq] == 7).all()
    qt = q.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)   # head-major
    ot = torch.empty(2, hq, tokens, D, dtype=torch.bfloat16, device="cuda").permute(0, 2, 1, 3)
    m.attend(cache, qt, lens, out=ot)
    assert torch.equal(ot, want)


@pytest.mark.parametrize("fmt", ["q4_0", "nvfp4"])
@pytest.mark.parametrize("tokens,hq,n", [(1, 4, 9000), (5, 8, 3000), (140, 4, 700)])
def test_attend_is_deterministic_and_capturable(fmt, tokens, hq, n):
    """Equal bits from call to call, on another stream, and replayed from a CUDA graph with a longer cache."""
    need_gpu()
    m, case = wq(), Case(41, fmt, 2, 128, 2, n, 16)
    cache, lens = case.upload(), ints([n, n - 100])
    q = bf16(case.rng, 2, tokens, hq, 128).cuda()
    ws = torch.empty(max(1, m.attend_workspace_bytes(cache, 2, tokens, hq)), dtype=torch.uint8, device="cuda")
    want = m.attend(cache, q, lens, workspace=ws).clone()
    ws.fill_(0xFF)                                        # the workspace needs no initial contents
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert torch.equal(m.attend(cache, q, lens), want)
    torch.cuda.current_stream().wait_stream(side)
    out = torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.attend(cache, q, lens, out=out, workspace=ws)
    for _ in range(3):
        out.fill_(0)
        g.replay()
        assert torch.equal(out, want)
    lens.sub_(60)
    g.replay()
    assert torch.equal(out, m.attend(cache, q, lens)) and m.last_device_status() == 0


def test_offsets_past_32_bits():
    """Code arrays of more than 2^32 bytes each: rows are found, written and read at both ends."""
    need_gpu()
    m = wq()
    pages, H, D, size = 70000, 8, 128, 128                # 4.6e9 bytes of codes for K, the same for V
    table = torch.tensor([[0, pages - 1, 33, pages - 2]], dtype=torch.int32, device="cuda")
    cache = m.kv_alloc("q4_0", pages, size, H, D, table)
    k = bf16(np.random.default_rng(50), 1, 400, H, D)
    m.kv_append(cache, k.cuda(), k.cuda())
    got = m.kv_read(cache, 400, out_f32=True)[1].cpu().numpy()
    c, s = OK.encode_rows("q4_0", k.float().numpy())
    want = OK.decode_rows("q4_0", c, s)
    assert np.array_equal(got, want)
    for tokens in (1, 130):
        q = bf16(np.random.default_rng(51), 1, tokens, H, D)
        out = m.attend(cache, q.cuda(), ints([400]), out_f32=True).cpu().numpy()
        ref, *_ = OK.attend(q[0].float().numpy(), want[0], want[0], tokens, D ** -0.5, True)
        assert rel_l2(out[0], ref) <= F32_REL_L2
    assert m.last_device_status() == 0


def test_a_page_is_a_packed_weight():
    """wq_dequant reads a contiguous q4_0 cache's K as the weight [heads * page_size, dim] that it is."""
    need_gpu()
    m, case = wq(), Case(52, "q4_0", 4, 64, 1, 64)
    case.upload()
    got = m.dequant("q4_0", case.t[0].view(-1), case.t[1].view(torch.uint8).view(-1), 4 * 64, 64)
    assert np.array_equal(got.cpu().numpy().reshape(4, 64, 64).transpose(1, 0, 2), case.values(0, 64)[0])
