"""The KV cache entry points refuse what they cannot take before any launch (no GPU needed: every
call here fails its checks, or only computes sizes), and the oracle of the cache is pinned."""
import ctypes

import numpy as np
import pytest

from oracle import kv as OK
from oracle import quant as Q


@pytest.fixture(scope="module")
def wq():
    from bit_weight_quantized_matmul_gb300 import build
    build.build()
    from bit_weight_quantized_matmul_gb300 import wq as mod
    return mod


FAKE = 0x10000     # never dereferenced: every call below fails its checks first


def cache(wq, **kw):
    c = wq.wq_kv_cache(FAKE, FAKE, FAKE, FAKE, None, None, FAKE, 4, 16, 64, wq.WQ_Q4_0, 8, 128)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def heads(wq, p=FAKE, batch=8192, token=1024, head=128):
    return wq.wq_heads(p, batch, token, head)


BAD_CACHE = [(dict(fmt=1), "WQ_ERR_FMT"), (dict(fmt=3), "WQ_ERR_FMT"), (dict(dim=96), "WQ_ERR_SHAPE"),
             (dict(dim=256), "WQ_ERR_SHAPE"), (dict(page_size=24), "WQ_ERR_SHAPE"), (dict(page_size=0), "WQ_ERR_SHAPE"),
             (dict(page_size=-16), "WQ_ERR_ARG"), (dict(heads=0), "WQ_ERR_ARG"), (dict(pages=-1), "WQ_ERR_ARG"),
             (dict(table_ld=-1), "WQ_ERR_ARG"), (dict(k_codes=None), "WQ_ERR_ARG"), (dict(v_scales=None), "WQ_ERR_ARG"),
             (dict(k_scales=FAKE + 8), "WQ_ERR_ALIGN"), (dict(v_codes=FAKE + 4), "WQ_ERR_ALIGN"),
             (dict(table=FAKE + 2), "WQ_ERR_ALIGN"), (dict(fmt=2, k_g=FAKE + 1), "WQ_ERR_ALIGN")]


@pytest.mark.parametrize("change,status", BAD_CACHE)
def test_bad_caches(wq, change, status):
    c, h, want = cache(wq, **change), heads(wq), getattr(wq, status)
    L, r = wq.lib, ctypes.byref
    assert L.wq_kv_append(r(c), r(h), r(h), 2, 3, None, None, None) == want
    assert L.wq_kv_read(r(c), r(h), r(h), 2, 3, None, None, 0, None) == want
    assert L.wq_attend(r(c), r(h), r(h), None, 2, 3, 32, FAKE, None, 0, 0.1, 0, 8, None, 0, None) == want
    assert L.wq_attend_workspace_bytes(r(c), 2, 3, 32, 0) == 0


def test_bad_move_arguments(wq):
    c, h, L, r = cache(wq), heads(wq), wq.lib, ctypes.byref
    assert L.wq_kv_append(None, r(h), r(h), 2, 3, None, None, None) == wq.WQ_ERR_ARG
    assert L.wq_kv_append(r(c), None, r(h), 2, 3, None, None, None) == wq.WQ_ERR_ARG
    assert L.wq_kv_append(r(c), r(h), r(heads(wq, p=None)), 2, 3, None, None, None) == wq.WQ_ERR_ARG
    assert L.wq_kv_append(r(c), r(heads(wq, p=FAKE + 8)), r(h), 2, 3, None, None, None) == wq.WQ_ERR_ALIGN
    assert L.wq_kv_append(r(c), r(heads(wq, token=1020)), r(h), 2, 3, None, None, None) == wq.WQ_ERR_ALIGN
    assert L.wq_kv_append(r(c), r(heads(wq, head=-128)), r(h), 2, 3, None, None, None) == wq.WQ_ERR_ARG
    assert L.wq_kv_append(r(c), r(h), r(h), -1, 3, None, None, None) == wq.WQ_ERR_ARG
    assert L.wq_kv_append(r(c), r(h), r(h), 1 << 20, 1 << 12, None, None, None) == wq.WQ_ERR_SHAPE
    assert L.wq_kv_append(r(c), r(h), r(h), 2, 3, FAKE + 2, None, None) == wq.WQ_ERR_ALIGN
    assert L.wq_kv_append(r(c), r(h), r(h), 2, 3, None, FAKE + 1, None) == wq.WQ_ERR_ALIGN
    assert L.wq_kv_append(r(cache(wq, table=None)), r(h), r(h), 17, 3, None, None, None) == wq.WQ_ERR_SHAPE
    assert L.wq_kv_append(r(c), None, None, 0, 3, None, None, None) == wq.WQ_OK     # nothing to do
    assert L.wq_kv_append(r(c), None, None, 2, 0, None, None, None) == wq.WQ_OK
    assert L.wq_kv_read(r(c), None, None, 2, 3, None, None, 0, None) == wq.WQ_ERR_ARG
    assert L.wq_kv_read(r(c), r(h), r(h), 2, 3, None, None, 2, None) == wq.WQ_ERR_ARG
    # fp32 rows need strides of 4 elements, bf16 rows of 8
    assert L.wq_kv_read(r(c), r(heads(wq, token=1026)), r(h), 2, 3, None, None, 1, None) == wq.WQ_ERR_ALIGN


def test_bad_attend_arguments(wq):
    c, h, L, r = cache(wq), heads(wq), wq.lib, ctypes.byref

    def call(c=c, q=h, out=h, lse=None, batch=2, tokens=3, q_heads=32, lens=FAKE, counts=None, max_len=0, scale=0.1, window=0,
             flags=8, ws=None, ws_bytes=0):
        return L.wq_attend(r(c), r(q), r(out), lse, batch, tokens, q_heads, lens, counts, max_len, scale, window, flags, ws,
                           ws_bytes, None)

    assert call(q_heads=12) == wq.WQ_ERR_SHAPE          # not a multiple of the cache's 8 heads
    assert call(lens=None) == wq.WQ_ERR_ARG
    assert call(lens=FAKE + 2) == wq.WQ_ERR_ALIGN
    assert call(lse=FAKE + 2) == wq.WQ_ERR_ALIGN
    assert call(flags=2) == wq.WQ_ERR_ARG
    assert call(window=-1) == wq.WQ_ERR_ARG
    assert call(window=5, flags=0) == wq.WQ_ERR_ARG     # a window is a causal one
    assert call(max_len=-1) == wq.WQ_ERR_ARG
    assert call(scale=float("inf")) == wq.WQ_ERR_ARG and call(scale=float("nan")) == wq.WQ_ERR_ARG
    assert call(q=heads(wq, p=FAKE + 2)) == wq.WQ_ERR_ALIGN
    assert call(out=heads(wq, head=132), flags=8) == wq.WQ_ERR_ALIGN
    assert call(batch=-1) == wq.WQ_ERR_ARG and call(tokens=-1) == wq.WQ_ERR_ARG
    assert call(batch=1 << 20, tokens=1 << 12) == wq.WQ_ERR_SHAPE
    assert call(c=cache(wq, table=None), batch=17) == wq.WQ_ERR_SHAPE
    assert call(batch=0) == wq.WQ_OK and call(tokens=0) == wq.WQ_OK and call(q_heads=0) == wq.WQ_OK
    need = L.wq_attend_workspace_bytes(r(c), 1, 1, 8, 0)
    if need:
        assert call(batch=1, tokens=1, q_heads=8, ws=None, ws_bytes=need) == wq.WQ_ERR_ARG
        assert call(batch=1, tokens=1, q_heads=8, ws=FAKE, ws_bytes=need - 1) == wq.WQ_ERR_ARG
        assert call(batch=1, tokens=1, q_heads=8, ws=FAKE + 8, ws_bytes=need) == wq.WQ_ERR_ALIGN


def test_workspace_is_the_same_for_the_same_sizes(wq):
    c = cache(wq, table_ld=4096)
    r = ctypes.byref(c)
    sizes = [wq.lib.wq_attend_workspace_bytes(r, b, t, 32, n) for b in (1, 3, 64) for t in (1, 5, 700) for n in (0, 1, 9000)]
    assert sizes == [wq.lib.wq_attend_workspace_bytes(r, b, t, 32, n) for b in (1, 3, 64) for t in (1, 5, 700)
                     for n in (0, 1, 9000)]
    assert wq.lib.wq_attend_workspace_bytes(r, 0, 1, 32, 0) == 0 and wq.lib.wq_attend_workspace_bytes(r, 1, 1, 30, 0) == 0


# ------------------------------------------------------------------ the oracle
@pytest.mark.parametrize("fmt", ["q4_0", "nvfp4"])
@pytest.mark.parametrize("D", [64, 128])
def test_oracle_rows_are_weight_rows(fmt, D):
    x = np.random.default_rng(3).standard_normal((5, 2, D)).astype(np.float32)
    g = np.float32(0.0021) if fmt == "nvfp4" else None
    codes, scales = OK.encode_rows(fmt, x, g)
    assert codes.shape == (5, 2, D // 2) and scales.shape == (5, 2, D // (32 if fmt == "q4_0" else 16))
    got = OK.decode_rows(fmt, codes, scales, g)
    if fmt == "q4_0":
        p = Q.q4_0_pack(x.reshape(10, D))
        packed, blob = Q.to_blobs(p)
        assert codes.tobytes() == packed and blob.startswith(scales.tobytes())
        assert np.array_equal(got.reshape(10, D), Q.q4_0_dequant(p))
    # half a step of the block's scale, q4_0's clipped side a whole one; NVFP4's largest gap is 2 scales
    step = np.abs(x).reshape(5, 2, -1, 32).max(-1).repeat(32, -1).reshape(x.shape)
    assert np.all(np.abs(got - x) <= step * (1 / 8 + 1e-3 if fmt == "q4_0" else 1 / 6 + 0.07))


def test_oracle_attention_by_hand():
    # one head of 2 elements, three tokens: softmax of (0, ln 2, ln 4) weighs 1 : 2 : 4
    k = np.array([[[0.0, 9.0]], [[np.log(2), 0.0]], [[np.log(4), 1.0]]])
    v = np.array([[[1.0, 0.0]], [[0.0, 1.0]], [[7.0, -7.0]]])
    q = np.array([[[1.0, 0.0]]])
    out, lse, _, _ = OK.attend(q, k, v, 1, 1.0, True)
    assert np.allclose(out[0, 0], [(1 + 28) / 7, (2 - 28) / 7]) and np.isclose(lse[0, 0], np.log(7))
    out, lse, _, _ = OK.attend(q, k, v, 1, 1.0, True, window=2)
    assert np.allclose(out[0, 0], [28 / 6, (2 - 28) / 6]) and np.isclose(lse[0, 0], np.log(6))
    # two query rows, causal: the first sees two tokens; four rows on three tokens: the first sees none
    q4 = np.repeat(q, 4, 0)
    out, lse, _, _ = OK.attend(q4[:2], k, v, 2, 1.0, True)
    assert np.isclose(lse[0, 0], np.log(3)) and np.isclose(lse[1, 0], np.log(7))
    out, lse, _, _ = OK.attend(q4, k, v, 4, 1.0, True)
    assert lse[0, 0] == -np.inf and not out[0].any() and np.isclose(lse[3, 0], np.log(7))
    # rows past the sequence's count are empty
    _, lse, _, _ = OK.attend(q4, k, v, 1, 1.0, False)
    assert np.isclose(lse[0, 0], np.log(7)) and np.all(lse[1:] == -np.inf)
