"""The workspace of attention: what wq_attend_workspace_bytes asks for is needed, checked, and enough for every window."""
import ctypes

import pytest
import torch

from tests.gpu_common import need_gpu


@pytest.fixture(scope="module")
def lib():
    from bit_weight_quantized_matmul_gb300 import build
    build.build()
    from bit_weight_quantized_matmul_gb300 import wq
    return wq


@pytest.mark.parametrize("fmt", ["q4_0", "nvfp4"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("batch,tokens,q_heads", [(1, 1, 8), (1, 4, 32), (1, 8, 32), (1, 40, 8), (2, 130, 16)])
def test_calls_without_their_workspace_are_refused(lib, fmt, dim, batch, tokens, q_heads):
    """Long sequences of few heads are shared by blocks and joined, which takes a workspace; nothing is launched without."""
    fake, r = 0x10000, ctypes.byref                  # never dereferenced
    c = lib.wq_kv_cache(fake, fake, fake, fake, None, None, fake, 4096, 4096 * batch, 64, lib.FMT[fmt], 8, dim)
    h = lib.wq_heads(fake, tokens * q_heads * dim, q_heads * dim, dim)
    need = lib.lib.wq_attend_workspace_bytes(r(c), batch, tokens, q_heads, 0)
    rows = batch * tokens * q_heads
    assert need >= 2 * rows * (dim + 2) * 4 and need % 8 == 0     # two partial rows at least for each row
    for ws, size, status in [(None, 0, lib.WQ_ERR_ARG), (None, need, lib.WQ_ERR_ARG), (fake, need - 1, lib.WQ_ERR_ARG),
                             (fake, 0, lib.WQ_ERR_ARG), (fake + 8, need, lib.WQ_ERR_ALIGN)]:
        for window in (0, 1, 100, 100000, 2 ** 63 - 1):
            assert lib.lib.wq_attend(r(c), r(h), r(h), None, batch, tokens, q_heads, fake, None, 0, 0.1, window, 8, ws, size, None) == status
    # one tile of tokens is not shared, and a bound past the capacity is none
    assert lib.lib.wq_attend_workspace_bytes(r(c), batch, tokens, q_heads, 1) == 0
    assert lib.lib.wq_attend_workspace_bytes(r(c), batch, tokens, q_heads, 2 ** 40) == need


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,D", [("q4_0", 64), ("nvfp4", 128)])
@pytest.mark.parametrize("heads,batch,tokens,q_heads", [(1, 1, 1, 1), (2, 1, 3, 8), (38, 4, 1, 38), (1, 3, 20, 1), (2, 1, 40, 4), (1, 2, 150, 2)])
def test_no_window_writes_past_the_workspace(lib, fmt, D, heads, batch, tokens, q_heads):
    need_gpu()
    from tests.test_gpu_kv_cache import Case, bf16, ints
    m, n = lib, 6400
    case = Case(97, fmt, heads, D, batch, n, 64)
    cache, q = case.upload(), bf16(case.rng, batch, tokens, q_heads, D).cuda()
    lens = ints([n - 17 * b for b in range(batch)])
    need = m.attend_workspace_bytes(cache, batch, tokens, q_heads)
    guarded = torch.full((need + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
    for window in (0, 1, 31, 300, 1500, 2047, 2048, 2500, 4100, 6300, 6400, 10 ** 9):
        want = m.attend(cache, q, lens, window=window)
        got = m.attend(cache, q, lens, window=window, workspace=guarded[4096:4096 + need])
        assert torch.equal(got, want)
        assert (guarded[:4096] == 0xA5).all() and (guarded[4096 + need:] == 0xA5).all()
    assert m.last_device_status() == 0
