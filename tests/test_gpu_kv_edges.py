"""Ends of the argument ranges of attention over the 4-bit cache."""
import numpy as np
import pytest
import torch

from oracle import kv as OK
from tests.gpu_common import need_gpu, wq
from tests.test_gpu_kv_cache import Case, bf16, check_attend, ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("signs", [(-1, 1), (1, -1), (-1, -1)])
@pytest.mark.parametrize("tokens,scale", [(1, None), (6, 0.2), (6, -0.2), (40, None), (40, -0.2)])
def test_attend_with_negative_global_scales(signs, tokens, scale):
    """A negative static g of K or V, with few and with many rows."""
    need_gpu()
    case = Case(83, "nvfp4", 2, 128, 2, 400, 16)
    case.g = tuple(np.float32(s * g) for s, g in zip(signs, case.g))
    check_attend(case, tokens, 4, [400, 211], scale=scale)


@pytest.mark.parametrize("fmt", ["q4_0", "nvfp4"])
@pytest.mark.parametrize("tokens", [4, 40])
@pytest.mark.parametrize("window", [0, 20])
@pytest.mark.parametrize("page", [0, 16])
def test_attend_lengths_past_the_capacity(fmt, tokens, window, page):
    """A length past the capacity is reported; the query rows keep their positions at its end, and see what there is."""
    need_gpu()
    m, case = wq(), Case(84, fmt, 2, 64, 3, 64, page)
    lens = [70, 64, 2 ** 31 - 1]
    q = bf16(case.rng, 3, tokens, 4, 64)
    assert m.last_device_status() == 0
    out, lse = m.attend(case.upload(), q.cuda(), ints(lens), window=window, out_f32=True, return_lse=True)
    assert m.last_device_status() == m.WQ_ERR_ARG
    for b in range(3):
        k, v = case.values(b, 64)
        p = lens[b] - tokens + np.arange(tokens)
        for i in range(tokens):
            lo = max(0, p[i] - window + 1) if window else 0
            hi = min(64, p[i] + 1)
            got, gl = out[b, i].cpu().double().numpy(), lse[b, i].cpu().double().numpy()
            if hi <= lo:
                assert not got.any() and np.isneginf(gl).all()
                continue
            ref, rlse, mean, top = OK.attend(q[b, i:i + 1].float().numpy(), k[lo:hi], v[lo:hi], 1, 0.125, False)
            assert np.all(np.abs(got - ref[0]) <= (2.0 ** -11 * (2 * top[0][:, None] + 4) + 2.0 ** -20) * mean[0] + 1e-30)
            assert np.all(np.abs(gl - rlse[0]) <= 2.0 ** -11 * top[0] + 2.0 ** -20 * np.abs(rlse[0]) + 2.0 ** -20)


@pytest.mark.parametrize("tokens", [1, 40])
@pytest.mark.parametrize("window", [20000, 2 ** 31, 2 ** 63 - 1])
def test_attend_with_a_window_wider_than_all(tokens, window):
    """Is planned and computed as no window: equal bits, and as many launches."""
    need_gpu()
    m, case = wq(), Case(85, "q4_0", 1, 64, 1, 20000, 64)
    cache, q, lens = case.upload(), bf16(case.rng, 1, tokens, 2, 64).cuda(), ints([20000])
    before = m.lib.wq_kernel_launches()
    want = m.attend(cache, q, lens)
    launches = m.lib.wq_kernel_launches() - before
    got = m.attend(cache, q, lens, window=window)
    assert torch.equal(got, want) and m.lib.wq_kernel_launches() - before == 2 * launches


@pytest.mark.parametrize("tokens", [1, 3, 40])
@pytest.mark.parametrize("window", [2 ** 31, 2 ** 63 - 40, 2 ** 63 - 1])
@pytest.mark.parametrize("page", [0, 16])
def test_the_widest_windows_of_rows_before_the_first_token(tokens, window, page):
    """p - window is below every 64-bit number for some of these rows: they see nothing, the others all there is."""
    need_gpu()
    m, case = wq(), Case(86, "q4_0", 2, 64, 5, 48, page)
    cache, q, lens = case.upload(), bf16(case.rng, 5, tokens, 4, 64).cuda(), ints([0, 1, 2, 17, 45])
    want, wlse = m.attend(cache, q, lens, return_lse=True)
    got, lse = m.attend(cache, q, lens, window=window, return_lse=True)
    assert torch.equal(got, want) and torch.equal(lse, wlse) and m.last_device_status() == 0


def test_memory_that_is_not_the_caches_devices_is_refused(monkeypatch):
    """Before any launch: host memory, another device's, a current device that is not the cache's."""
    need_gpu()
    m, case = wq(), Case(87, "q4_0", 2, 64, 2, 20000, 64)
    cache, q, lens = case.upload(), bf16(case.rng, 2, 1, 4, 64).cuda(), ints([20000, 3])
    k = bf16(case.rng, 2, 1, 2, 64).cuda()
    need = m.attend_workspace_bytes(cache, 2, 1, 4)
    assert need > 0
    want = m.attend(cache, q, lens)
    t, launches = cache.tensors, m.lib.wq_kernel_launches()
    workspaces = [torch.empty(need, dtype=torch.uint8), torch.empty(need, dtype=torch.float32, device="cuda"),
                  torch.empty(2 * need, dtype=torch.uint8, device="cuda")[::2]]
    calls = [lambda w=w: m.attend(cache, q, lens, workspace=w) for w in workspaces]
    calls += [lambda: m.attend(cache, q.cpu(), lens), lambda: m.attend(cache, q, lens.cpu()), lambda: m.attend(cache, q, lens, lens.cpu()),
              lambda: m.attend(cache, q, lens, out=torch.empty_like(q, device="cpu")), lambda: m.kv_append(cache, k, k.cpu()),
              lambda: m.kv_append(cache, k, k, lens.cpu()), lambda: m.kv_read(cache, 3, counts=lens.cpu()),
              lambda: m.KVCache("q4_0", t[0], t[1], t[2].cpu(), t[3], t[4]), lambda: m.KVCache("q4_0", t[0], t[1].cpu(), t[2], t[3], t[4]),
              lambda: m.KVCache("q4_0", *t[:4], t[4].cpu())]
    for call in calls:
        with pytest.raises(AssertionError):
            call()
    with pytest.raises(m.WQError):
        m.attend(cache, q, lens, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    here = [lambda: m.attend(cache, q, lens), lambda: m.kv_append(cache, k, k), lambda: m.kv_read(cache, 3)]
    with monkeypatch.context() as mp:
        mp.setattr(torch._C, "_cuda_getDevice", lambda: 1)
        for call in here:
            with pytest.raises(AssertionError):
                call()
    cache.index = 1
    for call in here:
        with pytest.raises(AssertionError):
            call()
    cache.index = 0
    assert m.lib.wq_kernel_launches() == launches
    assert torch.equal(m.attend(cache, q, lens, workspace=torch.empty(need, dtype=torch.uint8, device="cuda")), want)
