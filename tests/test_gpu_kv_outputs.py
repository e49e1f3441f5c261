"""Outputs that a call makes together: small ones share an allocation, large ones have their own, so that what is kept of a call
holds little else alive."""
import pytest
import torch

from tests.gpu_common import need_gpu, wq
from tests.test_gpu_kv_cache import Case, bf16, ints
from tests.test_gpu_kv_select import cuda, random_trees

pytestmark = pytest.mark.gpu
SMALL = 65536


def check(outputs):
    """Contiguous, apart from each other, and no storage of more than the small ones together, or than the tensor itself."""
    spans = []
    for t in outputs:
        n, held = t.numel() * t.element_size(), t.untyped_storage().nbytes()
        assert t.is_contiguous() and (n == 0 or t.data_ptr() % 16 == 0)
        assert held == n if n > SMALL else held <= len(outputs) * SMALL
        if n:
            spans.append((t.data_ptr(), t.data_ptr() + n))
    spans.sort()
    assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:]))


@pytest.mark.parametrize("tokens", [0, 1, 37, 8192, 8193, 16384, 16385, 300000])
@pytest.mark.parametrize("batch", [1, 3, 20000])
def test_reservations(tokens, batch):
    need_gpu()
    m = wq()
    cache = m.kv_alloc("q4_0", 40, 16, 1, 64, torch.full((batch, 3), -1, dtype=torch.int32, device="cuda"))
    got = m.kv_reserve(cache, ints(list(range(40))), ints([40]), ints([0] * batch), ints([min(tokens, 40)] + [0] * (batch - 1)), tokens)
    check(got)
    slots, positions, starts, granted = (t.cpu() for t in got)
    n = min(tokens, 40)
    assert positions.tolist() == list(range(n)) + [0] * (tokens - n) and granted.tolist() == [n] + [0] * (batch - 1)
    assert starts.tolist() == [0] + [n] * batch and slots.tolist() == [(39 - i // 16) * 16 + i % 16 for i in range(n)] + [-1] * (tokens - n)
    assert m.last_device_status() == 0


@pytest.mark.parametrize("batch,tokens", [(1, 1), (8, 64), (40, 64), (2, 1024), (300, 60), (0, 5)])
def test_masks(batch, tokens):
    need_gpu()
    m, rng = wq(), torch.Generator().manual_seed(1)
    parents = torch.stack([torch.randint(-1, max(i, 1), (batch,), generator=rng) for i in range(tokens)], 1).int().clamp(max=tokens - 1)
    parents = torch.minimum(parents, torch.arange(tokens).int() - 1).cuda()
    check(m.tree_mask(parents))
    assert m.last_device_status() == 0


@pytest.mark.parametrize("out_f32", [False, True])
@pytest.mark.parametrize("batch,tokens,hq", [(1, 1, 4), (2, 64, 2), (2, 256, 2), (2, 257, 2), (2, 300, 40)])
def test_attention_with_its_log_sum_exp(out_f32, batch, tokens, hq):
    need_gpu()
    m, case = wq(), Case(120, "q4_0", 2, 64, 2, 320, 16)
    cache, q, lens = case.upload(), bf16(case.rng, batch, tokens, hq, 64).cuda(), ints([320, 311][:batch])
    got = m.attend(cache, q, lens, out_f32=out_f32, return_lse=True)
    check(got)
    out = torch.empty_like(got[0])
    again = m.attend(cache, q, lens, out_f32=out_f32, return_lse=True, out=out)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    tree = m.tree_mask(cuda(random_trees(case.rng, batch, tokens)))
    check(m.attend(cache, q, lens, tree=tree, return_lse=True, out_f32=out_f32))
    assert m.last_device_status() == 0
