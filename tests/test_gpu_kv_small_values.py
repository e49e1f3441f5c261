"""Attention keeps its precision whatever the size of V and K: small and large values, blocks of very different size side by
side and one after the other, under weights that one token dominates.

The bounds are those of test_gpu_kv_cache.py (each operand of a product rounded to 11 significant bits at most), here against
values of every size: relative L2 of the fp32 output 1e-3, by block of 32 elements where the blocks differ in size."""
import numpy as np
import pytest
import torch

from oracle import kv as OK
from tests.gpu_common import need_gpu, wq
from tests.helpers import rel_l2
from tests.test_gpu_kv_cache import F32_REL_L2, Case, bf16, ints

pytestmark = pytest.mark.gpu

TOKENS = [1, 8, 12, 20]             # query tokens of 2 heads: each form of the few-row kernel, and the many-row kernel
FMTS = pytest.mark.parametrize("fmt", ["q4_0", "nvfp4"])


def peaked(seed, fmt, D, n, k_std, v_of, nats, tokens, page=64, g=None):
    """One cached head over n tokens whose token n // 3 scores about `nats` above the rest for every query row; v_of(rng, n, D)
    gives V.  Returns the case and q."""
    case = Case(seed, fmt, 1, D, 1, n, page)
    if fmt == "nvfp4" and g is not None:
        case.g = (np.float32(g[0]), np.float32(g[1]))
    rng = case.rng
    base = rng.choice([-1.0, 1.0], D)
    k = rng.standard_normal((n, D)) * k_std
    k[n // 3] = base * nats * k_std / np.sqrt(D)             # scale * q . k = D^-0.5 * (D / k_std) * ... = nats
    q = (base + 0.05 * rng.standard_normal((1, tokens, 2, D))) / k_std
    page_of, off = case.at(0, np.arange(n))
    for j, x in enumerate((k, v_of(rng, n, D))):
        x = torch.from_numpy(np.asarray(x, np.float32)).bfloat16().float().numpy()
        codes, scales = OK.encode_rows(fmt, x, case.g[j])
        case.rows[j][0][page_of, 0, off] = codes
        case.rows[j][1][page_of, 0, off] = scales
    return case, torch.from_numpy(q.astype(np.float32)).bfloat16()


def check(case, q, n, blocks=1, bound=F32_REL_L2):
    """Elementwise against the bound, and the relative L2 of each of `blocks` equal ranges of the elements."""
    m, tokens = wq(), q.shape[1]
    got, lse = m.attend(case.upload(), q.cuda(), ints([n]), out_f32=True, return_lse=True)
    assert m.last_device_status() == 0
    k, v = case.values(0, n)
    ref, rlse, mean, top = OK.attend(q[0].float().numpy(), k, v, tokens, case.D ** -0.5, True)
    got, lse = got[0].cpu().double().numpy(), lse[0].cpu().double().numpy()
    limit = (2.0 ** -11 * (2 * top[..., None] + 4) + 2.0 ** -20) * mean
    errs = [rel_l2(a, b) for a, b in zip(np.split(got, blocks, -1), np.split(ref, blocks, -1))]
    assert max(errs) <= bound, errs
    assert np.all(np.abs(got - ref) <= limit + 1e-30), np.max(np.abs(got - ref) / (limit + 1e-30))
    assert np.all(np.abs(lse - rlse) <= 2.0 ** -11 * top + 2.0 ** -20 * np.abs(rlse) + 2.0 ** -20)


def v_with_a_mean(std):
    return lambda rng, n, D: (rng.standard_normal((n, D)) + 1.0) * std


@FMTS
@pytest.mark.parametrize("tokens", TOKENS)
@pytest.mark.parametrize("v_std", [1.0, 1e-2, 1e-3, 1e-4, 1e-5])
@pytest.mark.parametrize("D,nats", [(64, 8.0), (128, 11.0)])
def test_small_values_under_a_dominant_token(fmt, tokens, v_std, D, nats):
    """8192 tokens, each with a weight e^-8 or e^-11 of the largest, that make up most of the output, or a tenth of it."""
    need_gpu()
    g = (0.0074, 0.0021 * v_std) if fmt == "nvfp4" else None
    case, q = peaked(90, fmt, D, 8192, 1.0, v_with_a_mean(v_std), nats, tokens, g=g)
    check(case, q, 8192)


@pytest.mark.parametrize("tokens", TOKENS)
@pytest.mark.parametrize("v_std", [1e-3, 1e-4])
def test_small_values_over_a_long_sequence(tokens, v_std):
    need_gpu()
    n = 60001
    case, q = peaked(91, "q4_0", 64, n, 1.0, v_with_a_mean(v_std), 10.0, tokens)
    check(case, q, n)


@pytest.mark.parametrize("tokens", TOKENS)
@pytest.mark.parametrize("sizes", [(1e-4, 1e2, 1e-3, 1.0), (1e-2, 1e5, 1.0, 30.0), (2.4e5, 1e-2, 6e4, 1e3), (1e-5, 1e-4, 1e-3, 1e-2)])
def test_blocks_of_different_size_in_a_row(tokens, sizes):
    """The four blocks of 32 elements of every V row differ in size by up to 10^7, to the largest that fp16 scales hold."""
    need_gpu()
    size = np.repeat(np.array(sizes), 32)
    case, q = peaked(92, "q4_0", 128, 6000, 1.0, lambda rng, n, D: (rng.standard_normal((n, D)) + 1.0).clip(-2, 2) * size, 9.0, tokens)
    check(case, q, 6000, blocks=4)


@pytest.mark.parametrize("tokens", TOKENS)
@pytest.mark.parametrize("small,large", [(1e-3, 1e2), (1e-2, 1.5e5), (1.0, 6e4)])
@pytest.mark.parametrize("hidden", [True, False])
def test_rows_of_different_size_one_after_the_other(tokens, small, large, hidden):
    """A few V rows are 10^5 or more times larger than the rest.  hidden: their keys make their weights vanish, and what
    is left is small."""
    need_gpu()
    n = 5000
    at = np.arange(40, n, 577)

    def v_of(rng, n, D):
        v = (rng.standard_normal((n, D)) + 1.0).clip(-2, 2) * small
        v[at] *= large / small
        return v
    case, q = peaked(93, "q4_0", 64, n, 1.0, v_of, 9.0, tokens)
    if hidden:
        page, off = case.at(0, at)
        base = np.sign(q[0, 0, 0].float().numpy())
        codes, scales = OK.encode_rows("q4_0", np.broadcast_to(-base * 100.0 / 8.0, (len(at), 64)).astype(np.float32))
        case.rows[0][0][page, 0, off], case.rows[0][1][page, 0, off] = codes, scales
    check(case, q, n)


@FMTS
@pytest.mark.parametrize("tokens", TOKENS)
@pytest.mark.parametrize("k_std", [1e-4, 1e-2, 300.0])
def test_keys_of_any_size(fmt, tokens, k_std):
    """Keys far from 1 with queries that make up for it."""
    need_gpu()
    g = (0.0074 * k_std, 0.0021) if fmt == "nvfp4" else None
    case, q = peaked(94, fmt, 128, 3000, k_std, v_with_a_mean(1.0), 7.0, tokens, g=g)
    check(case, q, 3000)


@pytest.mark.parametrize("tokens", TOKENS)
def test_keys_with_the_largest_scales(tokens):
    """K blocks whose scale is 8192 or more beside small ones, some tokens only."""
    need_gpu()
    n = 2000
    case, q = peaked(95, "q4_0", 64, n, 1.0, v_with_a_mean(1.0), 6.0, tokens)
    rng, at = np.random.default_rng(96), np.arange(5, n, 97)
    page, off = case.at(0, at)
    k = rng.standard_normal((len(at), 64))
    k[:, :32] *= 1.2e5 / np.abs(k[:, :32]).max(1, keepdims=True)
    codes, scales = OK.encode_rows("q4_0", k.astype(np.float32))
    assert (np.abs(scales[:, 0].astype(np.float32)) >= 8192).all()
    case.rows[0][0][page, 0, off], case.rows[0][1][page, 0, off] = codes, scales
    q[..., :32] *= 2.0 ** -17              # those blocks' part of a score is of order one
    check(case, q, n)
