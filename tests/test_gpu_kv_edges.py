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
