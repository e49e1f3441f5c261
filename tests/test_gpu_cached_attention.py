"""The example layer (grouped Q/K/V launch, append, attention, output projection) against the oracle, fed in one
prompt and then token by token, and the same from a CUDA graph."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import kv as OK
from oracle import linear as L
from oracle import quant as Q
from tests.gpu_common import need_gpu, wq, REL_L2_TOL
from tests.helpers import rel_l2

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


def bf16_round(a):
    return torch.from_numpy(np.asarray(a, np.float32)).bfloat16().float().numpy()


@pytest.mark.parametrize("fmt", ["q4_0", "nvfp4"])
@pytest.mark.parametrize("heads,dim,prompt", [(2, 64, 7), (3, 128, 45)])
def test_layer_matches_the_oracle(fmt, heads, dim, prompt):
    """Per step the oracle computes the layer on the cache's own contents, read back: a K or V element on the other side
    of a bf16 rounding can move a code by a step, which is no error of the layer.  Three rounded stages (Q/K/V,
    attention, output) of REL_L2_TOL each at most.  The cache itself: every element within half of its block's largest
    value of the oracle's (the widest step of a code is a third of it, and the block's scale can move by a sixteenth)."""
    need_gpu()
    import cached_attention as ex
    m = wq()
    d, batch = heads * dim, 2
    rng = np.random.default_rng(60)
    wqkv, wo = (rng.standard_normal((n, d)).astype(np.float32) * 0.05 for n in (3 * d, d))
    g = None
    if fmt == "nvfp4":
        g = tuple(torch.tensor([x], device="cuda") for x in (0.002, 0.002))
    layer = ex.CachedAttention(torch.from_numpy(wqkv).cuda(), torch.from_numpy(wo).cuda(), heads, dim, batch, prompt + 8, fmt, fmt,
                               page=16, g=g)
    pqkv, po = Q.PACK[fmt](wqkv), Q.PACK[fmt](wo)
    block, at = (32 if fmt == "q4_0" else 16), 0
    for n in [prompt] + [1] * 4:
        x = torch.from_numpy(rng.standard_normal((batch, n, d)).astype(np.float32)).bfloat16()
        y = layer(x.cuda()).float().cpu().numpy()
        qkv = bf16_round(L.linear_w4a16(x.float().numpy().reshape(-1, d), pqkv, None)).reshape(batch, n, 3, heads, dim)
        held = [t.cpu().numpy() for t in m.kv_read(layer.cache, at + n, out_f32=True, batch=batch)]
        for j in range(2):
            want = OK.decode_rows(fmt, *OK.encode_rows(fmt, qkv[:, :, 1 + j], None if g is None else 0.002), None if g is None else 0.002)
            off = np.abs(held[j][:, at:] - want).reshape(-1, block)
            assert (off <= 0.5 * np.abs(want).reshape(-1, block).max(1, keepdims=True)).all()
        at += n
        for b in range(batch):
            att, *_ = OK.attend(qkv[b, :, 0], held[0][b], held[1][b], n, dim ** -0.5, True)
            want = L.linear_w4a16(bf16_round(att).reshape(n, d), po, None).reshape(n, d)
            assert rel_l2(y[b], want) <= 3 * REL_L2_TOL
    assert layer.lens.tolist() == [prompt + 4] * batch and m.last_device_status() == 0


def test_ragged_prompts_and_a_graph():
    """Sequences of unequal prompts in one call give each what it gives alone; a captured step continues them."""
    need_gpu()
    import cached_attention as ex
    m = wq()
    torch.manual_seed(3)
    w = [torch.randn(3 * 256, 256, device="cuda") * 0.05, torch.randn(256, 256, device="cuda") * 0.05]
    x = torch.randn(3, 40, 256, device="cuda").bfloat16()
    counts = torch.tensor([40, 1, 23], dtype=torch.int32, device="cuda")
    step = torch.randn(3, 1, 256, device="cuda").bfloat16()
    together = ex.CachedAttention(w[0], w[1], 4, 64, 3, 64, page=16)
    y = together(x, counts)
    graph = torch.cuda.CUDAGraph()
    before = together.lens.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        together(step)                                   # warm up; the lengths go back, the token is written again
    torch.cuda.current_stream().wait_stream(side)
    together.lens.copy_(before)
    with torch.cuda.graph(graph):
        z = together(step)
    together.lens.copy_(before)
    graph.replay()
    for b, n in enumerate(counts.tolist()):
        alone = ex.CachedAttention(w[0], w[1], 4, 64, 1, 64, page=64)
        assert rel_l2(y[b, :n].float().cpu().numpy(), alone(x[b:b + 1, :n].contiguous())[0].float().cpu().numpy()) <= REL_L2_TOL
        assert rel_l2(z[b].float().cpu().numpy(), alone(step[b:b + 1])[0].float().cpu().numpy()) <= REL_L2_TOL
    assert together.lens.tolist() == [41, 2, 24] and m.last_device_status() == 0


def test_example_runs():
    need_gpu()
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "cached_attention.py"), "--prompt", "70", "--steps", "5", "--fmt",
                        "nvfp4"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "78 tokens" in r.stdout, r.stdout + r.stderr
