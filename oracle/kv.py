"""The 4-bit KV cache and attention over it (oracle side).

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

A cached row of one head is a weight row of the same format: ``quant.q4_0_pack`` (blocks of 32,
PR "Run quantized Whisper on the fused Metal decode path", "Summary") or ``quant.nvfp4_quantize``
with a static g (model card "whisper-large-v3-turbo -- NVFP4", "What is quantized").  Attention is
the textbook definition in fp64 on the decoded values.
"""
import numpy as np

from . import quant as Q


def encode_rows(fmt, x, g=None):
    """x float32 [..., D] -> (codes uint8 [..., D / 2], scales: fp16 [..., D / 32] or uint8 [..., D / 16])."""
    x = np.asarray(x, np.float32)
    flat = x.reshape(-1, x.shape[-1])
    if fmt == "q4_0":
        p = Q.q4_0_pack(flat)
        codes, scales = Q.pack_nibbles(p["codes"]), p["d"].reshape(x.shape[:-1] + (-1,))
    else:
        c, s, _ = Q.nvfp4_quantize(flat, np.float32(1.0 if g is None else g))
        codes, scales = Q.pack_nibbles(c), s.reshape(x.shape[:-1] + (-1,))
    return codes.reshape(x.shape[:-1] + (-1,)), scales


def decode_rows(fmt, codes, scales, g=None):
    """The float32 values [..., D] of encoded rows."""
    shape = codes.shape[:-1] + (2 * codes.shape[-1],)
    c = Q.unpack_nibbles(codes).reshape(codes.size * 2 // shape[-1], shape[-1])
    if fmt == "q4_0":
        p = dict(codes=c.reshape(-1), d=np.asarray(scales, np.float16).reshape(-1), N=c.shape[0], K=shape[-1])
        return Q.q4_0_dequant(p).reshape(shape)
    s = np.asarray(scales, np.uint8).reshape(c.shape[0], shape[-1] // Q.NVFP4_BLOCK)
    return Q.nvfp4_dequant_parts(c, s, np.float32(1.0 if g is None else g)).reshape(shape)


def attend(q, k, v, n_q, scale, causal, window=0):
    """q [L, Hq, D]; k, v [T, H, D]: one sequence, whose last n_q tokens are the first n_q rows of q.
    Returns out [L, Hq, D], lse [L, Hq] in fp64, and two arrays for error bounds: the weighted mean of
    |v| [L, Hq, D] and the largest sum of |scale q k| over the visible tokens [L, Hq]."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    L, Hq, D = q.shape
    T, H = k.shape[:2]
    out, mean, lse, top = np.zeros((L, Hq, D)), np.zeros((L, Hq, D)), np.full((L, Hq), -np.inf), np.zeros((L, Hq))
    t = np.arange(T)
    for i in range(min(L, n_q)):
        pos = T - n_q + i
        seen = np.ones(T, bool)
        if causal:
            seen &= t <= pos
        if window:
            seen &= t > pos - window
        if not seen.any():
            continue
        for h in range(Hq):
            kh, vh = k[seen, h * H // Hq], v[seen, h * H // Hq]
            s = scale * (kh @ q[i, h])
            m = s.max()
            e = np.exp(s - m)
            p = e / e.sum()
            lse[i, h] = m + np.log(e.sum())
            out[i, h], mean[i, h] = p @ vh, p @ np.abs(vh)
            top[i, h] = (abs(scale) * (np.abs(kh) @ np.abs(q[i, h]))).max()
    return out, lse, mean, top
