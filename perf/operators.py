"""The 4-bit KV cache: writing it, reading it back, and attention over it, as cases to measure.

A case has an ``op``: "write" appends new tokens to the cache and reads them back, "read" reads a range
back, "attend" is attention over the cache.  Every case gives the cache's format (``fmt``), the number of
K/V heads (``hkv``), the head size (``d``), the page size (``page``; 0: one contiguous slab per sequence)
and the batch.  Ragged lengths run evenly from ``lo`` to ``hi`` over the batch, in an order drawn from the
seed.  ``run`` computes in plain torch operations where ``own`` is false, and calls the library's
entry points where it is true.
"""
import math

import numpy as np
import torch

own = False

# E2M1 magnitudes, and the midpoints between them (ties go to the even code: the flags say whether a tie goes up)
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
MIDS = ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False))


def listed():
    return [
        # one decoding step of 32 audio windows: a token's K and V into the self-attention slabs (20 heads of 64 = 1280)
        dict(name="write step 32x1 h20 d64 q4_0", op="write", fmt="q4_0", batch=32, l=1, lo=1, hi=1, past=447, hkv=20, d=64,
             page=0),
        # the prompts of four requests of unequal length enter a paged cache, behind what it holds of them
        dict(name="write prompts 4x2048 h8 d128 nvfp4", op="write", fmt="nvfp4", batch=4, l=2048, lo=333, hi=2048,
             past=700, hkv=8, d=128, page=64),
        # the encoder's 1500 frames of 16 audio windows: the cross-attention cache, written once per window
        dict(name="write frames 16x1500 h20 d64 q4_0", op="write", fmt="q4_0", batch=16, l=1500, lo=1500, hi=1500, past=0,
             hkv=20, d=64, page=0),
        # a shared prefix of odd length read back for a request that moves elsewhere
        dict(name="read prefix 3x777 h8 d128 q4_0", op="read", fmt="q4_0", batch=3, l=777, lo=401, hi=777, past=19, hkv=8,
             d=128, page=16, f32=True),
        # a long context read back whole, for a consumer that wants bf16
        dict(name="read context 8x16384 h8 d128 nvfp4", op="read", fmt="nvfp4", batch=8, l=16384, lo=12000, hi=16384, past=0,
             hkv=8, d=128, page=64, f32=False),
        # the smallest call: one token of one audio window over its self-attention slab
        dict(name="decode 1x447 h20 d64 q4_0", op="attend", fmt="q4_0", batch=1, l=1, lo=447, hi=447, hq=20, hkv=20, d=64,
             page=0, causal=True, window=0),
        # cross-attention of one decoding step of 16 audio windows over 1500 frames
        dict(name="cross 16x1500 h20 d64 q4_0", op="attend", fmt="q4_0", batch=16, l=1, lo=1500, hi=1500, hq=20, hkv=20, d=64,
             page=0, causal=False, window=0),
        # one token over one very long context, grouped heads: the cache of a single request must fill the machine
        dict(name="decode 1x131071 h32/8 d128 q4_0", op="attend", fmt="q4_0", batch=1, l=1, lo=131071, hi=131071, hq=32,
             hkv=8, d=128, page=64, causal=True, window=0),
        # a serving batch of 64 requests with unequal contexts, small pages
        dict(name="decode 64x1000-8000 h32/8 d128 nvfp4", op="attend", fmt="nvfp4", batch=64, l=1, lo=1000, hi=8000, hq=32,
             hkv=8, d=128, page=16, causal=True, window=0),
        # five drafted tokens checked at once under a sliding window
        dict(name="draft 8x5 3000-9000 h32/4 d128 q4_0", op="attend", fmt="q4_0", batch=8, l=5, lo=3000, hi=9000, hq=32, hkv=4,
             d=128, page=32, causal=True, window=4096),
        # the first decoder pass of four audio windows: 224 prompt tokens over 1500 frames, no causal mask
        dict(name="prompt 4x224 over 1500 h20 d64 nvfp4", op="attend", fmt="nvfp4", batch=4, l=224, lo=1500, hi=1500, hq=20,
             hkv=20, d=64, page=0, causal=False, window=0),
        # a chunk of a long prompt behind what the cache holds of it
        dict(name="chunk 2x1024 over 16384 h32/8 d128 q4_0", op="attend", fmt="q4_0", batch=2, l=1024, lo=9000, hi=16384,
             hq=32, hkv=8, d=128, page=64, causal=True, window=0),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    fmt = rng.choice(["q4_0", "nvfp4"])
    page = rng.choice([0, 16, 32, 48, 64, 128])
    op = rng.choice(["write", "read", "attend", "attend", "attend"])
    heads = rng.choice([(20, 20, 64), (6, 6, 64), (32, 8, 128), (32, 4, 128), (16, 16, 128), (24, 8, 128), (8, 1, 64),
                        (40, 8, 128)])
    hq, hkv, d = heads
    if op in ("write", "read"):
        batch = _log(rng, 1, 64)
        most = 8 * 14000 * 8 * 128 // (batch * hkv * d) if op == "read" else 16 * 1500 * 20 * 64 // (batch * hkv * d)
        l = _log(rng, 1, max(1, min(16384, most)))
        lo = rng.randint(max(1, l // 3), l)
        c = dict(op=op, fmt=fmt, batch=batch, l=l, lo=lo, hi=l, past=rng.choice([0, rng.randint(1, 1000)]), hkv=hkv, d=d,
                 page=page)
        if op == "read":
            c["f32"] = rng.random() < 0.3
        return c
    kind = rng.choice(["token", "token", "some", "many"])
    batch = _log(rng, 1, 64 if kind != "many" else 4)
    l = 1 if kind == "token" else rng.randint(2, 9) if kind == "some" else _log(rng, 17, 1024)
    most = 48 * 4500 * 8 * 128 // (batch * hkv * d)
    if kind == "many":
        most = min(most, 2 * 1024 * 12000 * 32 * 128 // (batch * l * hq * d), 16384)
    hi = max(l, _log(rng, 40, max(41, min(131072, most))))
    lo = rng.randint(max(l, hi // 4), hi)
    causal = rng.random() < 0.7
    window = rng.choice([0, 0, rng.randint(16, 4096)]) if causal else 0
    return dict(op=op, fmt=fmt, batch=batch, l=l, lo=lo, hi=hi, hq=hq, hkv=hkv, d=d, page=page, causal=causal, window=window)


# ------------------------------------------------------------------ inputs
def _lengths(case):
    """The batch's lengths, whatever their order: evenly from lo to hi."""
    b = case["batch"]
    return [case["lo"] + (case["hi"] - case["lo"]) * i // max(1, b - 1) for i in range(b)][::-1]


def _quantise_rows(fmt, x, g):
    """x fp32 [..., d] -> (codes [..., d / 2] uint8, scales): two codes a byte, element 2j in the low nibble."""
    if fmt == "q4_0":
        blk = x.unflatten(-1, (-1, 32))
        at = blk.abs().argmax(-1, keepdim=True)
        scale = (blk.gather(-1, at) / -8.0).to(torch.float16)
        s = scale.float()
        codes = torch.where(s != 0, (torch.round(blk / torch.where(s != 0, s, 1.0)) + 8).clamp(0, 15), 8.0)
        scale = scale.squeeze(-1)
    else:
        blk = x.unflatten(-1, (-1, 16))
        scale = ((blk.abs().amax(-1, keepdim=True) / 6.0) / g).clamp(max=448.0).to(torch.float8_e4m3fn)
        s = scale.float() * g
        v = blk / torch.where(s != 0, s, 1.0)
        a = v.abs().unsqueeze(-1)
        mids = x.new_tensor([m for m, _ in MIDS])
        up = torch.tensor([t for _, t in MIDS], device=x.device)
        codes = ((a > mids) | ((a == mids) & up)).sum(-1) + 8 * torch.signbit(v)
        codes = torch.where(s != 0, codes, 0)
        scale = scale.squeeze(-1).view(torch.uint8)
    c = codes.to(torch.uint8).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), scale


def _values(fmt, codes, scales, g):
    """The values that codes and scales stand for, fp32 [..., d]."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    if fmt == "q4_0":
        return ((c.float() - 8.0).unflatten(-1, (-1, 32)) * scales.float().unsqueeze(-1)).flatten(-2)
    e = c.float().new_tensor(E2M1 + tuple(-v for v in E2M1))[c.long()]
    return ((e.unflatten(-1, (-1, 16)) * scales.view(torch.float8_e4m3fn).float().unsqueeze(-1)) * g).flatten(-2)


def _key_values(gen, shape, d):
    """K and V as projections give them: unit normal, the keys with a few channels of larger size."""
    k = torch.randn(*shape, d, generator=gen, device="cuda")
    v = torch.randn(*shape, d, generator=gen, device="cuda")
    loud = torch.ones(d, device="cuda")
    loud[torch.randperm(d, generator=gen, device="cuda")[:4]] = 4.0
    return k * loud, v


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    b, hkv, d, fmt = case["batch"], case["hkv"], case["d"], case["fmt"]
    order = torch.randperm(b, generator=gen, device="cuda")
    lens = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")[order]
    held = case["hi"] if case["op"] == "attend" else case["past"] + case["l"]
    state = dict(fmt=fmt, op=case["op"], l=case["l"])
    if case["page"]:
        per = -(-held // case["page"])
        size, pages = case["page"], b * per + 3
        table = torch.randperm(pages, generator=gen, device="cuda")[:b * per].to(torch.int32).view(b, per).contiguous()
    else:
        size, pages, table = -(-held // 16) * 16, b, None
    state["table"] = table
    # static global scales, as a calibration gives them: about the largest value met, over 2688
    g = torch.tensor([0.00743, 0.00211], device="cuda")
    state["k_g"], state["v_g"] = (g[:1].clone(), g[1:].clone()) if fmt == "nvfp4" else (None, None)
    k, v = (torch.empty(pages, hkv, size, d // 2, dtype=torch.uint8, device="cuda") for _ in range(2))
    sshape, stype = ((pages, hkv, size, d // 32), torch.float16) if fmt == "q4_0" else ((pages, hkv, size, d // 16), torch.uint8)
    ks, vs = (torch.empty(sshape, dtype=stype, device="cuda") for _ in range(2))
    step = max(1, (1 << 24) // (hkv * size * d))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        xk, xv = _key_values(gen, (n, hkv, size), d)
        k[p:p + n], ks[p:p + n] = _quantise_rows(fmt, xk.bfloat16().float(), state["k_g"])
        v[p:p + n], vs[p:p + n] = _quantise_rows(fmt, xv.bfloat16().float(), state["v_g"])
    state.update(k_codes=k, k_scales=ks, v_codes=v, v_scales=vs)
    if case["op"] == "attend":
        state.update(lens=lens, causal=case["causal"], window=case["window"], hi=case["hi"])
        state["q"] = torch.randn(b, case["l"], case["hq"], d, generator=gen, device="cuda").bfloat16()
    else:
        state.update(counts=lens, start=torch.full((b,), case["past"], dtype=torch.int32, device="cuda"))
        if case["op"] == "write":
            # K and V of the new tokens are column ranges of one buffer, as a fused projection leaves them
            xk, xv = _key_values(gen, (b, case["l"], hkv), d)
            kv = torch.cat((xk.flatten(2), xv.flatten(2)), -1).bfloat16()
            state["k_new"] = kv[..., :hkv * d].unflatten(-1, (hkv, d))
            state["v_new"] = kv[..., hkv * d:].unflatten(-1, (hkv, d))
        else:
            state["f32"] = case["f32"]
    return state


# ------------------------------------------------------------------ the plain form
def _where(state, pos):
    """(page, offset) of positions pos [batch, n]."""
    size = state["k_codes"].shape[2]
    if state["table"] is None:
        return torch.arange(pos.shape[0], device=pos.device)[:, None].expand_as(pos), pos
    return state["table"].long().gather(1, pos // size), pos % size


def _plain_read(state, start, counts, n, dtype):
    """K and V at start + 0..n-1 of each sequence, [batch, n, heads, d]; zero from counts on."""
    i = torch.arange(n, device=counts.device)[None]
    have = i < counts[:, None]
    page, off = _where(state, (start[:, None] + torch.minimum(i, counts[:, None] - 1)).long())
    out = []
    for x in ("k", "v"):
        got = _values(state["fmt"], state[x + "_codes"][page, :, off], state[x + "_scales"][page, :, off], state[x + "_g"])
        out.append(torch.where(have[..., None, None], got, 0.0).to(dtype))
    return out


def _plain_write(state):
    l, counts = state["l"], state["counts"]
    i = torch.minimum(torch.arange(l, device=counts.device)[None], counts[:, None] - 1).long()
    page, off = _where(state, state["start"][:, None].long() + i)
    rows = torch.arange(i.shape[0], device=i.device)[:, None]
    for x in ("k", "v"):
        codes, scales = _quantise_rows(state["fmt"], state[x + "_new"][rows, i].float(), state[x + "_g"])
        state[x + "_codes"][page, :, off] = codes
        state[x + "_scales"][page, :, off] = scales
    return _plain_read(state, state["start"], counts, l, torch.bfloat16)


def _plain_attend(state):
    q, lens = state["q"].float(), state["lens"].long()
    b, l, hq, d = q.shape
    k, v = _plain_read(state, torch.zeros_like(lens), lens, state["hi"], torch.float32)
    hkv = k.shape[2]
    k, v = k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3)
    rows = q.view(b, l, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, l * (hq // hkv), d)
    s = rows @ k.transpose(-1, -2) * (1.0 / math.sqrt(d))
    t = torch.arange(state["hi"], device=q.device)
    p = (lens[:, None] - l + torch.arange(l, device=q.device)).repeat_interleave(hq // hkv, 1)[:, :, None]
    seen = (t < lens[:, None, None]).expand(b, p.shape[1], -1)
    if state["causal"]:
        seen = seen & (t <= p)
    if state["window"]:
        seen = seen & (t > p - state["window"])
    s = s.masked_fill_(~seen[:, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    s = s.sub_(top).exp_()
    total = s.sum(-1, keepdim=True)
    out = (s @ v) / total
    lse = (top + total.log()).squeeze(-1)
    back = lambda x: x.view(b, hkv, l, hq // hkv, -1).permute(0, 2, 1, 3, 4).reshape(b, l, hq, -1)  # noqa: E731
    return back(out).bfloat16(), back(lse).squeeze(-1).contiguous()


# ------------------------------------------------------------------ the framework's operators
def _cache(state):
    """The handle of the cache's buffers, made once a state as a program makes it."""
    if "cache" not in state:
        from bit_weight_quantized_matmul_gb300 import wq
        state["wq"] = wq
        state["cache"] = wq.KVCache(state["fmt"], state["k_codes"], state["k_scales"], state["v_codes"], state["v_scales"],
                                    table=state["table"], k_g=state["k_g"], v_g=state["v_g"])
    return state["wq"], state["cache"]


def run(state):
    if own:
        wq, cache = _cache(state)
        if state["op"] == "write":
            wq.kv_append(cache, state["k_new"], state["v_new"], start=state["start"], counts=state["counts"])
            return wq.kv_read(cache, state["l"], start=state["start"], counts=state["counts"])
        if state["op"] == "read":
            return wq.kv_read(cache, state["l"], start=state["start"], counts=state["counts"], out_f32=state["f32"])
        return wq.attend(cache, state["q"], state["lens"], causal=state["causal"], window=state["window"], return_lse=True)
    if state["op"] == "write":
        return _plain_write(state)
    if state["op"] == "read":
        return _plain_read(state, state["start"], state["counts"], state["l"], torch.float32 if state["f32"] else torch.bfloat16)
    return _plain_attend(state)


# ------------------------------------------------------------------ work, and the definition in 64 bits
def work(case):
    """Each input read once, each output written once; a cached element and its share of a scale are 0.5625 bytes."""
    lens, width = np.array(_lengths(case), np.int64), case["hkv"] * case["d"]
    if case["op"] != "attend":
        new, whole = 2 * width * int(lens.sum()), 2 * width * case["batch"] * case["l"]
        if case["op"] == "write":  # read bf16, write codes, read them back, write bf16
            return {"bytes": new * (2 + 2 * 0.5625) + whole * 2, "flops": 0}
        return {"bytes": new * 0.5625 + whole * (4 if case["f32"] else 2), "flops": 0}
    l, w = case["l"], case["window"]
    p = lens[:, None] - l + np.arange(l)[None]
    hi = np.minimum(p + 1, lens[:, None]) if case["causal"] else np.broadcast_to(lens[:, None], p.shape)
    lo = np.maximum(0, p - w + 1) if w else np.zeros_like(p)
    seen = int(np.maximum(0, hi - lo).sum())
    touched = int((hi.max(1) - lo.min(1)).sum())
    rows = case["batch"] * l * case["hq"]
    return {"bytes": 2 * 0.5625 * width * touched + rows * (4 * case["d"] + 4), "flops": 4 * case["d"] * case["hq"] * seen}


def _decoded64(fmt, codes, scales, g):
    """The definition, in 64 bits: (c - 8) d for q4_0, E2M1(c) s g for NVFP4."""
    low, high = (codes % 16).long(), torch.div(codes, 16, rounding_mode="floor").long()
    c = torch.empty(codes.shape[:-1] + (2 * codes.shape[-1],), dtype=torch.int64, device=codes.device)
    c[..., 0::2], c[..., 1::2] = low, high
    if fmt == "q4_0":
        return (c - 8).double() * scales.double().repeat_interleave(32, -1)
    exp, man, neg = (c // 2) % 4, c % 2, c // 8
    size = torch.where(exp == 0, man.double() / 2, (1 + man.double() / 2) * torch.exp2((exp - 1).double()))
    b = scales.long()
    e, m = (b // 8) % 16, b % 8
    s = torch.where(e == 0, m.double() / 512, (1 + m.double() / 8) * torch.exp2((e - 7).double()))
    return torch.where(neg == 1, -size, size) * s.repeat_interleave(16, -1) * g.double()


def _quantised64(fmt, x, g):
    """What x fp64 [..., d] becomes in the cache, in 64 bits."""
    if fmt == "q4_0":
        blocks = x.reshape(*x.shape[:-1], -1, 32)
        size = blocks.abs()
        first = (size == size.max(-1, keepdim=True).values).to(torch.uint8).argmax(-1, keepdim=True)
        d = (torch.take_along_dim(blocks, first, -1) / -8).half().double()
        q = torch.clip(torch.round(blocks / torch.where(d == 0, 1.0, d)), -8, 7)
        return torch.where(d == 0, 0.0, q * d).reshape(x.shape)
    blocks, gg = x.reshape(*x.shape[:-1], -1, 16), g.double()
    ratio = torch.clip(blocks.abs().max(-1, keepdim=True).values / 6 / gg, max=448.0)
    step = torch.exp2(torch.clip(torch.floor(torch.log2(torch.where(ratio == 0, 1.0, ratio))), min=-6) - 3)
    s = torch.round(ratio / step) * step * gg
    y = blocks / torch.where(s == 0, 1.0, s)
    a = y.abs()
    grid = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).to(a.dtype)
    a = torch.clip(torch.round(a / grid) * grid, max=6.0)
    return torch.where(s == 0, 0.0, torch.sign(y) * a * s).reshape(x.shape)


def _rows64(state, x, b, start, n):
    """n tokens of sequence b from start on, [n, heads, d], in 64 bits."""
    size, pos = state["k_codes"].shape[2], np.arange(start, start + n)
    page = np.full(n, b) if state["table"] is None else state["table"][b].cpu().numpy()[pos // size]
    page, off = torch.as_tensor(page).long().cuda(), torch.as_tensor(pos % size).cuda()
    g = state[x + "_g"]
    return _decoded64(state["fmt"], state[x + "_codes"][page, :, off], state[x + "_scales"][page, :, off], g)


def exact(case, seed):
    if work(case)["flops"] > 2e12:
        return None
    state = prepare(case, seed)
    if case["op"] != "attend":
        out = []
        for x in ("k", "v"):
            got = torch.zeros(case["batch"], case["l"], case["hkv"], case["d"], dtype=torch.float64, device="cuda")
            for b, n in enumerate(state["counts"].tolist()):
                if case["op"] == "write":
                    got[b, :n] = _quantised64(case["fmt"], state[x + "_new"][b, :n].double(), state[x + "_g"])
                else:
                    got[b, :n] = _rows64(state, x, b, case["past"], n)
            out.append(got)
        return out
    l, hq, d, group = case["l"], case["hq"], case["d"], case["hq"] // case["hkv"]
    out = torch.zeros(case["batch"], l, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((case["batch"], l, hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(state["lens"].tolist()):
        k, v = _rows64(state, "k", b, 0, n), _rows64(state, "v", b, 0, n)
        behind = (n - l + torch.arange(l, device="cuda"))[:, None] - torch.arange(n, device="cuda")[None]
        hide = torch.zeros(l, n, dtype=torch.bool, device="cuda")
        if case["causal"]:
            hide |= behind < 0
        if case["window"]:
            hide |= behind >= case["window"]
        for h in range(hq):
            s = (state["q"][b, :, h].double() @ k[:, h // group].T) / math.sqrt(d)
            s[hide] = -math.inf
            lse[b, :, h] = torch.logsumexp(s, -1)
            out[b, :, h] = torch.exp(s - lse[b, :, h, None]) @ v[:, h // group]
    return out, lse
