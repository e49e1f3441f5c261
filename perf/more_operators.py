"""Serving from the 4-bit KV cache, as cases to measure: attention that sees a sliding window and the first tokens,
attention of trees of drafted tokens, the page tables and slot maps of a changing batch, and the writes that go with them.

A case has an ``op``:

* "window": attention of the last tokens of each sequence over a window of the cache and ``sinks`` first tokens;
* "tree": the ancestor bits and depths of trees of drafted tokens (``l`` nodes at most), and their attention;
* "turn": a scheduler's step: pages of finished requests go back to the stack of free pages, every request gets the
  pages of its next tokens, and each of these tokens its slot;
* "pack": K and V of new tokens, laid end to end, go to their slots (and are read back);
* "keep": the K and V of drafted nodes are appended, the rows of the accepted path move up behind the context (and are
  read back).

Ragged lengths run evenly from ``lo`` to ``hi`` over the batch, in an order drawn from the seed.  ``run`` computes in plain
torch operations where ``own`` is false, and calls the library's entry points where it is true.
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
        # the smallest call: one token of one stream (20 heads of 64 = 1280) that has run for long, in a slab
        dict(name="window 1x1 over 2000 w256+4 h20 d64 q4_0", op="window", fmt="q4_0", batch=1, l=1, lo=2000, hi=2000, hq=20,
             hkv=20, d=64, page=0, window=256, sinks=4),
        # a serving batch of 64 endless conversations, grouped heads, small pages
        dict(name="window 64x1 over 1000-32000 w4096+4 h32/8 d128 nvfp4", op="window", fmt="nvfp4", batch=64, l=1, lo=1000,
             hi=32000, hq=32, hkv=8, d=128, page=16, window=4096, sinks=4),
        # a chunk of two long prompts in a model whose layers see a window
        dict(name="window 2x1024 over 16384 w2048+16 h32/8 d128 q4_0", op="window", fmt="q4_0", batch=2, l=1024, lo=9000,
             hi=16384, hq=32, hkv=8, d=128, page=64, window=2048, sinks=16),
        # a small tree behind one audio window's decoded text
        dict(name="tree 1x13 over 447 h20 d64 q4_0", op="tree", fmt="q4_0", batch=1, l=13, nodes=13, lo=447, hi=447, hq=20, hkv=20,
             d=64, page=0, window=0, sinks=0),
        # a tree behind one very long context: a single request has to fill the machine
        dict(name="tree 1x26 over 60001 h32/8 d128 q4_0", op="tree", fmt="q4_0", batch=1, l=26, nodes=26, lo=60001, hi=60001,
             hq=32, hkv=8, d=128, page=64, window=0, sinks=0),
        # a serving batch whose requests draft trees of unequal sizes
        dict(name="tree 32x20-64 over 2000-16000 h32/8 d128 nvfp4", op="tree", fmt="nvfp4", batch=32, l=64, nodes=20, lo=2000,
             hi=16000, hq=32, hkv=8, d=128, page=32, window=0, sinks=0),
        # one decoding step of a batch: most requests get one more token, some end, a few begin
        dict(name="turn 48 decode page 64", op="turn", batch=48, lo=100, hi=8000, ends=3, begins=2, prompt=300, page=64, tight=False),
        # many prompts at once, and a pool that does not hold the last of them
        dict(name="turn 256 prompts page 16", op="turn", batch=256, lo=300, hi=5000, ends=40, begins=200, prompt=8000, page=16,
             tight=True),
        # the step's K and V of 48 requests, one token each
        dict(name="pack 48x1 h8 d128 nvfp4", op="pack", fmt="nvfp4", batch=48, lo=1, hi=1, past=900, hkv=8, d=128, page=64),
        # prompts of unequal length, laid end to end as a fused projection leaves them
        dict(name="pack 24x100-1500 h20 d64 q4_0", op="pack", fmt="q4_0", batch=24, lo=100, hi=1500, past=0, hkv=20, d=64, page=32),
        # the accepted path of one small tree
        dict(name="keep 1x13 h20 d64 q4_0", op="keep", fmt="q4_0", batch=1, l=13, past=434, hkv=20, d=64, page=0),
        # the accepted paths of a batch of large trees
        dict(name="keep 64x64 h8 d128 nvfp4", op="keep", fmt="nvfp4", batch=64, l=64, past=3001, hkv=8, d=128, page=16),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    fmt = rng.choice(["q4_0", "nvfp4"])
    page = rng.choice([0, 16, 32, 48, 64, 128])
    op = rng.choice(["window", "window", "tree", "tree", "turn", "pack", "keep"])
    hq, hkv, d = rng.choice([(20, 20, 64), (6, 6, 64), (32, 8, 128), (32, 4, 128), (16, 16, 128), (8, 1, 64), (40, 8, 128)])
    if op == "turn":
        batch = _log(rng, 1, 256)
        hi = _log(rng, 10, 8000)
        rest = rng.randint(0, batch)
        ends = rng.randint(0, rest)
        return dict(op=op, batch=batch, lo=rng.randint(1, hi), hi=hi, ends=ends, begins=rest - ends,
                    prompt=_log(rng, 1, 8000), page=page or 64, tight=rng.random() < 0.3)
    if op == "pack":
        batch = _log(rng, 1, 64)
        hi = _log(rng, 1, max(1, min(4000, 24 * 1500 * 20 * 64 // (batch * hkv * d))))
        return dict(op=op, fmt=fmt, batch=batch, lo=rng.randint(max(1, hi // 10), hi), hi=hi, past=rng.choice([0, rng.randint(1, 1000)]),
                    hkv=hkv, d=d, page=page)
    if op == "keep":
        return dict(op=op, fmt=fmt, batch=_log(rng, 1, 64), l=_log(rng, 1, 64), past=_log(rng, 1, 4000), hkv=hkv, d=d, page=page)
    if op == "tree":
        batch, l = _log(rng, 1, 32), _log(rng, 2, 64)
        most = 32 * 64 * 9000 * 32 * 128 // (batch * l * hq * d)
        hi = max(l + 1, _log(rng, 40, max(41, min(60000, most, 32 * 9000 * 8 * 128 // (batch * hkv * d)))))
        c = dict(op=op, fmt=fmt, batch=batch, l=l, nodes=rng.randint(max(1, l // 3), l), lo=rng.randint(max(l, hi // 4), hi), hi=hi)
        c.update(window=rng.choice([0, 0, rng.randint(16, 4096)]), sinks=0)
        c["sinks"] = rng.choice([0, rng.randint(1, 40)]) if c["window"] else 0
    else:
        kind = rng.choice(["token", "token", "some", "many"])
        batch = _log(rng, 1, 64 if kind != "many" else 4)
        l = 1 if kind == "token" else rng.randint(2, 9) if kind == "some" else _log(rng, 17, 1024)
        most = 64 * 16000 * 8 * 128 // (batch * hkv * d)
        hi = max(l, _log(rng, 40, max(41, min(32000, most))))
        c = dict(op=op, fmt=fmt, batch=batch, l=l, lo=rng.randint(max(l, hi // 4), hi), hi=hi,
                 window=_log(rng, 16, 4096 if kind != "many" else 2048), sinks=rng.choice([1, 4, 16, rng.randint(1, 200)]))
    c.update(hq=hq, hkv=hkv, d=d, page=page)
    return c


# ------------------------------------------------------------------ inputs
def _even(lo, hi, n):
    """n whole numbers evenly from hi down to lo."""
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)][::-1]


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


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _trees(rng, batch, l):
    """Parents [batch, l] of trees that grow at random: a node hangs below one of the last few, or is one of the first ones."""
    out = np.full((batch, l), -1, np.int32)
    for b in range(batch):
        reach = int(rng.integers(1, 12))
        for i in range(1, l):
            out[b, i] = rng.integers(max(0, i - reach), i) if rng.random() > 0.1 else -1
    return out


def _prepare_turn(case, seed):
    """Who holds what: the first rows' requests end (or lose some last tokens), then come those that begin, then those that go on."""
    rng = np.random.default_rng(seed)
    batch, size, ends, begins = case["batch"], case["page"], case["ends"], case["begins"]
    kind = np.array([0] * ends + [1] * begins + [2] * (batch - ends - begins))[rng.permutation(batch)]
    lens, counts = np.zeros(batch, np.int64), np.where(kind == 2, 1, 0)
    lens[kind != 1] = rng.permutation(_even(case["lo"], case["hi"], batch - begins))
    counts[kind == 1] = rng.permutation(_even(max(1, case["prompt"] // 3), case["prompt"], begins))
    keep = np.where(kind == 0, np.where(rng.random(batch) < 0.8, 0, lens * rng.random(batch)).astype(np.int64), lens)
    held = -(-lens // size)
    need = -(-(keep + counts) // size) - -(-keep // size)
    back = int((held - -(-keep // size)).sum())
    pages = int(held.sum() + (-(-counts // size)).sum()) + 7      # some of them with requests of another batch
    free = min(pages - int(held.sum()), max(0, int(need.sum()) - back + (-max(1, int(need.sum()) // 20) if case["tight"] else 7)))
    order = rng.permutation(pages).astype(np.int32)
    ld = -(-max(case["hi"] + 1, case["prompt"]) // size)
    table = np.full((batch, ld), -1, np.int32)
    at = free
    for b in range(batch):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    stack = np.full(pages, -1, np.int32)
    stack[:free] = order[:free]
    return dict(op="turn", lens=_ints(lens), keep=_ints(keep), counts=_ints(counts), table=_ints(table), free=_ints(stack),
                top=_ints([free]), between=_ints([0]), after=_ints([0]), size=size, pages=pages,
                tokens=int(counts.sum()) + 5)     # a program knows an upper bound of the step's tokens


def prepare(case, seed):
    if case["op"] == "turn":
        return _prepare_turn(case, seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = np.random.default_rng(seed)
    b, hkv, d, fmt, op = case["batch"], case["hkv"], case["d"], case["fmt"], case["op"]
    held = case["hi"] if op in ("window", "tree") else case["past"] + (case["hi"] if op == "pack" else case["l"])
    state = dict(fmt=fmt, op=op)
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
    if op in ("window", "tree"):
        state.update(lens=_ints(rng.permutation(_even(case["lo"], case["hi"], b))), l=case["l"], hi=case["hi"], window=case["window"],
                     sinks=case["sinks"], parents=None, counts=None)
        state["q"] = torch.randn(b, case["l"], case["hq"], d, generator=gen, device="cuda").bfloat16()
        if op == "tree":
            state.update(parents=_ints(_trees(rng, b, case["l"])), counts=_ints(rng.permutation(_even(case["nodes"], case["l"], b))))
        return state
    state["start"] = _ints([case["past"]] * b)
    if op == "pack":
        lens = rng.permutation(_even(case["lo"], case["hi"], b))
        where = np.concatenate([case["past"] + np.arange(n) for n in lens])
        owner = np.repeat(np.arange(b), lens)
        page = owner if table is None else table.cpu().numpy()[owner, where // size]
        state.update(l=case["hi"], counts=_ints(lens), slots=torch.as_tensor(page.astype(np.int64) * size + where % size).cuda())
        shape = (len(where), hkv)
    else:
        paths, counts = np.zeros((b, case["l"]), np.int32), np.zeros(b, np.int32)
        for i, parents in enumerate(_trees(rng, b, case["l"])):
            node, path = int(rng.integers(0, case["l"])), []
            while node >= 0:
                path.append(node)
                node = int(parents[node])
            counts[i] = len(path)
            paths[i, :len(path)] = path[::-1]
        state.update(l=case["l"], path=_ints(paths), counts=_ints(counts))
        shape = (b, case["l"], hkv)
    # K and V of the new tokens are column ranges of one buffer, as a fused projection leaves them
    xk, xv = _key_values(gen, shape, d)
    kv = torch.cat((xk.flatten(-2), xv.flatten(-2)), -1).bfloat16()
    state["k_new"] = kv[..., :hkv * d].unflatten(-1, (hkv, d))
    state["v_new"] = kv[..., hkv * d:].unflatten(-1, (hkv, d))
    return state


# ------------------------------------------------------------------ the plain form
def _where(state, pos):
    """(page, offset) of positions pos [batch, n]."""
    size = state["k_codes"].shape[2]
    if state["table"] is None:
        return torch.arange(pos.shape[0], device=pos.device)[:, None].expand_as(pos), pos
    return state["table"].long().gather(1, pos // size), pos % size


def _at(state, pos):
    """K and V at positions pos [batch, n], fp32 [batch, n, heads, d]."""
    page, off = _where(state, pos)
    return [_values(state["fmt"], state[x + "_codes"][page, :, off], state[x + "_scales"][page, :, off], state[x + "_g"]) for x in "kv"]


def _plain_read(state, start, counts, n):
    """K and V at start + 0..n-1 of each sequence, bf16 [batch, n, heads, d]; zero from counts on."""
    i = torch.arange(n, device=counts.device)[None]
    have = (i < counts[:, None])[..., None, None]
    got = _at(state, (start[:, None] + torch.minimum(i, counts[:, None] - 1).clamp(min=0)).long())
    return [torch.where(have, x, 0.0).bfloat16() for x in got]


def _plain_pack(state):
    size = state["k_codes"].shape[2]
    page, off = state["slots"] // size, state["slots"] % size
    for x in "kv":
        codes, scales = _quantise_rows(state["fmt"], state[x + "_new"].float(), state[x + "_g"])
        state[x + "_codes"][page, :, off] = codes
        state[x + "_scales"][page, :, off] = scales
    return _plain_read(state, state["start"], state["counts"], state["l"])


def _plain_keep(state):
    l, start, counts = state["l"], state["start"].long(), state["counts"]
    i = torch.arange(l, device=counts.device)
    page, off = _where(state, start[:, None] + i)
    moves = i < counts[:, None]
    node = torch.where(moves, state["path"].long(), i)
    for x in "kv":
        codes, scales = _quantise_rows(state["fmt"], state[x + "_new"].float(), state[x + "_g"])
        at = node[..., None, None].expand_as(codes)
        state[x + "_codes"][page, :, off] = codes.gather(1, at)
        state[x + "_scales"][page, :, off] = scales.gather(1, node[..., None, None].expand_as(scales))
    return _plain_read(state, state["start"], torch.full_like(counts, l), l)


def _plain_tree(parents, counts, window):
    """Ancestors-or-self [batch, l, l], their bits in 32-bit words, and depths; nothing for nodes from counts on."""
    b, l = parents.shape
    i = torch.arange(l, device=parents.device)
    there = i < counts[:, None]
    reach = ((parents[:, :, None] == i) | (i[:, None] == i)) & there[:, :, None]
    for _ in range(max(1, (l - 1).bit_length())):
        reach = (reach.float() @ reach.float()) > 0.5
    depth = torch.where(there, reach.sum(-1) - 1, 0)
    if window:
        reach = reach & (depth[:, :, None] - depth[:, None, :] < window)
    words = -(-l // 32)
    bits = torch.nn.functional.pad(reach.long(), (0, words * 32 - l)).unflatten(-1, (words, 32))
    word = (bits << torch.arange(32, device=parents.device)).sum(-1)
    return reach, torch.where(word >= 1 << 31, word - (1 << 32), word).int(), depth.int()


def _plain_attend(state):
    q, lens, window, sinks = state["q"].float(), state["lens"].long(), state["window"], state["sinks"]
    b, l, hq, d = q.shape
    i = torch.arange(l, device=q.device)
    n = torch.full_like(lens, l) if state["counts"] is None else state["counts"].long()
    base = lens - n
    tree = None
    if state["parents"] is not None:
        tree, words, depth = _plain_tree(state["parents"], n, window)
    p = base[:, None] + (i if tree is None else depth)
    # the first tokens, and those from the first that some row's window holds
    wide = min(state["hi"], window + l) if window else state["hi"]
    first = (lens - wide).clamp(min=0)
    t = first[:, None] + torch.arange(wide, device=q.device)
    if window and sinks:
        few = torch.arange(min(sinks, state["hi"]), device=q.device).expand(b, -1)
        t = torch.cat((torch.where(few < first[:, None], few, -1), t), 1)
    k, v = _at(state, t.clamp(min=0).minimum(lens[:, None] - 1))
    hkv = k.shape[2]
    k, v = k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3)
    rows = q.view(b, l, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, l * (hq // hkv), d)
    s = rows @ k.transpose(-1, -2) * (1.0 / math.sqrt(d))
    t = t[:, None, :]
    seen = (t >= 0) & (t < lens[:, None, None]) & (i[:, None] < n[:, None, None])
    near = (t > p[:, :, None] - window) | (t < sinks) if window else torch.ones_like(seen)
    if tree is None:
        seen = seen & near & (t <= p[:, :, None])
    else:
        j = t - base[:, None, None]
        seen = seen & torch.where(j < 0, near, tree.gather(2, j.clamp(0, l - 1).expand(b, l, -1)))
    s = s.masked_fill_(~seen.repeat_interleave(hq // hkv, 1)[:, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    s = s.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = s.sum(-1, keepdim=True)
    out = torch.where(total > 0, (s @ v) / total, 0.0)
    lse = (top + total.log()).squeeze(-1)
    back = lambda x: x.view(b, hkv, l, hq // hkv, -1).permute(0, 2, 1, 3, 4).reshape(b, l, hq, -1)  # noqa: E731
    res = back(out).bfloat16(), back(lse).squeeze(-1).contiguous()
    return res if tree is None else res + (words, depth)


def _spread(counts, total):
    """Owner and index within it of `total` things, counts[b] of each owner one after the other; and which are there."""
    ends = counts.cumsum(0)
    k = torch.arange(total, device=counts.device)
    owner = torch.searchsorted(ends, k, right=True)
    there = owner < counts.numel()
    owner = owner.clamp(max=counts.numel() - 1)
    return owner, k - (ends - counts)[owner], there


def _put(to, at, values):
    """to[at] = values where at is not -1."""
    wide = torch.cat((to, to.new_zeros(1)))
    wide[at] = values
    to.copy_(wide[:-1])


def _plain_turn(state):
    size, table, free = state["size"], state["table"], state["free"]
    lens, keep, counts, top = state["lens"].long(), state["keep"].long(), state["counts"].long(), state["top"].long()
    up = lambda x: (x + size - 1) // size  # noqa: E731
    # pages behind the kept tokens go on the stack
    gone = up(lens) - up(keep)
    owner, j, there = _spread(gone, state["pages"])
    page = table[owner, torch.where(there, up(keep)[owner] + j, 0)]
    _put(free, torch.where(there, top + torch.arange(state["pages"], device=top.device), -1), page)
    between = top + gone.sum()
    # and come off it, for the requests in turn while they last
    need = up(keep + counts) - up(keep)
    ends = need.cumsum(0)
    ok = (need == 0) | (ends <= between)
    taken = torch.where(ok & (need > 0), ends, 0).amax()
    owner, j, there = _spread(need, table.numel())
    there = there & ok[owner]
    at = torch.where(there, between - 1 - (ends - need)[owner] - j, 0)
    _put(table.view(-1), torch.where(there, owner * table.shape[1] + up(keep)[owner] + j, -1), free[at])
    # a slot for each token
    owner, i, there = _spread(counts, state["tokens"])
    pos = torch.where(there, keep[owner] + i, 0)
    good = there & ok[owner]
    page = table[owner, torch.where(good, pos // size, 0)].long()
    slots = torch.where(good, page * size + pos % size, -1)
    starts = torch.cat((torch.zeros_like(top), counts.cumsum(0)))
    return slots, pos.int(), starts.int(), torch.where(ok, counts, 0).int(), (between - taken).int(), table, free


# ------------------------------------------------------------------ the framework's operators
def _cache(state):
    """The handle of the cache's buffers, made once a state as a program makes it."""
    if "cache" not in state:
        from bit_weight_quantized_matmul_gb300 import wq
        state["wq"] = wq
        if state["op"] == "turn":      # tables do not depend on what the pages hold
            state["cache"] = wq.kv_alloc("q4_0", state["pages"], state["size"], 1, 64, state["table"])
        else:
            state["cache"] = wq.KVCache(state["fmt"], state["k_codes"], state["k_scales"], state["v_codes"], state["v_scales"],
                                        table=state["table"], k_g=state["k_g"], v_g=state["v_g"])
    return state["wq"], state["cache"]


def run(state):
    op = state["op"]
    if not own:
        return {"turn": _plain_turn, "pack": _plain_pack, "keep": _plain_keep}.get(op, _plain_attend)(state)
    wq, cache = _cache(state)
    if op == "window":
        return wq.attend(cache, state["q"], state["lens"], window=state["window"], sinks=state["sinks"], return_lse=True)
    if op == "tree":
        mask, depth = tree = wq.tree_mask(state["parents"], state["counts"], window=state["window"])
        return wq.attend(cache, state["q"], state["lens"], counts=state["counts"], window=state["window"], sinks=state["sinks"],
                         tree=tree, return_lse=True) + (mask, depth)
    if op == "turn":
        wq.kv_release(cache, state["free"], state["top"], state["lens"], state["keep"], top_out=state["between"])
        got = wq.kv_reserve(cache, state["free"], state["between"], state["keep"], state["counts"], state["tokens"],
                            top_out=state["after"])
        return got + (state["after"], state["table"], state["free"])
    if op == "pack":
        wq.kv_append_slots(cache, state["k_new"], state["v_new"], state["slots"])
        return wq.kv_read(cache, state["l"], start=state["start"], counts=state["counts"])
    wq.kv_append(cache, state["k_new"], state["v_new"], start=state["start"])
    wq.kv_keep(cache, state["start"], state["path"], state["counts"])
    return wq.kv_read(cache, state["l"], start=state["start"])


# ------------------------------------------------------------------ work, and the definition in 64 bits
def work(case):
    """Each input read once, each output written once; a cached element and its share of a scale are 0.5625 bytes."""
    op, batch = case["op"], case["batch"]
    if op == "turn":
        size = case["page"]
        prompts = _even(max(1, case["prompt"] // 3), case["prompt"], case["begins"])
        tokens = sum(prompts) + batch - case["ends"] - case["begins"]
        back = case["ends"] * (case["lo"] + case["hi"]) // 2 // size
        return {"bytes": 16 * batch + 12 * tokens + 8 * (tokens // size + back), "flops": 0}
    width = case["hkv"] * case["d"]
    if op == "pack":     # read bf16, write codes, read them back, write bf16
        lens = sum(_even(case["lo"], case["hi"], batch))
        return {"bytes": 2 * width * (lens * (2 + 2 * 0.5625) + 2 * batch * case["hi"]) + 8 * lens, "flops": 0}
    if op == "keep":
        return {"bytes": 2 * width * batch * case["l"] * (2 + 2 * 0.5625 + 2), "flops": 0}
    l, w, sinks = case["l"], case["window"], case["sinks"]
    lens = np.array(_even(case["lo"], case["hi"], batch), np.int64)
    n = np.array(_even(case["nodes"], l, batch) if op == "tree" else [l] * batch, np.int64)
    base = lens - n
    seen = touched = 0
    for first, m in zip(base.tolist(), n.tolist()):
        p = first + np.arange(m)
        if op == "tree":     # a tree's depth is about twice the logarithm of its size
            p = first + np.minimum(np.arange(m), 2 * int(math.log2(m + 1)))
        lo = np.maximum(0, p - w + 1) if w else np.zeros_like(p)
        seen += int((p + 1 - lo + np.minimum(lo, sinks)).sum())
        touched += int(first + m - lo.min() + min(lo.min(), sinks))
    rows = batch * l * case["hq"]
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


def _rows64(state, x, b, pos):
    """Positions pos of sequence b, [n, heads, d], in 64 bits."""
    size = state["k_codes"].shape[2]
    page = np.full(len(pos), b) if state["table"] is None else state["table"][b].cpu().numpy()[pos // size]
    page, off = torch.as_tensor(page).long().cuda(), torch.as_tensor(pos % size).cuda()
    return _decoded64(state["fmt"], state[x + "_codes"][page, :, off], state[x + "_scales"][page, :, off], state[x + "_g"])


def _exact_turn(state):
    size, stack = state["size"], state["free"].tolist()
    table, top = state["table"].tolist(), int(state["top"])
    lens, keep, counts = (state[x].tolist() for x in ("lens", "keep", "counts"))
    for b, held in enumerate(lens):
        for page in range(math.ceil(keep[b] / size), math.ceil(held / size)):
            stack[top] = table[b][page]
            top += 1
    slots, pos, starts, granted, empty = [], [], [0], [], False
    for b, held in enumerate(keep):
        new = range(math.ceil(held / size), math.ceil((held + counts[b]) / size))
        empty = empty or len(new) > top
        ok = len(new) == 0 or not empty
        for page in new if ok else ():
            top -= 1
            table[b][page] = stack[top]
        slots += [table[b][t // size] * size + t % size if ok else -1 for t in range(held, held + counts[b])]
        pos += range(held, held + counts[b])
        starts.append(len(pos))
        granted.append(counts[b] if ok else 0)
    more = state["tokens"] - len(pos)
    return (torch.tensor(slots + [-1] * more), _ints(pos + [0] * more), _ints(starts), _ints(granted), _ints([top]), _ints(table),
            _ints(stack))


def _exact_tree(parents, n, l, window):
    """Ancestors-or-self of each node, the words of their bits, and depths, one node after the other."""
    seen, words, depth = np.zeros((l, l), bool), np.zeros((l, -(-l // 32)), np.uint32), np.zeros(l, np.int32)
    for i in range(n):
        node, up = i, 0
        while node >= 0:
            if not window or up < window:
                seen[i, node] = True
                words[i, node // 32] |= np.uint32(1 << (node % 32))
            node, up = int(parents[node]), up + 1
        depth[i] = up - 1
    return seen, words.view(np.int32), depth


def exact(case, seed):
    op = case["op"]
    if op in ("window", "tree") and work(case)["flops"] > 2e12:
        return None
    state = prepare(case, seed)
    if op == "turn":
        return _exact_turn(state)
    batch, l = case["batch"], state["l"]
    if op in ("pack", "keep"):
        out = []
        for x in "kv":
            got = torch.zeros(batch, l, case["hkv"], case["d"], dtype=torch.float64, device="cuda")
            at = 0
            for b, n in enumerate(state["counts"].tolist()):
                if op == "pack":
                    got[b, :n] = _quantised64(case["fmt"], state[x + "_new"][at:at + n].double(), state[x + "_g"])
                    at += n
                else:
                    new = _quantised64(case["fmt"], state[x + "_new"][b].double(), state[x + "_g"])
                    got[b] = new
                    got[b, :n] = new[state["path"][b, :n].long()]
            out.append(got)
        return out
    hq, group = case["hq"], case["hq"] // case["hkv"]
    out = torch.zeros(batch, l, hq, case["d"], dtype=torch.float64, device="cuda")
    lse = torch.full((batch, l, hq), -math.inf, dtype=torch.float64, device="cuda")
    masks, depths = [], []
    for b, length in enumerate(state["lens"].tolist()):
        n = int(state["counts"][b]) if op == "tree" else l
        base = length - n
        t, p = np.arange(length), base + np.arange(n)
        if op == "tree":
            kin, words, depth = _exact_tree(state["parents"][b].tolist(), n, l, state["window"])
            masks.append(words)
            depths.append(depth)
            p = base + depth[:n]
        see = np.ones((n, length), bool)
        if case["window"]:
            see &= (p[:, None] - t < case["window"]) | (t < case["sinks"])
        if op == "tree":
            see[:, base:] = kin[:n, :n]
        else:
            see &= t <= p[:, None]
        pos = np.flatnonzero(see.any(0))
        hide = torch.as_tensor(~see[:, pos]).cuda()
        k, v = _rows64(state, "k", b, pos), _rows64(state, "v", b, pos)
        for h in range(hq):
            s = (state["q"][b, :n, h].double() @ k[:, h // group].T) / math.sqrt(case["d"])
            s[hide] = -math.inf
            lse[b, :n, h] = torch.logsumexp(s, -1)
            out[b, :n, h] = torch.exp(s - lse[b, :n, h, None]) @ v[:, h // group]
    if op == "window":
        return out, lse
    return out, lse, torch.as_tensor(np.stack(masks)), torch.as_tensor(np.stack(depths))
