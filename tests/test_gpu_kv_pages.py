"""Pages and slots of a changing batch, packed appends, trees' masks and kept paths: whole numbers and bits, all exact."""
import numpy as np
import pytest
import torch

from oracle import kv as OK
from tests.gpu_common import need_gpu, wq
from tests.test_gpu_kv_cache import Case, bf16, ints, raw
from tests.test_gpu_kv_select import cuda, random_trees

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ reserve and release
def reserve(size, pages, table, stack, top, lens, counts, tokens):
    """The definition, one sequence after the other; changes `table`, returns (slots, positions, starts, granted, top)."""
    cap = table.shape[1] * size
    slots, positions, starts, granted, short = [], [], [0], [], False
    for b in range(len(lens)):
        n, held = max(int(counts[b]), 0), max(int(lens[b]), 0)
        new = range(-(-held // size), -(-(held + n) // size))
        ok = held + n <= cap
        if ok and len(new):
            short = short or len(new) > top
            ok = not short
        if ok:
            for p in new:
                top -= 1
                table[b, p] = stack[top]
        granted.append(n if ok else 0)
        for t in range(held, held + n):
            page = int(table[b, t // size]) if ok else -1
            slots.append(page * size + t % size if 0 <= page < pages else -1)
            positions.append(min(t, 2 ** 31 - 1))
        starts.append(len(slots))
    more = max(0, tokens - len(slots))
    return (slots + [-1] * more)[:tokens], (positions + [0] * more)[:tokens], starts, granted, top


def small_cache(size, pages, table):
    return wq().kv_alloc("q4_0", pages, size, 1, 64, table)


def check_reserve(seed, batch, ld, size, lens, counts, short=0, extra=5, in_place=True):
    m, rng = wq(), np.random.default_rng(seed)
    lens, counts = np.asarray(lens), np.asarray(counts)
    held = -(-np.maximum(lens, 0) // size)
    pages = int(np.minimum(held, ld).sum() + (-(-np.maximum(counts, 0) // size)).clip(max=ld).sum()) + batch + 2
    order = rng.permutation(pages)
    table = np.full((batch, ld), -7, np.int32)
    at = 0
    for b in range(batch):
        n = min(int(held[b]), ld)
        table[b, :n] = order[at:at + n]
        at += n
    need = int(np.where(np.maximum(lens, 0) + np.maximum(counts, 0) <= ld * size,
                        -(-(np.maximum(lens, 0) + np.maximum(counts, 0)) // size) - held, 0).sum())
    free = max(0, min(pages - at, need - short))
    stack = np.full(pages, -9, np.int32)
    stack[:free] = order[at:at + free]
    tokens = int(np.maximum(counts, 0).sum()) + extra
    want_table = table.copy()
    want = reserve(size, pages, want_table, stack, free, lens, counts, tokens)
    dev_table, top, left = cuda(table), ints([free]), ints([-1])
    cache = small_cache(size, pages, dev_table)
    got = m.kv_reserve(cache, cuda(stack), top, ints(list(lens)), ints(list(counts)), tokens, top_out=top if in_place else left)
    for g, w, dt in zip(got, want, (torch.int64, torch.int32, torch.int32, torch.int32)):
        assert g.dtype == dt and g.tolist() == w
    assert int(top if in_place else left) == want[4] and int(top) == (want[4] if in_place else free)
    assert np.array_equal(dev_table.cpu().numpy(), want_table)
    assert m.last_device_status() == 0
    return want


@pytest.mark.parametrize("size", [16, 48, 64])
@pytest.mark.parametrize("in_place", [True, False])
def test_reserve_small_batches(size, in_place):
    need_gpu()
    check_reserve(1, 1, 3, size, [0], [1], in_place=in_place)
    check_reserve(2, 1, 3, size, [size], [0], in_place=in_place)
    check_reserve(3, 5, 9, size, [0, 1, size - 1, size, 3 * size + 1], [1, 1, 1, 1, 5 * size], in_place=in_place)
    check_reserve(4, 4, 9, size, [-5, 7, 0, 2], [3, -1, 0, 4 * size + 1], in_place=in_place)


@pytest.mark.parametrize("seed", range(6))
def test_reserve_many_sequences(seed):
    need_gpu()
    rng = np.random.default_rng(100 + seed)
    batch, size = [33, 257, 1024, 1025, 3000, 130][seed], [16, 32, 48, 16, 16, 256][seed]
    lens, counts = rng.integers(0, 40 * size, batch), rng.integers(0, 3, batch)
    counts[rng.permutation(batch)[:batch // 3]] = rng.integers(0, 9 * size, batch // 3)
    check_reserve(seed, batch, 50, size, lens, counts)
    want = check_reserve(seed, batch, 50, size, lens, counts, short=batch // 4 + 1, in_place=seed % 2 == 0)
    assert 0 in [g for g, n in zip(want[3], counts) if n > 0]
    check_reserve(seed, batch, 50, size, lens, counts, extra=0)


def test_reserve_when_the_stack_is_empty_or_a_row_is_full():
    need_gpu()
    want = check_reserve(7, 4, 3, 16, [0, 5, 16, 30], [1, 4, 1, 2], short=9)          # no page at all: 1 and 3 need none
    assert want[3] == [0, 4, 0, 2]
    want = check_reserve(8, 4, 3, 16, [0, 40, 48, 47], [49, 9, 1, 1])                 # past the capacity of 48
    assert want[3] == [0, 0, 0, 1]
    check_reserve(9, 3, 300, 16, [0, 0, 0], [4800, 4801, 4799])


def test_reserve_with_less_room_than_tokens_and_with_bad_pages():
    need_gpu()
    m = wq()
    table = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    cache, stack, top = small_cache(16, 8, table), ints([3, 900, 5]), ints([3])
    guard = [torch.full((12,), 77, dtype=dt, device="cuda") for dt in (torch.int64, torch.int32)]
    got = m.kv_reserve(cache, stack, top, ints([0, 0]), ints([20, 4]), 10, out=(guard[0][:10], guard[1][:10], *m.kv_reserve(
        small_cache(16, 8, table.clone()), stack, top.clone(), ints([0, 0]), ints([0, 0]), 1)[2:]))
    assert m.last_device_status() == m.WQ_ERR_ARG                    # page 900, and more tokens than slots
    assert got[0].tolist() == [5 * 16 + i for i in range(10)] and got[1].tolist() == list(range(10))
    assert got[2].tolist() == [0, 20, 24] and got[3].tolist() == [20, 4] and int(top) == 0
    assert guard[0][10:].tolist() == [77, 77] and guard[1][10:].tolist() == [77, 77]
    assert table.tolist() == [[5, 900, -1, -1], [3, -1, -1, -1]]
    got = m.kv_reserve(cache, stack, ints([0]), ints([20, 4]), ints([3, 1]), 4)      # tokens on the bad page
    assert m.last_device_status() == m.WQ_ERR_ARG and got[0].tolist() == [-1, -1, -1, 3 * 16 + 4]
    got = m.kv_reserve(cache, stack, ints([-4]), ints([4, 4]), ints([2 ** 31 - 1, 2 ** 31 - 1]), 7)   # counts of old buffers
    assert got[0].tolist() == [-1] * 7 and got[3].tolist() == [0, 0] and got[2].tolist() == [0, 2 ** 31 - 1, 2 ** 31 - 1]
    assert m.last_device_status() == m.WQ_ERR_ARG


@pytest.mark.parametrize("batch", [2, 1500])
def test_a_map_of_no_tokens_is_too_short(batch):
    """Slots or positions are asked for, and there is no room for any: reported as any other length that does not do."""
    need_gpu()
    m, table = wq(), torch.full((batch, 3), -1, dtype=torch.int32, device="cuda")
    cache, stack, top, left = small_cache(16, 9, table), ints([4, 7, 5]), ints([3]), ints([-1])
    lens, counts, guard = ints([0] * batch), ints([5] + [0] * (batch - 1)), torch.full((4,), 77, dtype=torch.int64, device="cuda")
    for slots, positions, status in ((guard, None, m.WQ_ERR_ARG), (None, guard, m.WQ_ERR_ARG), (None, None, 0)):
        at = [None if x is None else x.data_ptr() for x in (slots, positions)]
        rc = m.lib.wq_kv_reserve(cache.ref, stack.data_ptr(), 3, top.data_ptr(), left.data_ptr(), batch, lens.data_ptr(), counts.data_ptr(),
                                 None, 0, *at, None, torch.cuda.current_stream().cuda_stream)
        assert rc == 0 and m.last_device_status() == status and int(left) == 2 and int(table[0, 0]) == 5
    counts[0] = 0
    rc = m.lib.wq_kv_reserve(cache.ref, stack.data_ptr(), 3, top.data_ptr(), left.data_ptr(), batch, lens.data_ptr(), counts.data_ptr(), None,
                             0, guard.data_ptr(), None, None, torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and m.last_device_status() == 0 and int(left) == 3 and guard.tolist() == [77] * 4


@pytest.mark.parametrize("batch,ld,size", [(1, 4, 16), (40, 7, 64), (300, 90, 16), (2500, 5, 48)])
def test_release(batch, ld, size):
    need_gpu()
    m, rng = wq(), np.random.default_rng(batch)
    lens = rng.integers(-3, ld * size + 40, batch)
    keep = np.where(rng.random(batch) < 0.5, lens, rng.integers(-5, ld * size + 5, batch))
    table = rng.permutation(batch * ld).astype(np.int32).reshape(batch, ld)
    for keeps in (keep, None):
        want = []
        for b in range(batch):
            held = -(-min(max(int(lens[b]), 0), ld * size) // size)
            stay = 0 if keeps is None else -(-max(int(keep[b]), 0) // size)
            want += table[b, stay:held].tolist()
        stack, top, out = np.full(batch * ld + 3, -9, np.int32), ints([2]), ints([-1])
        cache, dev = small_cache(size, batch * ld, cuda(table)), cuda(stack)
        m.kv_release(cache, dev, top, ints(list(lens)), None if keeps is None else ints(list(keeps)), top_out=out)
        assert int(out) == 2 + len(want) and int(top) == 2
        assert dev.tolist() == [-9, -9] + want + [-9] * (batch * ld + 1 - len(want))
        m.kv_release(cache, dev, top, ints(list(lens)), None if keeps is None else ints(list(keeps)))
        assert int(top) == 2 + len(want) and np.array_equal(cache.tensors[4].cpu().numpy(), table)
        assert m.last_device_status() == 0
        if len(want) > 3:                                             # no room for the last three
            small = torch.full((2 + len(want) - 3,), -9, dtype=torch.int32, device="cuda")
            m.kv_release(cache, small, ints([2]), ints(list(lens)), None if keeps is None else ints(list(keeps)), top_out=out)
            assert int(out) == small.numel() and small.tolist() == [-9, -9] + want[:-3] and m.last_device_status() == m.WQ_ERR_ARG


@pytest.mark.parametrize("bad", [-1, 9, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("batch", [2, 1500])
def test_release_of_what_is_no_page_is_reported(bad, batch):
    """lens past what was granted: the entries behind a sequence's pages go back, and the call that takes them says so."""
    need_gpu()
    m, table = wq(), np.full((batch, 3), bad, np.int32)
    table[0], table[-1] = [4, 2, bad], [7, bad, bad]
    lens = np.zeros(batch, np.int64)
    lens[0], lens[-1] = 32, 16
    cache, stack, top = small_cache(16, 9, cuda(table)), torch.full((9,), -9, dtype=torch.int32, device="cuda"), ints([0])
    m.kv_release(cache, stack, top, ints(list(lens)))
    assert m.last_device_status() == 0 and stack[:3].tolist() == [4, 2, 7] and int(top) == 3
    lens[-1] = 17
    m.kv_release(cache, stack, ints([0]), ints(list(lens)), top_out=top)
    assert m.last_device_status() == m.WQ_ERR_ARG and stack[:4].tolist() == [4, 2, 7, bad] and int(top) == 4
    assert stack[4:].tolist() == [-9] * 5
    m.kv_release(cache, stack, ints([0]), ints(list(lens)), ints([40] * batch), top_out=top)      # kept: not looked at
    assert m.last_device_status() == 0 and int(top) == 0


def test_release_then_reserve_gives_every_page_once():
    """Twenty steps of requests that come, grow and go, replayed from one graph: no page is held twice, none is lost."""
    need_gpu()
    m, rng, size, batch, ld = wq(), np.random.default_rng(5), 16, 37, 20
    pages = 260
    table = torch.full((batch, ld), -1, dtype=torch.int32, device="cuda")
    cache, stack, top = small_cache(size, pages, table), cuda(rng.permutation(pages).astype(np.int32)), ints([pages])
    lens, keep, counts = (ints([0] * batch) for _ in range(3))
    out = m.kv_reserve(cache, stack, top, keep, counts, 4000)

    def step():
        m.kv_release(cache, stack, top, lens, keep)
        m.kv_reserve(cache, stack, top, keep, counts, 4000, out=out)
        torch.add(keep, out[3], out=lens)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(20):
        held = lens.cpu().numpy()
        ends = rng.random(batch) < 0.2
        keep.copy_(cuda(np.where(ends, 0, held).astype(np.int32)))
        counts.copy_(cuda(np.where(held == 0, rng.integers(0, 200, batch), rng.integers(0, 9, batch)).astype(np.int32)))
        g.replay()
        now = lens.cpu().numpy()
        assert np.array_equal(now, keep.cpu().numpy() + out[3].cpu().numpy())
        mine = [table[b, :-(-int(now[b]) // size)].tolist() for b in range(batch)]
        assert sorted(sum(mine, []) + stack[:int(top)].tolist()) == list(range(pages))
        slots, starts = out[0].tolist(), out[2].tolist()
        for b in range(batch):
            at = range(int(keep[b]), int(now[b]))
            assert slots[starts[b]:starts[b] + len(at)] == [mine[b][t // size] * size + t % size for t in at]
    assert m.last_device_status() == 0


# ------------------------------------------------------------------ packed appends
@pytest.mark.parametrize("fmt", ["q4_0", "nvfp4"])
@pytest.mark.parametrize("H,D,page", [(20, 64, 0), (8, 128, 16), (1, 64, 48), (3, 128, 32), (6, 64, 64)])
@pytest.mark.parametrize("tokens", [1, 5, 37, 200])
def test_append_slots_bits_and_nothing_else(fmt, H, D, page, tokens):
    need_gpu()
    m, case = wq(), Case(81, fmt, H, D, 3, 150, page)
    cache, before = case.upload(), [a.copy() for pair in case.rows for a in pair]
    slots = case.rng.permutation(case.pages * case.size)[:tokens].astype(np.int64)
    slots[case.rng.random(tokens) < 0.1] = -1
    kv = bf16(case.rng, tokens, 2 * H * D + 8)
    k, v = (kv[:, j * H * D:(j + 1) * H * D].unflatten(-1, (H, D)) for j in range(2))     # rows of a wider buffer
    dev = kv.cuda()
    m.kv_append_slots(cache, *(dev[:, j * H * D:(j + 1) * H * D].unflatten(-1, (H, D)) for j in range(2)), cuda(slots))
    there = slots >= 0
    for j, x in enumerate((k, v)):
        codes, scales = OK.encode_rows(fmt, x.float().numpy()[there], case.g[j])
        before[2 * j][slots[there] // case.size, :, slots[there] % case.size] = codes
        before[2 * j + 1][slots[there] // case.size, :, slots[there] % case.size] = scales
    for j in range(4):
        assert np.array_equal(raw(case.t[j]), before[j].view(np.uint8)), ("k codes", "k scales", "v codes", "v scales")[j]
    assert m.last_device_status() == 0


def test_append_slots_outside_the_cache():
    need_gpu()
    m, case = wq(), Case(82, "q4_0", 2, 64, 1, 64, 16)
    cache, before = case.upload(), [a.copy() for pair in case.rows for a in pair]
    k = bf16(case.rng, 4, 2, 64).cuda()
    m.kv_append_slots(cache, k, k, torch.tensor([case.pages * 16, 2 ** 40 + 5, -(2 ** 50), 2 ** 62], device="cuda"))
    assert m.last_device_status() == m.WQ_ERR_ARG
    assert all(np.array_equal(raw(t), b.view(np.uint8)) for t, b in zip(case.t, before))
    m.kv_append_slots(cache, k[:0], k[:0], torch.empty(0, dtype=torch.int64, device="cuda"))
    assert m.last_device_status() == 0


def test_append_slots_past_32_bits():
    """Slots of 2^31 and more, in code arrays of more than 2^32 bytes."""
    need_gpu()
    m = wq()
    pages, size, H, D = 4720000, 464, 1, 64                              # 2.19e9 slots, 7e10 bytes of codes for K and for V
    if torch.cuda.mem_get_info()[0] < 2.1e11:
        pytest.skip("needs 210 GB of free memory")
    cache = m.kv_alloc("q4_0", pages, size, H, D, ints([[pages - 1, 0], [pages - 2, 4629430]]))
    slots = torch.tensor([(pages - 1) * size + i for i in (0, 1, 463)] + [5, 4629430 * size + 3, 2 ** 31 - 1, 2 ** 31], device="cuda")
    x = bf16(np.random.default_rng(3), 7, H, D)
    m.kv_append_slots(cache, x.cuda(), x.cuda(), slots)
    codes, _ = OK.encode_rows("q4_0", x.float().numpy())
    for i, s in enumerate(slots.tolist()):
        assert np.array_equal(cache.tensors[2][s // size, :, s % size].cpu().numpy(), codes[i])
    assert m.last_device_status() == 0


# ------------------------------------------------------------------ trees
@pytest.mark.parametrize("tokens", [1, 2, 31, 32, 33, 64, 100, 1024])
@pytest.mark.parametrize("window", [0, 1, 3, 40])
def test_tree_mask(tokens, window):
    need_gpu()
    m, rng = wq(), np.random.default_rng(tokens)
    parents = random_trees(rng, 6, tokens, int(rng.integers(1, 9)))
    parents[5] = np.arange(tokens) - 1                                   # a chain
    counts = [tokens, max(1, tokens // 2), 0, -3, tokens + 9, tokens]
    for c in (counts, None):
        mask, depth = m.tree_mask(cuda(parents), None if c is None else ints(c), window=window)
        for b in range(6):
            n = tokens if c is None else min(max(c[b], 0), tokens)
            seen, d = OK.ancestors(parents[b], n, window)
            assert np.array_equal(mask[b].cpu().numpy(), OK.mask_words(seen)) and np.array_equal(depth[b].cpu().numpy(), d)
    assert m.last_device_status() == 0


def test_tree_mask_of_parents_that_come_late():
    need_gpu()
    m = wq()
    bad = ints([[-1, 1, 5, -2, 3, 2 ** 31 - 1]])
    mask, depth = m.tree_mask(bad)
    assert m.last_device_status() == m.WQ_ERR_ARG
    assert mask.flatten().tolist() == [1, 2, 4, 8, 24, 32] and depth.tolist() == [[0, 0, 0, 0, 1, 0]]
    mask, _ = m.tree_mask(bad, ints([1]))                                # nodes past the count are not looked at
    assert m.last_device_status() == 0 and mask.flatten().tolist() == [1, 0, 0, 0, 0, 0]


# ------------------------------------------------------------------ kept paths
@pytest.mark.parametrize("fmt", ["q4_0", "nvfp4"])
@pytest.mark.parametrize("H,D,page", [(20, 64, 0), (8, 128, 16), (3, 64, 48)])
@pytest.mark.parametrize("n", [1, 4, 17, 64, 512])
def test_keep_moves_rows_and_nothing_else(fmt, H, D, page, n):
    """Any path: rising ones, and permutations whose rows overwrite each other."""
    need_gpu()
    m, case = wq(), Case(83, fmt, H, D, 4, 100 + n, page)
    cache, before = case.upload(), [a.copy() for pair in case.rows for a in pair]
    start, counts = [7, 0, 93, 50], [n, n, max(0, n - 3), 0]
    path = np.stack([np.sort(case.rng.permutation(n + 7)[:n]), case.rng.permutation(n), np.arange(n), case.rng.permutation(n)]).astype(np.int32)
    m.kv_keep(cache, ints(start), cuda(path), ints(counts))
    want = [a.copy() for a in before]
    for b in range(4):
        to, off = case.at(b, start[b] + np.arange(counts[b]))
        frm, foff = case.at(b, start[b] + path[b, :counts[b]])
        for w, a in zip(want, before):
            w[to, :, off] = a[frm, :, foff]
    assert all(np.array_equal(raw(t), w.view(np.uint8)) for t, w in zip(case.t, want))
    assert m.last_device_status() == 0


def test_keep_of_rows_outside_the_cache():
    need_gpu()
    m, case = wq(), Case(84, "q4_0", 2, 64, 3, 64, 16)
    case.table[1, 1] = 10 ** 6
    cache, before = case.upload(), [a.copy() for pair in case.rows for a in pair]
    path = np.array([[1, 2, 60, -70], [0, 9, 1, 2], [2 ** 31 - 1, -2 ** 31, 3, 2]], np.int32)
    m.kv_keep(cache, ints([5, 10, 62]), cuda(path), None)
    assert m.last_device_status() == m.WQ_ERR_ARG
    want = [a.copy() for a in before]
    for b, to, frm in [(0, 5, 6), (0, 6, 7), (1, 12, 11), (1, 13, 12)]:      # everything else starts or ends nowhere
        (p, o), (q, r) = case.at(b, np.array([to])), case.at(b, np.array([frm]))
        for w, a in zip(want, before):
            w[p, :, o] = a[q, :, r]
    assert all(np.array_equal(raw(t), w.view(np.uint8)) for t, w in zip(case.t, want))


@pytest.mark.parametrize("fmt", ["q4_0", "nvfp4"])
@pytest.mark.parametrize("page", [0, 16])
def test_keep_of_no_node(fmt, page):
    """A node of -1 (the parent of a root, and what short paths are filled with) is no row of the context."""
    need_gpu()
    m, case = wq(), Case(86, fmt, 2, 64, 2, 64, page)
    cache, before = case.upload(), [a.copy() for pair in case.rows for a in pair]
    path = np.array([[2, 3, -1, -1, -5], [-1, 4, -2 ** 31, 6, -30]], np.int32)
    m.kv_keep(cache, ints([30, 30]), cuda(path))
    assert m.last_device_status() == m.WQ_ERR_ARG
    want = [a.copy() for a in before]
    for b, to, frm in [(0, 30, 32), (0, 31, 33), (1, 31, 34), (1, 33, 36)]:
        (p, o), (q, r) = case.at(b, np.array([to])), case.at(b, np.array([frm]))
        for w, a in zip(want, before):
            w[p, :, o] = a[q, :, r]
    assert all(np.array_equal(raw(t), w.view(np.uint8)) for t, w in zip(case.t, want))
    m.kv_keep(cache, ints([30, 30]), cuda(path), ints([2, 0]))             # behind the counts it is not looked at
    assert m.last_device_status() == 0


# ------------------------------------------------------------------ a run of them
@pytest.mark.parametrize("fmt", ["q4_0", "nvfp4"])
def test_a_drafting_step(fmt):
    """Pages for the drafts, their rows to the slots, attention of the trees, the accepted paths kept, the rest given back:
    the sequences then hold what appending the paths alone leaves, and the next token sees it."""
    need_gpu()
    m, rng, B, L, H, D, size = wq(), np.random.default_rng(9), 3, 9, 2, 64, 16
    table = torch.full((B, 6), -1, dtype=torch.int32, device="cuda")
    g = [None, None] if fmt == "q4_0" else [torch.tensor([0.002], device="cuda")] * 2
    cache, stack, top = m.kv_alloc(fmt, 12, size, H, D, table, *g), ints(list(range(12))), ints([12])
    ctx = [30, 16, 5]
    k, v = (bf16(rng, sum(ctx), H, D).cuda() for _ in range(2))
    slots, _, starts, granted = m.kv_reserve(cache, stack, top, ints([0] * B), ints(ctx), sum(ctx))
    assert granted.tolist() == ctx and int(top) == 12 - 4
    m.kv_append_slots(cache, k, v, slots)
    parents, counts = random_trees(rng, B, L), [L, 4, 7]
    nodes = [OK.ancestors(p, n) for p, n in zip(parents, counts)]
    dk, dv = (bf16(rng, B, L, H, D).cuda() for _ in range(2))
    slots, positions, starts, granted = m.kv_reserve(cache, stack, top, ints(ctx), ints(counts), 3 * L)
    assert granted.tolist() == counts
    flat = torch.cat([torch.arange(n) + b * L for b, n in enumerate(counts)]).cuda()
    m.kv_append_slots(cache, dk.flatten(0, 1)[flat], dv.flatten(0, 1)[flat], slots[:len(flat)])
    lens = ints([c + n for c, n in zip(ctx, counts)])
    q = bf16(rng, B, L, 4, D)
    mask, depth = m.tree_mask(cuda(parents), ints(counts))
    out = m.attend(cache, q.cuda(), lens, counts=ints(counts), tree=(mask, depth), out_f32=True).cpu().numpy()
    gv = [None if x is None else np.float32(0.002) for x in g]
    rows = [[OK.decode_rows(fmt, *OK.encode_rows(fmt, x.float().cpu().numpy(), gv[0]), gv[0]) for x in pair] for pair in ((k, v), (dk, dv))]
    paths, kept = np.zeros((B, L), np.int32), []
    for b in range(B):
        at = sum(ctx[:b])
        kk, vv = (np.concatenate([rows[0][j][at:at + ctx[b]], rows[1][j][b, :counts[b]]]) for j in range(2))
        seen = OK.visible(L, counts[b], len(kk), nodes=nodes[b][0], depth=nodes[b][1])
        ref, *_ = OK.attend_seen(q[b].float().numpy(), kk, vv, seen, D ** -0.5)
        assert np.allclose(out[b], ref, atol=2e-2)
        path = np.flatnonzero(nodes[b][0][counts[b] - 1])               # the last node's ancestors are accepted
        paths[b, :len(path)] = path
        kept.append(np.concatenate([np.arange(ctx[b]), ctx[b] + path]))
        rows.append((kk[kept[b]], vv[kept[b]]))
    n = ints([len(x) for x in kept])
    m.kv_keep(cache, ints(ctx), cuda(paths), ints([len(x) - c for x, c in zip(kept, ctx)]))
    m.kv_release(cache, stack, top, lens, n)
    assert int(top) == 12 - sum(-(-len(x) // size) for x in kept)
    got = m.kv_read(cache, 40, counts=n, out_f32=True)
    for b in range(B):
        for j in range(2):
            assert np.array_equal(got[j][b, :len(kept[b])].cpu().numpy(), rows[2 + b][j])
    assert m.last_device_status() == 0


# ------------------------------------------------------------------ how calls may be made
def test_on_a_stream_that_is_given():
    need_gpu()
    m, case, side = wq(), Case(85, "q4_0", 2, 64, 2, 96, 16), torch.cuda.Stream()
    cache, before = case.upload(), [a.copy() for pair in case.rows for a in pair]
    table = torch.full((2, 3), -1, dtype=torch.int32, device="cuda")
    turns, stack, top = small_cache(16, 9, table), ints([4, 7, 2, 0, 8, -1, -1, -1, -1]), ints([5])
    k, path, parents = bf16(case.rng, 3, 2, 64).cuda(), ints([[2, 1, 4]]), ints([[-1, 0, 0]])
    side.wait_stream(torch.cuda.current_stream())
    got = m.kv_reserve(turns, stack, top, ints([0, 0]), ints([17, 1]), 20, stream=side)
    m.kv_release(turns, stack, top, ints([17, 1]), ints([16, 1]), stream=side)
    m.kv_append_slots(cache, k, k, torch.tensor([1, 40, 3], device="cuda"), stream=side)
    m.kv_keep(cache, ints([50]), path, stream=side)
    mask, depth = m.tree_mask(parents, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert got[0].tolist() == [8 * 16 + i for i in range(16)] + [0, 2 * 16, -1, -1] and table.tolist() == [[8, 0, -1], [2, -1, -1]]
    assert int(top) == 3 and stack.tolist() == [4, 7, 0, 0, 8, -1, -1, -1, -1]
    assert mask.flatten().tolist() == [1, 3, 5] and depth.tolist() == [[0, 1, 1]]
    codes, scales = OK.encode_rows("q4_0", k.float().cpu().numpy())
    for j in range(2):
        for i, slot in enumerate((1, 40, 3)):
            before[2 * j][slot // 16, :, slot % 16], before[2 * j + 1][slot // 16, :, slot % 16] = codes[i], scales[i]
        for a in before[2 * j:2 * j + 2]:
            (p, o), (s, t) = case.at(0, np.arange(50, 53)), case.at(0, 50 + np.array([2, 1, 4]))
            a[p, :, o] = a[s, :, t].copy()
    assert all(np.array_equal(raw(t), b.view(np.uint8)) for t, b in zip(case.t, before)) and m.last_device_status() == 0


def test_empty_calls():
    need_gpu()
    m = wq()
    table = torch.full((2, 3), -1, dtype=torch.int32, device="cuda")
    cache, stack, top, none = small_cache(16, 9, table), ints([4, 7]), ints([2]), ints([])
    got = m.kv_reserve(cache, stack, top, none, none, 3)
    assert got[0].tolist() == [-1] * 3 and got[1].tolist() == [0] * 3 and got[2].tolist() == [0] and got[3].tolist() == [] and int(top) == 2
    got = m.kv_reserve(cache, stack, top, ints([0, 3]), ints([5, 0]), 0)         # tables without slots
    assert m.last_device_status() == 0 and got[0].numel() == 0 and got[3].tolist() == [5, 0] and int(top) == 1 and int(table[0, 0]) == 7
    m.kv_release(cache, stack, top, none)
    assert int(top) == 1
    m.kv_release(cache, none, ints([0]), ints([0, 0]))
    m.kv_keep(cache, ints([0, 0]), torch.empty((2, 0), dtype=torch.int32, device="cuda"))
    mask, depth = m.tree_mask(torch.empty((0, 5), dtype=torch.int32, device="cuda"))
    assert mask.shape == (0, 5, 1) and depth.shape == (0, 5) and m.last_device_status() == 0


def test_refusals_from_python():
    need_gpu()
    m = wq()
    table = torch.full((2, 3), -1, dtype=torch.int32, device="cuda")
    cache, slab = small_cache(16, 9, table), small_cache(16, 9, None)
    stack, top, two = ints([4, 7]), ints([2]), ints([0, 1])
    launches = m.lib.wq_kernel_launches()
    for call in (lambda: m.kv_reserve(slab, stack, top, two, two, 3), lambda: m.kv_reserve(cache, stack.cpu(), top, two, two, 3),
                 lambda: m.kv_reserve(cache, stack, top.cpu(), two, two, 3), lambda: m.kv_reserve(cache, stack, top, two, ints([1]), 3),
                 lambda: m.kv_reserve(cache, stack, top, ints([0] * 3), ints([0] * 3), 3), lambda: m.kv_reserve(cache, stack, None, two, two, 3),
                 lambda: m.kv_reserve(cache, stack, top, two, two, -1), lambda: m.kv_reserve(cache, stack, top, two, two, 3, out=(two,) * 4),
                 lambda: m.kv_reserve(cache, stack, top, two, two, 3, top_out=two), lambda: m.kv_release(slab, stack, top, two),
                 lambda: m.kv_release(cache, stack, top, two, ints([1])), lambda: m.kv_release(cache, stack.long(), top, two),
                 lambda: m.kv_keep(cache, two, ints([0, 1])), lambda: m.kv_keep(cache, ints([0]), ints([[0, 1], [1, 0]])),
                 lambda: m.kv_keep(cache, ints([0] * 3), ints([[0], [1], [2]])),
                 lambda: m.kv_append_slots(cache, torch.zeros(2, 1, 64, device="cuda"), torch.zeros(2, 1, 64, device="cuda"), two.long()),
                 lambda: m.kv_append_slots(cache, torch.zeros(2, 1, 64, device="cuda").bfloat16(), torch.zeros(2, 1, 64, device="cuda").bfloat16(), two),
                 lambda: m.kv_append_slots(cache, torch.zeros(2, 2, 64, device="cuda").bfloat16(), torch.zeros(2, 2, 64, device="cuda").bfloat16(),
                                           two.long())):
        with pytest.raises(AssertionError):
            call()
    with pytest.raises(m.WQError):
        m.kv_keep(cache, ints([0]), torch.zeros((1, 513), dtype=torch.int32, device="cuda"))
    with pytest.raises(m.WQError):
        m.kv_reserve(cache, stack, top, two, two, 0, out=(torch.empty(0, dtype=torch.int64, device="cuda"), ints([]), ints([0] * 3), two))
    with pytest.raises(m.WQError):
        m.tree_mask(torch.full((1, 1025), -1, dtype=torch.int32, device="cuda"))
    assert m.lib.wq_kernel_launches() == launches and m.last_device_status() == 0
