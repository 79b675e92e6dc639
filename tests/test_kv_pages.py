"""kv_reserve and kv_append against their definitions in plain Python, exactly; a prompt, drafted tokens and an
eviction on one cache; refusals."""
import ctypes

import numpy as np
import pytest

import sparse_weight_matmul_amd as swm
from test_prompt_attention import attend, bounds, check, ints

gpu = pytest.mark.gpu


def reserve(table, lengths, counts, free, count, pages, S, tokens):
    """The definition, page by page; arrays change in place.  (starts, slots, granted, free pages)."""
    B, per = table.shape
    stack = free[:count].tolist()
    granted, slots, starts, room = np.zeros(B, np.int32), np.full(tokens, -1, np.int64), [0], True
    old = np.clip(lengths, 0, per * S)
    for b in range(B):
        new = int(old[b]) + int(counts[b])
        if new < old[b]:
            new = max(0, new)
            for i in range(-(-new // S), -(-int(old[b]) // S)):
                if 0 <= table[b, i] < pages:
                    stack.append(int(table[b, i]))
                table[b, i] = -1
            granted[b], lengths[b] = new - old[b], new
    free[:len(stack)] = stack
    for b in range(B):
        starts.append(starts[-1] + max(0, int(counts[b])))
        new = int(old[b]) + int(counts[b])
        if counts[b] < 0:
            continue
        lengths[b] = old[b]
        if new > per * S:
            continue
        first, last = -(-int(old[b]) // S), -(-new // S)
        if last > first:
            room = room and last - first <= len(stack)
            if not room:
                continue
        for i in range(first, last):
            table[b, i] = stack.pop()
        t = np.arange(old[b], new)
        page = table[b, t // S].astype(np.int64)
        slots[starts[-2]:starts[-1]] = np.where((page >= 0) & (page < pages), page * S + t % S, -1)[:tokens]
        granted[b], lengths[b] = counts[b], new
    return np.minimum(starts, 2**31 - 1).astype(np.int32), slots, granted, len(stack)


def pool_of(pages, S, heads=1, dim=8):
    import torch
    return torch.zeros((pages, S, heads, dim), dtype=torch.float16, device="cuda")


def state(lengths, per, S, spare, seed=0):
    """(table, free pages, how many, pages of the pool): pages dealt at random."""
    r = np.random.default_rng([seed, len(lengths), per, S])
    need = [-(-n // S) for n in lengths]
    P = sum(need) + spare
    pages, at = r.permutation(P), 0
    table = np.full((len(lengths), per), -1, np.int32)
    for b, x in enumerate(need):
        table[b, :x] = pages[at:at + x]
        at += x
    free = np.full(P, -7, np.int32)
    free[:spare] = pages[at:]
    return table, free, spare, P


def run_both(table, lengths, counts, free, count, P, S, tokens=None, steps=1, **kw):
    """The call and the definition on the same state, everything compared; the device's tensors."""
    import torch
    lengths, counts = np.asarray(lengths, np.int32), np.asarray(counts, np.int32)
    tokens = int(np.maximum(counts, 0).sum()) if tokens is None else tokens
    k = pool_of(P, S)
    dev = [ints(table), ints(lengths), ints(counts), ints(free), ints([count])]
    c = swm.PagedCache(k, k, dev[0], dev[1])
    got = swm.kv_reserve(c, dev[2], dev[3], dev[4], tokens, **kw)
    torch.cuda.synchronize()
    want = reserve(table, lengths, counts, free, count, P, S, tokens)
    for name, a, b in zip(("starts", "slots", "granted"), got, want):
        assert np.array_equal(a.cpu().numpy(), b), name
    for name, a, b in (("table", dev[0], table), ("lengths", dev[1], lengths), ("free", dev[3], free)):
        assert np.array_equal(a.cpu().numpy(), b), name
    assert dev[4].tolist() == [want[3]]
    return c, got


RESERVES = [
    # lengths, counts, slots in a page, pages of a table, spare pages
    ([5], [1], 16, 4, 3),
    ([16], [1], 16, 4, 3),
    ([0], [0], 16, 4, 3),
    ([0, 1, 15, 16, 17], [1, 1, 1, 1, 1], 16, 3, 5),
    ([20, 40, 7], [-3, -40, -1], 8, 6, 0),
    ([20, 40, 7], [-100, 3, -7], 8, 6, 0),               # dropped past the start; pages come back in the same call
    ([30, 30, 30, 30], [10, 50, 1, 3], 8, 16, 3),        # the second does not fit: only what needs no page follows
    ([30, 30], [200, 2], 8, 6, 60),                      # the first would outgrow its table
    ([47, 48, 49], [1, 1, 1], 1, 60, 3),                 # pages of one slot
    ([90, 250, 3], [130, -249, 64], 100, 4, 2),
    ([0] * 70, [100] * 70, 32, 4, 280),                  # prompts
    ([(31 * b) % 90 for b in range(300)], [1] * 300, 16, 8, 40),
    ([(31 * b) % 90 + 1 for b in range(1500)], [(b % 3 - 1) * (b % 17) for b in range(1500)], 4, 64, 200),
    ([(7 * b) % 50 for b in range(5000)], [5 - (b * b) % 11 for b in range(5000)], 8, 16, 3000),
    ([10, 4000], [9000, -4000], 16, 600, 800),
]


@gpu
@pytest.mark.parametrize("lengths,counts,S,per,spare", RESERVES)
def test_reserve_is_its_definition(gpu_lib, lengths, counts, S, per, spare):
    table, free, count, P = state(lengths, per, S, spare)
    run_both(table, lengths, counts, free, count, P, S)


@gpu
def test_dropped_drafts_give_back_the_pages_they_leave(gpu_lib):
    """One page here: 76 -> 71, 21 -> 2 and 36 -> 34 tokens keep 5 of 5, 1 of 2 and 3 of 3."""
    table, free, count, P = state([76, 21, 36], 12, 16, 20)
    left = table[1, 1]
    c, got = run_both(table, [76, 21, 36], [-5, -19, -2], free, count, P, 16)
    assert free[20] == left and (table >= 0).sum(1).tolist() == [5, 1, 3] and got[2].tolist() == [-5, -19, -2]


@gpu
def test_many_steps_keep_every_page(gpu_lib):
    """Random growth and shrinkage: after every step each page has one owner."""
    import torch
    r = np.random.default_rng(4)
    B, S, per = 23, 16, 20
    lengths = r.integers(0, 200, B).astype(np.int32)
    table, free, count, P = state(lengths.tolist(), per, S, 60)
    k = pool_of(P, S)
    dt, dl, df, dc = ints(table), ints(lengths), ints(free), ints([count])
    c = swm.PagedCache(k, k, dt, dl)
    for step in range(40):
        counts = r.integers(-60, 70, B).astype(np.int32) if step % 3 else np.ones(B, np.int32)
        tokens = int(np.maximum(counts, 0).sum())
        got = swm.kv_reserve(c, ints(counts), df, dc, tokens)
        want = reserve(table, lengths, counts, free, count, P, S, tokens)
        count = want[3]
        assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(got, want[:3]))
        assert np.array_equal(dt.cpu().numpy(), table) and np.array_equal(dl.cpu().numpy(), lengths)
        owned = table[np.arange(per) < -(-lengths[:, None] // S)].tolist() + df[:count].tolist()
        assert sorted(owned) == list(range(P))


@gpu
def test_reserve_of_any_content(gpu_lib):
    """Entries that name no page, lengths and a number of free pages out of range, counts next to 2^31."""
    S, per = 8, 6
    table, free, count, P = state([40, 33, 20, 48], per, S, 4)
    table[0, 3], table[0, 4], table[2, 2] = -1, P, 1 << 30
    run_both(table, [40, 33, 20, 48], [-40, 5, 2, (1 << 31) - 1], free, count, P, S, tokens=64)
    table, free, count, P = state([40, 33, 20], per, S, 4)
    run_both(table, [40, 33, 20], [-(1 << 31), 1, 4], free, count, P, S)
    table, free, count, P = state([0, 48, 0, 9], per, S, 4)
    lengths = [-5, 1000, -(1 << 31), 9]
    run_both(table, lengths, [3, 1, 0, 0], free, count, P, S)
    import torch
    for count in (-3, 1 << 30):  # none, or as many as the list holds
        table, free, _, P = state([8, 8], per, S, 4)
        free[:] = np.arange(P)
        k, dt, dl, df, dc = pool_of(P, S), ints(table), ints([8, 8]), ints(free), ints([count])
        _, _, granted = swm.kv_reserve(swm.PagedCache(k, k, dt, dl), ints([8, 8]), df, dc, 16)
        assert granted.tolist() == ([0, 0] if count < 0 else [8, 8])
        assert dc.tolist() == ([0] if count < 0 else [P - 2])


@gpu
def test_more_rows_than_tokens(gpu_lib):
    """Rows of the slot map behind the last token hold -1, also those that a second launch fills."""
    table, free, count, P = state([3, 0, 9], 8, 16, 20)
    run_both(table, [3, 0, 9], [2, 60, -9], free, count, P, 16, tokens=100)
    table, free, count, P = state([3, 0, 9], 8, 16, 20)
    run_both(table, [3, 0, 9], [2, 60, -9], free, count, P, 16, tokens=9000)
    table, free, count, P = state([3, 0, 9], 8, 16, 20)
    run_both(table, [3, 0, 9], [0, 0, 0], free, count, P, 16, tokens=0)


@gpu
@pytest.mark.parametrize("each", [40, 5000])
def test_reserve_in_a_graph_and_on_a_stream(gpu_lib, each):
    import torch
    S, per, B = 16, 700, 3
    table, free, count, P = state([100, 0, 33], per, S, 2100)
    lengths = np.array([100, 0, 33], np.int32)
    k = pool_of(P, S)
    dt, dl, df, dc = ints(table), ints(lengths), ints(free), ints([count])
    c = swm.PagedCache(k, k, dt, dl)
    counts, tokens = ints([0, 0, 0]), B * each
    outs = dict(starts=ints([0] * 4), slots=torch.zeros(tokens, dtype=torch.int64, device="cuda"), granted=ints([0] * 3))
    swm.kv_reserve(c, counts, df, dc, tokens, **outs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        swm.kv_reserve(c, counts, df, dc, tokens, **outs)
    side = torch.cuda.Stream()
    for step, n in enumerate(([each, 3, 0], [-each, each, 1], [1, -2, each], [2, 0, -each], [-9000, 5, 5])):
        counts.copy_(ints(n))
        if step % 2:
            side.wait_stream(torch.cuda.current_stream())
            got = swm.kv_reserve(c, counts, df, dc, tokens, stream=side)
            torch.cuda.current_stream().wait_stream(side)
        else:
            graph.replay()
            got = tuple(outs.values())
        torch.cuda.synchronize()
        want = reserve(table, lengths, np.array(n, np.int32), free, count, P, S, tokens)
        count = want[3]
        assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(got, want[:3]))
        assert np.array_equal(dt.cpu().numpy(), table) and np.array_equal(dl.cpu().numpy(), lengths)
        assert np.array_equal(df.cpu().numpy(), free) and dc.tolist() == [count]


APPENDS = [
    # tokens, heads, dim, slots in a page, layout of the pools, of the rows
    (1, 1, 8, 16, "token", "separate"),
    (1, 32, 128, 16, "token", "stacked"),
    (33, 4, 80, 24, "head", "stacked"),
    (500, 3, 136, 8, "token", "head"),
    (77, 8, 256, 5, "head", "separate"),
    (1000, 12, 64, 1, "token", "separate"),
    (3000, 2, 128, 100, "head", "head"),
    (5, 40, 248, 16, "token", "separate"),
]


@gpu
@pytest.mark.parametrize("T,H,D,S,layout,rows", APPENDS)
@pytest.mark.parametrize("sums", [False, True])
def test_append_writes_its_rows_and_no_other(gpu_lib, T, H, D, S, layout, rows, sums):
    import torch
    r = np.random.default_rng([T, H, D])
    P = -(-T // S) * 2 + 3
    shape = (P, S, H, D)
    pools = [torch.from_numpy(r.standard_normal(shape).astype(np.float16)).cuda() for _ in range(2)]
    if layout == "head":
        pools = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in pools]
    k, v = (torch.from_numpy(r.standard_normal((T, H, D)).astype(np.float16)).cuda() for _ in range(2))
    k[0, 0, 0], v[-1, -1, -1] = float("nan"), -float("inf")  # rows are copied, whatever they hold
    if rows == "stacked":
        y = torch.cat([k, k, v], 1)
        k, v = y[:, H:2 * H], y[:, 2 * H:]
    elif rows == "head":
        k, v = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (k, v))
    slots = r.permutation(P * S)[:T].astype(np.int64)
    slots[r.random(T) < 0.2] = -1
    if T > 4:
        slots[1], slots[2], slots[3] = P * S, 1 << 40, -(1 << 40)  # outside the pool
    want = [x.clone() for x in pools]
    keep = (slots >= 0) & (slots < P * S)
    at, page, slot = torch.from_numpy(np.nonzero(keep)[0]).cuda(), *(torch.from_numpy(x[keep]).cuda()
                                                                      for x in (slots // S, slots % S))
    want[0][page, slot], want[1][page, slot] = k[at], v[at]
    c = swm.PagedCache(*pools, ints([[0]]), ints([0]))
    kw = {}
    if sums:
        w = torch.from_numpy(r.random((P, H, S)).astype(np.float32)).cuda()
        pos = torch.full((P, H, S), -3, dtype=torch.int32, device="cuda")
        t = torch.from_numpy(r.integers(0, 1 << 30, T).astype(np.int32)).cuda()
        want_w, want_p = w.clone(), pos.clone()
        want_w[page, :, slot], want_p[page, :, slot] = 0.0, t[at][:, None]
        kw = dict(weights=w, positions=pos, at=t)
    assert swm.kv_append(c, k, v, torch.from_numpy(slots).cuda(), **kw) is None
    for a, b in zip(pools, want):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    if sums:
        assert torch.equal(w, want_w) and torch.equal(pos, want_p)


@gpu
def test_append_past_32_bits(gpu_lib):
    """Pools of 32 GiB, more than 2^31 slots of one row: slots at their very end."""
    import torch
    P, S, D = (1 << 18) + 1, 1 << 13, 8
    k, v = (torch.empty((P, S, 1, D), dtype=torch.float16, device="cuda") for _ in range(2))
    at = [P * S - 1, P * S, 0, (1 << 31) + 5, 1 << 62]
    for i in at:
        if i < P * S:
            k[i // S, i % S], v[i // S, i % S] = 0, 0
    rows = torch.arange(40, dtype=torch.float16, device="cuda").view(5, 1, 8) + 1
    c = swm.PagedCache(k, v, ints([[0]]), ints([0]))
    swm.kv_append(c, rows, -rows, torch.tensor(at, dtype=torch.int64, device="cuda"))
    for x, i in enumerate(at):
        if i < P * S:
            assert torch.equal(k[i // S, i % S], rows[x]) and torch.equal(v[i // S, i % S], -rows[x])


@gpu
def test_append_next_to_its_limit(gpu_lib):
    """Almost 2^37 halves of keys, as many as a call takes, of which the last token alone has a slot; with a token
    more they are refused."""
    import torch
    H, D, T = 65535, 256, 8192
    assert T * H * D < 2**37 - 2**13 <= (T + 1) * H * D
    row = torch.randn((1, H, D), device="cuda").half()
    k, v = (torch.zeros((2, 1, H, D), dtype=torch.float16, device="cuda") for _ in range(2))
    c = swm.PagedCache(k, v, ints([[0]]), ints([0]))
    slots = torch.full((T + 1,), -1, dtype=torch.int64, device="cuda")
    slots[T - 1] = 1
    swm.kv_append(c, row.expand(T, H, D), (-row).expand(T, H, D), slots[:T])
    assert torch.equal(k[1, 0], row[0]) and torch.equal(v[1, 0], -row[0])
    assert not bool(k[0].any()) and not bool(v[0].any())
    with pytest.raises(swm.SwmError, match="UNSUPPORTED"):
        swm.kv_append(c, row.expand(T + 1, H, D), row.expand(T + 1, H, D), slots)


@gpu
def test_append_on_a_stream_and_in_a_graph(gpu_lib):
    import torch
    pools = [torch.zeros((9, 16, 2, 64), dtype=torch.float16, device="cuda") for _ in range(2)]
    c = swm.PagedCache(*pools, ints([[0]]), ints([0]))
    k, v = (torch.randn(20, 2, 64, device="cuda").half() for _ in range(2))
    slots = torch.arange(20, dtype=torch.int64, device="cuda")
    swm.kv_append(c, k, v, slots)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        swm.kv_append(c, k, v, slots)
    side = torch.cuda.Stream()
    for i in range(1, 5):
        slots.copy_(torch.arange(20, device="cuda") * 7 % 141 + i)
        k.mul_(-1)
        for p in pools:
            p.zero_()
        if i % 2:
            graph.replay()
        else:
            side.wait_stream(torch.cuda.current_stream())
            swm.kv_append(c, k, v, slots, stream=side)
            torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        for p, x in zip(pools, (k, v)):
            want = torch.zeros_like(p)
            want.view(144, 2, 64)[slots] = x
            assert torch.equal(p, want)


@gpu
def test_a_prompt_drafts_and_an_eviction_on_one_cache(gpu_lib):
    """Pages reserved, rows appended, drafts verified and rolled back, a token attended to, the cache cut back:
    at each step the cache's tokens are the sequences'."""
    import torch
    r = np.random.default_rng(8)
    B, Hq, Hkv, D, S, per, P = 3, 4, 2, 64, 16, 12, 30
    k, v = (torch.full((P, S, Hkv, D), float("nan"), dtype=torch.float16, device="cuda") for _ in range(2))
    table, lengths = ints(np.full((B, per), -1)), ints([0] * B)
    free, count = ints(r.permutation(P)), ints([P])
    w, pos = torch.full((P, Hkv, S), 9.0, device="cuda"), ints(np.zeros((P, Hkv, S)))
    c = swm.PagedCache(k, v, table, lengths)
    have = [np.zeros((0, Hq + 2 * Hkv, D), np.float16) for _ in range(B)]
    scale = D ** -0.5

    def rows(n):
        x = r.standard_normal((sum(n), Hq + 2 * Hkv, D)).astype(np.float16)
        return x, torch.from_numpy(x).cuda()

    def add(n):
        """n new tokens of each sequence into the cache: (rows of the stacked product, starts)."""
        x, y = rows(n)
        at = ints(np.concatenate([np.arange(len(have[b]), len(have[b]) + n[b]) for b in range(B)]))
        starts, slots, granted = swm.kv_reserve(c, ints(n), free, count, sum(n))
        assert granted.tolist() == list(n)
        swm.kv_append(c, y[:, Hq:Hq + Hkv], y[:, Hq + Hkv:], slots, weights=w, positions=pos, at=at)
        for b, a in enumerate(bounds(n)[:-1]):
            have[b] = np.concatenate([have[b], x[a:a + n[b]]])
        return x, y, starts

    def want(q, b, sees):
        ref = [attend(q[:, h], have[b][:, Hq + h * Hkv // Hq], have[b][:, Hq + Hkv + h * Hkv // Hq], scale, sees)
               for h in range(Hq)]
        return np.stack([x[0] for x in ref], 1), np.stack([x[1] for x in ref], 1)

    n = [70, 1, 33]
    x, y, starts = add(n)
    out = swm.prompt_attention(y[:, :Hq], y[:, Hq:Hq + Hkv], y[:, Hq + Hkv:], starts)
    for b, a in enumerate(bounds(n)[:-1]):
        check(out[a:a + n[b]], *want(x[a:a + n[b], :Hq], b, np.tril(np.ones((n[b], n[b]), bool))), "prompt")
    n = [6, 20, 3]  # drafts: all children of the first
    x, y, starts = add(n)
    parents = ints(np.concatenate([[-1] + [0] * (t - 1) for t in n]))
    out = swm.tree_attention(c, y[:, :Hq], starts, parents, max_tokens=20)
    for b, a in enumerate(bounds(n)[:-1]):
        sees = np.ones((n[b], len(have[b])), bool)
        sees[:, -n[b] + 1:] = np.eye(n[b], dtype=bool)[:, 1:]
        check(out[a:a + n[b]], *want(x[a:a + n[b], :Hq], b, sees), "drafts")
    left = int(count[0])
    swm.kv_reserve(c, ints([-5, -19, -2]), free, count, 0)  # the first draft of each is kept
    assert int(count[0]) >= left
    have[:] = [h[:len(h) - d] for h, d in zip(have, (5, 19, 2))]
    x, y, starts = add([1, 1, 1])
    out = swm.paged_attention(c, y[:, :Hq].contiguous(), weights=w)
    for b in range(B):
        check(out[b:b + 1], *want(x[b:b + 1, :Hq], b, np.ones((1, len(have[b])), bool)), "token")
        t = np.arange(len(have[b]))
        page = table[b].cpu().numpy()[t // S]
        total = w.cpu().numpy()[page, :, t % S].sum()  # the appended rows began at zero
        assert abs(total - Hq) < 1e-4
        assert np.array_equal(pos.cpu().numpy()[page, :, t % S], np.repeat(t[:, None], Hkv, 1))
    new, kept = swm.kv_evict(c, w, pos, 32, recent=4)
    assert new.tolist() == [32, 3, 32]
    pages = [-(-int(x) // S) for x in lengths.tolist()]
    swm.kv_reserve(c, new - lengths, free, count, 0)  # the pages that the eviction left
    assert lengths.tolist() == [32, 3, 32]
    used = table[table >= 0].tolist() + free[: int(count[0])].tolist()
    assert sorted(used) == list(range(P)) and sum(pages) > int((table >= 0).sum())


@gpu
def test_new_tensors_are_memory_of_the_stream(gpu_lib):
    """What the calls allocate on a stream that is not the current one is no block that the current one just gave back."""
    import torch
    k = torch.randn((40, 16, 2, 64), device="cuda").half()
    c = swm.PagedCache(k, k.clone(), ints(np.arange(40).reshape(1, 40)), ints([640]))
    q, starts = torch.randn((30, 4, 64), device="cuda").half(), ints([0, 30])
    free, count, n = ints(np.zeros(40)), ints([0]), ints([0])
    for call in (lambda s: [swm.prompt_attention(q, q, q, starts, stream=s)],
                 lambda s: [swm.tree_attention(c, q, starts, max_tokens=30, stream=s)],
                 lambda s: list(swm.kv_reserve(c, n, free, count, 5, stream=s))):
        want = call(None)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        given = [torch.empty_like(t) for t in want for _ in range(4)]
        held = {t.data_ptr() for t in given}
        del given
        side.wait_stream(torch.cuda.current_stream())
        got = call(side)
        assert not held & {t.data_ptr() for t in got}
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@gpu
def test_bindings_refuse(gpu_lib):
    import torch
    k = pool_of(4, 16, 2, 64)
    c = swm.PagedCache(k, k.clone(), ints([[0, 1], [2, -1]]), ints([3, 4]))
    n, free, count = ints([1, 1]), ints([3, 0, 0, 0]), ints([1])
    for bad in (n.long(), n.cpu(), [1, 1]):
        with pytest.raises(TypeError):
            swm.kv_reserve(c, bad, free, count, 2)
    for bad in (n[:1], ints([1, 0, 1, 0])[::2]):
        with pytest.raises(ValueError):
            swm.kv_reserve(c, bad, free, count, 2)
    with pytest.raises(TypeError):
        swm.kv_reserve(c, n, free.view(2, 2), count, 2)
    with pytest.raises(ValueError):
        swm.kv_reserve(c, n, free, free, 2)
    with pytest.raises(ValueError):
        swm.kv_reserve(c, n, free, count, -1)
    with pytest.raises(TypeError):
        swm.kv_reserve(c, n, free, count, 2, slots=ints([0, 0]))
    with pytest.raises(ValueError):
        swm.kv_reserve(c, n, free, count, 2, starts=ints([0, 0]))
    with pytest.raises(swm.SwmError, match="SHAPE"):  # no place for every page
        swm.kv_reserve(c, n, free[:3], count, 2)
    with pytest.raises(swm.SwmError, match="INVALID"):
        swm.kv_reserve(c, n, free, count, 2, granted=n)
    x, slots = torch.zeros((2, 2, 64), dtype=torch.float16, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda")
    for bad in (x.float(), x[0], x.cpu()):
        with pytest.raises(TypeError):
            swm.kv_append(c, bad, x, slots)
    for a, b in ((x[:, :1], x[:, :1]), (x, x[:1]), (x[..., :32], x[..., :32])):
        with pytest.raises(ValueError):
            swm.kv_append(c, a, b, slots)
    with pytest.raises(TypeError):
        swm.kv_append(c, x, x, ints([0, 1]))
    with pytest.raises(ValueError):
        swm.kv_append(c, x, x, slots[:1])
    with pytest.raises(ValueError):
        swm.kv_append(c, x, x, slots, positions=ints(np.zeros((4, 2, 16))))
    with pytest.raises(TypeError):
        swm.kv_append(c, x, x, slots, weights=ints(np.zeros((4, 2, 16))))
    with pytest.raises(swm.SwmError, match="INVALID"):  # entries that heads share
        swm.kv_append(c, x, x, slots, weights=torch.zeros((4, 1, 16), device="cuda").expand(4, 2, 16))
    shared = swm.PagedCache(k[:, :, :1].expand(4, 16, 2, 64), k, ints([[0]]), ints([0]))
    with pytest.raises(swm.SwmError, match="INVALID"):  # rows that heads share
        swm.kv_append(shared, x, x, slots)


def cache_struct(**kw):
    f = dict(k=4096, v=4096, table=4096, lengths=8192, k_page=1024, k_slot=64, k_head=64, v_page=1024, v_slot=64,
             v_head=64, table_ld=4, pages=8, page_size=16, heads=1, dim=64, batch=2, pages_per_seq=4)
    f.update(kw)
    return swm.KvCache(**f)


@pytest.mark.parametrize("change,code", [
    (dict(counts=None), 1), (dict(free=None), 1), (dict(free_count=None), 1), (dict(starts=None), 1),
    (dict(slots=None), 1), (dict(granted=None), 1), (dict(free_size=-1), 1), (dict(tokens=-1), 1),
    (dict(free_size=7), 2), (dict(free_size=1 << 31), 8), (dict(tokens=1 << 31), 8), (dict(granted=12288), 1),
    (dict(granted=8192), 1), (dict(counts=8192), 1), (dict(starts=12288), 1), (dict(starts=8192), 1),
    (dict(starts=28672), 1),
])
def test_reserve_refusals(change, code):
    a = dict(counts=12288, free=16384, free_size=8, free_count=20480, tokens=3, starts=24576, slots=32768,
             granted=28672, stream=None)
    a.update(change)
    assert swm.load().swm_kv_reserve(ctypes.addressof(cache_struct()), *a.values()) == code
    assert swm.load().swm_kv_reserve(None, *a.values()) == 1


# (address, bytes) of every argument's memory: two sequences, rows of three pages and an entry between them,
# eight free pages, three added tokens
SPANS = dict(table=(4096, 28), lengths=(8192, 8), counts=(12288, 8), free=(16384, 32), free_count=(20480, 4),
             starts=(24576, 12), slots=(32768, 24), granted=(28672, 8))


def reserve_at(tokens=3, **at):
    """Status of a call with some arguments at other addresses."""
    a = {name: at.get(name, SPANS[name][0]) for name in SPANS}
    cache = cache_struct(table=a["table"], lengths=a["lengths"], table_ld=4, pages_per_seq=3)
    return swm.load().swm_kv_reserve(ctypes.addressof(cache), a["counts"], a["free"], 8, a["free_count"], tokens,
                                     a["starts"], a["slots"], a["granted"], None)


@pytest.mark.parametrize("one", SPANS)
@pytest.mark.parametrize("two", SPANS)
def test_reserve_refuses_memory_that_is_shared(one, two):
    """All but counts is written: no two of the arguments may have an entry in common, in whole or in part."""
    if one == two:
        return
    at, n = SPANS[one]
    assert reserve_at(**{two: at}) == 1                              # the same address
    assert reserve_at(**{two: at + n - 4}) == 1                      # from its last entry on
    assert reserve_at(**{two: at + 4 - SPANS[two][1]}) == 1          # up to its first entry


def test_reserve_refuses_entries_of_any_table_row():
    for one in SPANS:
        if one != "table":
            assert reserve_at(**{one: 4096 + 16 + 8}) == 1           # the second sequence's last page


@pytest.mark.gpu
def test_reserve_between_the_rows_of_a_table(gpu_lib):
    """Arguments side by side in one buffer share nothing, the number of free pages in a column that the table's
    rows leave out among them."""
    import torch
    y = torch.zeros(64, dtype=torch.int32, device="cuda")
    table, lengths, counts, free, starts, granted = (y[:8].view(2, 4)[:, :3], y[8:10], y[10:12], y[12:20], y[20:23],
                                                     y[23:25])
    table.fill_(-1)
    count = y[3:4]
    count.fill_(8)
    counts.copy_(ints([17, 1]))
    free.copy_(ints(range(8)))
    slots = torch.zeros(18, dtype=torch.int64, device="cuda")
    k = pool_of(8, 16)
    c = swm.PagedCache(k, k, table, lengths)
    swm.kv_reserve(c, counts, free, count, 18, starts=starts, slots=slots, granted=granted)
    assert table.tolist() == [[7, 6, -1], [5, -1, -1]] and lengths.tolist() == [17, 1] and count.tolist() == [5]
    assert starts.tolist() == [0, 17, 18] and granted.tolist() == [17, 1]
    assert slots.tolist() == list(range(7 * 16, 8 * 16)) + [6 * 16, 5 * 16]
    counts.fill_(0)
    swm.kv_reserve(c, counts, free, count, 0, starts=starts, slots=slots[:0], granted=granted)
    assert granted.tolist() == [0, 0] and lengths.tolist() == [17, 1]
    for bad in (dict(starts=starts, granted=starts[:2]), dict(starts=starts, granted=starts[1:]),
                dict(starts=free[5:]), dict(granted=table[0, :2])):
        with pytest.raises(swm.SwmError, match="INVALID"):
            swm.kv_reserve(c, counts, free, count, 0, **bad)
    with pytest.raises(swm.SwmError, match="INVALID"):
        swm.kv_reserve(c, counts, free, free[7:], 0)


@pytest.mark.parametrize("fields,code", [
    (dict(batch=-1), 1), (dict(table=None), 1), (dict(lengths=None), 1), (dict(table_ld=3), 1), (dict(pages=0), 1),
    (dict(dim=60), 8), (dict(page_size=1 << 30), 8), (dict(k=4104), 3),
])
def test_reserve_refuses_caches(fields, code):
    assert swm.load().swm_kv_reserve(ctypes.addressof(cache_struct(**fields)), 12288, 16384, 8, 20480, 3, 24576, 32768,
                                     28672, None) == code


@pytest.mark.parametrize("change,code", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(slots=None), 1), (dict(tokens=-1), 1), (dict(k_token=-8), 1),
    (dict(v_head=-8), 1), (dict(weights=4096, w_page=-1), 1), (dict(weights=4096, w_page=8), 1),
    (dict(positions=4096, p_page=16), 1), (dict(positions=4096, p_page=16, p_head=-1, at=4096), 1),
    (dict(positions=4096, p_page=15, at=4096), 1), (dict(k=4104), 3), (dict(v_token=4), 3), (dict(k_head=12), 3),
    (dict(tokens=1 << 31), 8), (dict(tokens=(1 << 31) - 70000), 8), (dict(tokens=0, k=None), 0),
])
def test_append_refusals(change, code):
    a = dict(k=4096, k_token=64, k_head=64, v=4096, v_token=64, v_head=64, tokens=2, slots=4096, weights=None, w_page=0,
             w_head=0, positions=None, p_page=0, p_head=0, at=None, stream=None)
    a.update(change)
    # heads of their own pages of the pool: 8 pages of 16 slots
    cache = cache_struct(heads=64, k_slot=64 * 64, k_page=16 * 64 * 64, v_slot=64 * 64, v_page=16 * 64 * 64)
    if "w_page" in change or "p_page" in change:
        cache = cache_struct()
    assert swm.load().swm_kv_append(ctypes.addressof(cache), *a.values()) == code
    assert swm.load().swm_kv_append(None, *a.values()) == 1


@pytest.mark.parametrize("fields", [dict(heads=2, k_head=0), dict(heads=2, v_head=32), dict(k_page=32),
                                    dict(v_slot=0), dict(heads=2, k_head=64, k_slot=64)])
def test_append_refuses_rows_that_share_memory(fields):
    assert swm.load().swm_kv_append(ctypes.addressof(cache_struct(**fields)), 4096, 64, 64, 4096, 64, 64, 2, 4096, None,
                                    0, 0, None, 0, 0, None, None) == 1
