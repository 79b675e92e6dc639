"""tree_attention against softmax attention in 64 bits, and its refusals.
Tolerances as derived in test_prompt_attention, with a rounding for each of the
pieces that a sequence may be cut into (within its 2^-19)."""
import ctypes

import numpy as np
import pytest

import sparse_weight_matmul_amd as swm
from test_prompt_attention import attend, bounds, check, ints

gpu = pytest.mark.gpu


def sees_of(n, t, parents, live):
    """(t, n) bool: what each drafted token sees, by walking up its parents."""
    out = np.zeros((t, n), bool)
    for i in range(t):
        out[i, :max(n - t, 0)] = True
        j = i
        while True:
            if n - t + j >= 0:
                out[i, n - t + j] = True
            up = parents[j]
            if up < 0 or up >= j:
                break
            j = up
    return out & live


def reference(q, k, v, table, lengths, starts, parents, scale, mask=None, most=64):
    """(out, bound, rows written) for host arrays."""
    T, Hq, D = q.shape
    P, S, Hkv, _ = k.shape
    cap = table.shape[1] * S
    out, tol, rows = np.zeros((T, Hq, D)), np.zeros((T, Hq, D)), np.zeros(T, bool)
    for b in range(len(lengths)):
        n, a = min(max(int(lengths[b]), 0), cap), starts[b]
        t = min(starts[b + 1] - a, most)
        rows[a:a + t] = True
        tok = np.arange(n)
        page = table[b][tok // S]
        live = (page >= 0) & (page < P)
        if mask is not None:
            live &= mask[b][:n] != 0
        up = np.arange(t) - 1 if parents is None else parents[a:a + t]
        sees = sees_of(n, t, up, live)
        page = np.where(live, page, 0)
        for h in range(Hq if t else 0):
            K, V = (np.where(live[:, None], x[page, tok % S, h // (Hq // Hkv)], 0) for x in (k, v))
            out[a:a + t, h], tol[a:a + t, h] = attend(q[a:a + t, h], K, V, scale, sees)
    return out, tol, rows


def make(Hq, Hkv, D, S, lengths, drafts, layout="token", kind="tree", seed=0, extra=3):
    """Host arrays and device tensors; spare pages and slots past the lengths hold the worst of values."""
    import torch
    r = np.random.default_rng([seed, Hq, D, S, sum(lengths), sum(drafts)])
    need = [-(-max(n, 0) // S) for n in lengths]
    per, P = max(max(need), 1) + 1, sum(need) + extra
    k, v = (r.standard_normal((P, S, Hkv, D)).astype(np.float16) for _ in range(2))
    T = sum(drafts)
    q = (2 * r.standard_normal((T, Hq, D))).astype(np.float16)
    pages, table, at = r.permutation(P), np.full((len(lengths), per), -1, np.int32), 0
    for b, n in enumerate(lengths):
        table[b, :need[b]] = pages[at:at + need[b]]
        at += need[b]
        if need[b]:
            last = table[b, need[b] - 1]
            k[last, n - (need[b] - 1) * S:], v[last, n - (need[b] - 1) * S:] = np.nan, np.inf
    k[pages[at:]], v[pages[at:]] = np.nan, np.nan
    parents = None
    if kind == "tree":
        parents = np.concatenate([[r.integers(-1, i) if i else -1 for i in range(t)] for t in drafts] or [[]])
        parents = parents.astype(np.int32)
    elif kind == "star":  # all of them children of the first
        parents = np.concatenate([[-1] + [0] * (t - 1) for t in drafts if t]).astype(np.int32)

    def pool(x):
        x = torch.from_numpy(x)
        return x.cuda() if layout == "token" else x.transpose(1, 2).contiguous().cuda().transpose(1, 2)

    dev = {"q": torch.from_numpy(q).cuda(), "k": pool(k), "v": pool(v), "table": ints(table),
           "lengths": ints(lengths), "starts": ints(bounds(drafts)),
           "parents": None if parents is None else ints(parents)}
    return q, k, v, table, parents, dev


def cache_of(dev):
    return swm.PagedCache(dev["k"], dev["v"], dev["table"], dev["lengths"])


CASES = [
    # Hq, Hkv, D, S, lengths, drafts, layout, kind
    (1, 1, 64, 16, [1], [1], "token", "tree"),
    (4, 4, 128, 16, [137], [25], "token", "tree"),
    (4, 4, 128, 16, [64, 65, 128, 1], [64, 1, 33, 1], "head", "tree"),
    (8, 2, 128, 32, [31, 200, 0, 127], [7, 20, 0, 32], "token", "tree"),
    (6, 2, 80, 24, [100, 257], [5, 64], "head", "chain"),
    (5, 1, 96, 8, [640, 77], [13, 9], "token", "star"),
    (16, 1, 64, 64, [1000, 20], [16, 20], "head", "tree"),
    (34, 2, 128, 16, [300], [3], "token", "tree"),
    (40, 1, 64, 16, [1500], [31], "token", "chain"),
    (6, 3, 256, 16, [513, 40], [40, 2], "token", "tree"),
    (4, 2, 136, 40, [90, 200], [64, 63], "head", "tree"),
    (4, 2, 192, 16, [300], [8], "token", "tree"),
    (3, 3, 8, 16, [64, 200], [4, 64], "token", "tree"),
    (4, 4, 40, 1, [19, 260], [19, 11], "token", "tree"),
    (4, 2, 128, 5, [131, 12], [6, 12], "head", "tree"),
    (2, 2, 200, 100, [350], [50], "token", "chain"),
    (8, 1, 128, 128, [9001], [64], "head", "tree"),
    (2, 2, 64, 20, [9000, 4097], [3, 4], "token", "tree"),
    (64, 8, 128, 16, [700], [64], "token", "tree"),
    (4, 4, 64, 16, [(37 * b) % 700 + 9 for b in range(130)], [b % 10 for b in range(130)], "token", "tree"),
]


@gpu
@pytest.mark.parametrize("Hq,Hkv,D,S,lengths,drafts,layout,kind", CASES)
@pytest.mark.parametrize("masked", [False, True])
def test_against_64_bits(gpu_lib, Hq, Hkv, D, S, lengths, drafts, layout, kind, masked):
    import torch
    q, k, v, table, parents, dev = make(Hq, Hkv, D, S, lengths, drafts, layout, kind)
    cap = table.shape[1] * S
    r = np.random.default_rng(7)
    mask = dmask = None
    if masked:
        mask = r.random((len(lengths), cap + 3)) < 0.7  # rows longer than the capacity
        mask[0] = False                                 # rows that the mask leaves empty
        for b, n in enumerate(lengths):                 # masked tokens of the worst kind
            t = np.arange(n)[~mask[b, :n]]
            k[table[b][t // S], t % S], v[table[b][t // S], t % S] = np.nan, np.inf
        dev["k"].copy_(torch.from_numpy(k))
        dev["v"].copy_(torch.from_numpy(v))
        dmask = torch.from_numpy(mask).cuda()
    starts = bounds(drafts)
    out = torch.full(dev["q"].shape, 7.0, dtype=torch.float16, device="cuda")
    swm.tree_attention(cache_of(dev), dev["q"], dev["starts"], dev["parents"], mask=dmask, out=out)
    ref, tol, rows = reference(q, k, v, table, lengths, starts, parents, D ** -0.5, mask)
    assert rows.all()
    check(out, ref, tol)
    if masked:
        assert bool((out[: drafts[0]] == 0).all())
    most = max(drafts)
    again = swm.tree_attention(cache_of(dev), dev["q"], dev["starts"], dev["parents"], max_tokens=most, mask=dmask)
    check(again, ref, tol)


@gpu
@pytest.mark.parametrize("lengths", [[200, 90], [5000, 3000]])
def test_one_drafted_token_is_paged_attention(gpu_lib, lengths):
    """The two calls round their weights differently: each is within its own bound of the definition."""
    q, k, v, table, parents, dev = make(8, 2, 128, 16, lengths, [1, 1])
    c = cache_of(dev)
    out = swm.tree_attention(c, dev["q"], dev["starts"], dev["parents"])
    one = swm.paged_attention(c, dev["q"])
    ref, tol, _ = reference(q, k, v, table, lengths, [0, 1, 2], parents, 128 ** -0.5)
    check(out, ref, tol)
    check(one, ref, tol)


@gpu
@pytest.mark.parametrize("Hq,Hkv,lengths,drafts", [(2, 1, [300, 90], [20, 30]), (16, 2, [6000, 40], [64, 40])])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_what_is_not_finite_stays_with_its_readers(gpu_lib, Hq, Hkv, lengths, drafts, bad):
    """A drafted token's value that is no number reaches the rows below it in the tree and no other."""
    q, k, v, table, parents, dev = make(Hq, Hkv, 64, 16, lengths, drafts)
    n, t, G = lengths[0], drafts[0], Hq // Hkv
    for j in (0, 3, t - 1):
        at = n - t + j
        page, slot = int(table[0, at // 16]), at % 16
        keep = dev["v"][page, slot, 0, 17].clone()
        dev["v"][page, slot, 0, 17] = bad
        out = swm.tree_attention(cache_of(dev), dev["q"], dev["starts"], dev["parents"]).double().cpu().numpy()
        hit = np.zeros(out.shape, bool)
        hit[:t, :G, 17] = sees_of(n, t, parents[:t], True)[:, at][:, None]
        assert np.array_equal(~np.isfinite(out), hit)
        ref, tol, _ = reference(q, k, v, table, lengths, bounds(drafts), parents, 0.125)
        assert np.all(np.abs(out - ref)[~hit] <= tol[~hit])
        dev["v"][page, slot, 0, 17] = keep
        key = dev["k"][page, slot, 0].clone()
        dev["k"][page, slot, 0] = float("nan")
        out = swm.tree_attention(cache_of(dev), dev["q"], dev["starts"], dev["parents"]).double().cpu().numpy()
        hit[:t, :G] = sees_of(n, t, parents[:t], True)[:, at][:, None, None]
        assert np.array_equal(np.isnan(out), hit)
        dev["k"][page, slot, 0] = key
    page, slot = int(table[0, 1]), 5  # a token that all rows see
    dev["v"][page, slot, 0, 9] = bad
    out = swm.tree_attention(cache_of(dev), dev["q"], dev["starts"], dev["parents"]).double().cpu().numpy()
    hit = np.zeros(out.shape, bool)
    hit[:t, :G, 9] = True
    assert np.array_equal(~np.isfinite(out), hit)


@gpu
@pytest.mark.parametrize("D,lengths", [(64, [4000]), (128, [700]), (256, [900])])
@pytest.mark.parametrize("gap", [2.0, 17.0, 40.0])
def test_one_token_far_above_the_others(gpu_lib, D, lengths, gap):
    import torch
    q, k, v, table, parents, dev = make(2, 1, D, 16, lengths, [12])
    q[:], k[:] = 1, 0
    k[table[0, 0], 0] = np.float16(gap) / np.float16(D ** 0.5)
    v[:] = np.abs(np.nan_to_num(v, posinf=1.0)) + np.float16(0.25)
    v[table[0, 0], 0] = 0
    for name, x in (("q", q), ("k", k), ("v", v)):
        dev[name].copy_(torch.from_numpy(x))
    out = swm.tree_attention(cache_of(dev), dev["q"], dev["starts"], dev["parents"])
    ref, tol, _ = reference(q, k, v, table, lengths, [0, 12], parents, D ** -0.5)
    check(out, ref, tol)


@gpu
def test_lengths_tables_and_parents_of_any_content(gpu_lib):
    """Lengths past the capacity or below the drafted tokens, entries outside the pool, parents that are none."""
    q, k, v, table, parents, dev = make(4, 2, 64, 16, [100, 60, 40], [10, 12, 8])
    table[0, 1], table[1, 0], table[0, 6] = k.shape[0], -7, 0
    lengths = [1000, 60, 3]  # the third counts three of its eight drafted tokens
    parents[:] = [-1, 0, 5, 2, -9, 4, 6, 3, 1 << 30, 7, -1, 0, 1, 1, 2, 2, 9, 16, 12, 8, 9, 30, -1, 0, 1, 2, 3, 4, 5, 6]
    dev["table"].copy_(ints(table))
    dev["lengths"].copy_(ints(lengths))
    dev["parents"].copy_(ints(parents))
    cap = table.shape[1] * 16
    page0 = table[0, -1] = table[0, 0]  # the capacity's last page is a page of the pool
    dev["table"].copy_(ints(table))
    k[page0], v[page0] = np.nan_to_num(k[page0]), np.nan_to_num(v[page0])
    live = np.isfinite(k).all((2, 3)) & np.isfinite(v).all((2, 3))
    mask = np.zeros((3, cap), bool)  # only rows that hold numbers count
    for b in range(3):
        for t in range(cap):
            p = table[b, t // 16]
            mask[b, t] = 0 <= p < k.shape[0] and live[p, t % 16]
    import torch
    out = swm.tree_attention(cache_of(dev), dev["q"], dev["starts"], dev["parents"],
                             mask=torch.from_numpy(mask).cuda())
    ref, tol, _ = reference(q, k, v, table, lengths, bounds([10, 12, 8]), parents, 0.125, mask)
    check(out, ref, tol)


@gpu
def test_rows_of_no_sequence_are_left(gpu_lib):
    import torch
    q, k, v, table, parents, dev = make(4, 2, 64, 16, [2000, 300], [30, 20])
    starts = ints([5, 25, 40])
    out = torch.full_like(dev["q"], 7.0)
    swm.tree_attention(cache_of(dev), dev["q"], starts, dev["parents"], max_tokens=12, out=out)
    ref, tol, rows = reference(q, k, v, table, [2000, 300], [5, 25, 40], parents, 0.125, most=12)
    # of a sequence with more rows than max_tokens the first ones count, as its last tokens
    check(out[5:17], ref[5:17], tol[5:17])
    check(out[25:37], ref[25:37], tol[25:37])
    assert bool((out[torch.from_numpy(~rows).cuda()] == 7.0).all())


@gpu
def test_strided_operands_stream_and_scale(gpu_lib):
    import torch
    q, k, v, table, parents, dev = make(4, 2, 80, 16, [900, 33], [9, 33])
    wide = torch.zeros((42, 12, 80), dtype=torch.float16, device="cuda")
    wide[:, 4:8] = dev["q"]
    big = torch.full((42, 6, 96), 5.0, dtype=torch.float16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = swm.tree_attention(cache_of(dev), wide[:, 4:8], dev["starts"], dev["parents"], scale=-0.2,
                             out=big[:, 1:5, :80], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    ref, tol, _ = reference(q, k, v, table, [900, 33], bounds([9, 33]), parents, -0.2)
    check(got, ref, tol)
    assert bool((big[:, 0] == 5).all()) and bool((big[:, 5] == 5).all()) and bool((big[:, :, 80:] == 5).all())
    zero = swm.tree_attention(cache_of(dev), dev["q"], dev["starts"], dev["parents"], scale=0.0)
    ref, tol, _ = reference(q, k, v, table, [900, 33], bounds([9, 33]), parents, 0.0)
    check(zero, ref, tol)


@gpu
@pytest.mark.parametrize("Hq,Hkv,drafts", [(4, 2, [20, 8]), (16, 1, [64, 33]), (2, 1, [8, 15])])
def test_graph_follows_everything_in_device_memory(gpu_lib, Hq, Hkv, drafts):
    import torch
    lengths = [3000, 2500]
    q, k, v, table, parents, dev = make(Hq, Hkv, 64, 16, lengths, drafts)
    c, most = cache_of(dev), max(drafts)
    ws = torch.empty(c.tree_workspace_bytes(Hq, most), dtype=torch.uint8, device="cuda")
    other = torch.empty_like(ws)
    assert ws.numel() > 0
    outs = [torch.zeros_like(dev["q"]) for _ in range(2)]

    def call(i, w):
        swm.tree_attention(c, dev["q"], dev["starts"], dev["parents"], max_tokens=most, out=outs[i], workspace=w)
    call(0, ws)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i, w in enumerate((ws, other)):  # a workspace of its own each: they run at the same time
        with torch.cuda.graph(graphs[i]):
            call(i, w)
    side = torch.cuda.Stream()
    for n in ([100, 2500], [3000, 64], [1234, 777], [3000, 2500]):
        dev["lengths"].copy_(ints(n))
        starts = bounds(drafts) if n[0] != 1234 else np.array([0, 3, 3 + drafts[1]], np.int32)
        dev["starts"].copy_(ints(starts))
        side.wait_stream(torch.cuda.current_stream())
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.current_stream().wait_stream(side)
        eager = swm.tree_attention(c, dev["q"], dev["starts"], dev["parents"], max_tokens=most)
        torch.cuda.synchronize()
        ref, tol, rows = reference(q, k, v, table, n, starts, parents, 0.125)
        rows_d = torch.from_numpy(rows).cuda()
        for o in outs:
            assert torch.equal(o[rows_d], eager[rows_d])
            check(o[rows_d], ref[rows], tol[rows], str(n))


@gpu
def test_offsets_past_32_bits(gpu_lib):
    """A head-major pool of 6 GiB, its last pages in use."""
    import torch
    P, S, H, D = 13000, 128, 2, 128
    k = torch.zeros((P, H, S, D), dtype=torch.float16, device="cuda").transpose(1, 2)
    r = np.random.default_rng(2)
    table = np.array([[P - 1, 3, P - 2], [P - 4, P - 3, 7]], np.int32)
    n, t = [300, 290], [5, 9]
    hk, hv = np.zeros((P, 1, 1, 1), np.float16), None
    rows = {}
    for p in table.ravel():
        rows[p] = [r.standard_normal((S, H, D)).astype(np.float16) for _ in range(2)]
    v = torch.empty_like(k)
    for p, (a, b) in rows.items():
        k[int(p)], v[int(p)] = torch.from_numpy(a).cuda(), torch.from_numpy(b).cuda()
    q = r.standard_normal((14, 4, D)).astype(np.float16)
    c = swm.PagedCache(k, v, ints(table), ints(n))
    out = swm.tree_attention(c, torch.from_numpy(q).cuda(), ints([0, 5, 14]))
    small = {p: i for i, p in enumerate(rows)}
    hk, hv = (np.stack([rows[p][i] for p in rows]) for i in range(2))
    ref, tol, _ = reference(q, hk, hv, np.vectorize(small.get)(table), n, [0, 5, 14], None, D ** -0.5)
    check(out, ref, tol)


@gpu
@pytest.mark.parametrize("Hq", [2, 16, 64])  # few query rows, many, more than 128
def test_lengths_next_to_2_31(gpu_lib, Hq):
    """One page of a thousand million slots and a table of two: the tokens that count are the last ones."""
    import torch
    S, D, t = (1 << 30) - 40000, 8, 9
    n = 2 * S - 5
    k = torch.zeros((1, S, 1, D), dtype=torch.float16, device="cuda")
    r = np.random.default_rng(3)
    hk = r.standard_normal((2, 300, D)).astype(np.float16)
    k[0, S - 305:S - 5, 0] = torch.from_numpy(hk[0]).cuda()
    v = torch.zeros_like(k)
    v[0, S - 305:S - 5, 0] = torch.from_numpy(hk[1]).cuda()
    mask = torch.zeros((1, 2 * S), dtype=torch.bool, device="cuda")
    mask[0, n - 300:] = True  # of the second time that the page comes
    c = swm.PagedCache(k, v, ints([[0, 0]]), ints([n]))
    q = r.standard_normal((t, Hq, D)).astype(np.float16)
    out = swm.tree_attention(c, torch.from_numpy(q).cuda(), ints([0, t]), max_tokens=t, mask=mask)
    sees = np.tril(np.ones((t, 300), bool), 300 - t)
    for h in range(Hq):
        ref, tol = attend(q[:, h], hk[0], hk[1], D ** -0.5, sees)
        check(out[:, h], ref, tol)


def against_shared_heads(G, Hkv, D, S, lengths, drafts, masked, pieces=None):
    """Many key-value heads over one head's rows, so that there is work for the whole device and one head to check
    against 64 bits; the others have to be equal to it.  pieces: of a sequence at most, None: sequences are whole."""
    import torch
    q, k, v, table, parents, dev = make(G, 1, D, S, lengths, drafts)
    cap = table.shape[1] * S
    r = np.random.default_rng(11)
    mask = dmask = None
    if masked:
        mask = r.random((len(lengths), cap)) < 0.8
        for b, n in enumerate(lengths):
            mask[b, n // 3:n // 3 + 200] = False  # whole tiles, whole loads, and the ends of both
            mask[b, n // 2:n // 2 + 24] = False
            table[b, n // 2 // S + 3] = -1 if b % 2 else k.shape[0]
            t = np.arange(n)[~mask[b, :n]]
            page = table[b][t // S]
            on = (page >= 0) & (page < k.shape[0])
            k[page[on], t[on] % S], v[page[on], t[on] % S] = np.nan, np.inf
        for name, x in (("k", k), ("v", v), ("table", table), ("mask", mask)):
            dev[name] = torch.from_numpy(x).cuda()
        dmask = dev["mask"]
    c = swm.PagedCache(*(dev[x].expand(-1, -1, Hkv, -1) for x in "kv"), dev["table"], dev["lengths"])
    most = max(drafts)
    # the workspace holds D + 2 words for every piece, key-value head and row, rows up to the next 256
    room = c.tree_workspace_bytes(G * Hkv, most) // (4 * (D + 2) * Hkv * -(-G * most // 256) * 256)
    assert room == (pieces or 0) * len(lengths)
    out = torch.full((sum(drafts), G * Hkv, D), 7.0, dtype=torch.float16, device="cuda")
    swm.tree_attention(c, dev["q"].repeat(1, Hkv, 1), dev["starts"], dev["parents"], max_tokens=most, mask=dmask,
                       out=out)
    ref, tol, rows = reference(q, k, v, table, lengths, bounds(drafts), parents, D ** -0.5, mask)
    assert rows.all()
    out = out.view(-1, Hkv, G, D)
    check(out[:, 0], ref, tol)
    assert torch.equal(out, out[:, :1].expand_as(out))


@gpu
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("G,Hkv,D,S,lengths,drafts,pieces", [
    (3, 256, 128, 16, [1700, 901], [43, 43], None),        # a workgroup's whole sequence, 14 to 26 tiles of 64
    (3, 256, 80, 16, [1500, 1023], [64, 50], None),
    (5, 128, 96, 5, [1301, 1100, 1000], [60, 40, 64], None),  # rows of a load on several pages
    (3, 256, 128, 5, [64 * 14 + 1, 64 * 20], [43, 50], None),
    (4, 512, 72, 4, [2000], [64], None),
    (9, 64, 128, 16, [16 * 900], [20], 4),                 # pieces of 3600 tokens
    (3, 64, 104, 3, [9001], [43], 4),
])
def test_more_than_128_rows_over_many_tiles(gpu_lib, G, Hkv, D, S, lengths, drafts, pieces, masked):
    """Tiles come into places that were read before, entries of the table into places that were used: twice and more."""
    assert 64 < D <= 128 and G * max(drafts) > 128 and min(lengths) // (pieces or 1) >= 13 * 64
    against_shared_heads(G, Hkv, D, S, lengths, drafts, masked, pieces)


def unlike(B, most, drafts):
    """Lengths and drafted tokens of a batch: long, short, equal ones, empty ones, some with nothing drafted."""
    n = [(most, 700, 300, 300, 64, 17, 1, 0)[b % 8] + (b % 3 if b % 8 < 3 else 0) for b in range(B)]
    if B > 2:
        n[1], n[2] = most, most
    t = [0 if b % 5 == 3 else 1 + b % drafts for b in range(B)]
    t[0] = drafts
    return n, t


@gpu
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("G,Hkv,D,S,B,drafts", [
    (1, 32, 128, 16, 17, 8),    # up to 32 rows
    (2, 16, 128, 5, 33, 16),
    (1, 4, 128, 16, 128, 8),
    (4, 8, 64, 16, 128, 8),
    (1, 256, 200, 16, 2, 20),
    (2, 8, 128, 16, 128, 31),   # up to 128
    (3, 32, 64, 8, 33, 40),
    (1, 512, 256, 16, 3, 40),
    (4, 4, 128, 16, 128, 40),   # more
    (5, 33, 96, 5, 31, 64),
])
def test_whole_sequences_by_their_lengths(gpu_lib, G, Hkv, D, S, B, drafts, masked):
    """More workgroups than places, sequences of unlike lengths: each is done once, whatever the order."""
    lengths, t = unlike(B, 1500, drafts)
    against_shared_heads(G, Hkv, D, S, lengths, t, masked)


@gpu
def test_equal_lengths_by_their_order(gpu_lib):
    against_shared_heads(1, 8, 128, 16, [1100] * 128, [2] * 128, False)
    against_shared_heads(1, 32, 128, 16, [0] * 16 + [1100], [2] * 17, False)


@gpu
def test_as_many_sequences_as_there_may_be(gpu_lib):
    """65535 of one or two tokens on a page each, of which every other one drafts its last."""
    import torch
    B, D = 65535, 8
    r = np.random.default_rng(6)
    k, v = (r.standard_normal((B, 2, 1, D)).astype(np.float16) for _ in range(2))
    q = r.standard_normal(((B + 1) // 2, 2, D)).astype(np.float16)
    n = 1 + np.arange(B) // 2 % 2
    starts = bounds(np.arange(B) % 2 == 0)
    c = swm.PagedCache(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), ints(np.arange(B)[::-1].reshape(B, 1).copy()),
                       ints(n))
    out = swm.tree_attention(c, torch.from_numpy(q).cuda(), ints(starts), max_tokens=1)
    at, page = np.arange(0, B, 2), B - 1 - np.arange(0, B, 2)
    one = n[at] == 1
    assert np.array_equal(out.cpu().numpy()[one], np.broadcast_to(v[page[one], :1, 0], (int(one.sum()), 2, D)))
    x = np.einsum("bhd,btd->bht", q[~one].astype(np.float64), k[page[~one], :, 0].astype(np.float64)) * D ** -0.5
    p = np.exp(x - x.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    V = v[page[~one], :, 0].astype(np.float64)
    want = np.einsum("bht,btd->bhd", p, V)
    # as derived in test_prompt_attention, sum |q_d k_d| below 40 here: a score's error is below 2^-17, twice, and the
    # roundings of the weights and the sums
    tol = (2.0**-16 + 2.0**-19 + 2.0**-11 + 2.0**-17) * np.einsum("bht,btd->bhd", p, np.abs(V)) + \
        2.0**-10 * np.abs(want) + 2.0**-25
    check(out[torch.from_numpy(~one).cuda()], want, tol)


@gpu
def test_nothing_to_do(gpu_lib):
    import torch
    q, k, v, table, parents, dev = make(4, 2, 64, 16, [40, 30], [4, 4])
    c = cache_of(dev)
    assert swm.tree_attention(c, dev["q"][:0], ints([0, 0, 0])).shape == (0, 4, 64)
    out = torch.full_like(dev["q"], 2.0)
    swm.tree_attention(c, dev["q"], ints([3, 3, 3]), out=out)
    swm.tree_attention(c, dev["q"], dev["starts"], max_tokens=0, out=out)
    assert bool((out == 2.0).all())
    none = swm.PagedCache(dev["k"], dev["v"], dev["table"][:0], dev["lengths"][:0])
    swm.tree_attention(none, dev["q"], ints([0]), out=out)
    assert bool((out == 2.0).all())
    nowhere = swm.PagedCache(dev["k"], dev["v"], dev["table"][:, :0], dev["lengths"])
    assert bool((swm.tree_attention(nowhere, dev["q"], dev["starts"]) == 0).all())


@gpu
def test_binding_refuses(gpu_lib):
    import torch
    q, k, v, table, parents, dev = make(4, 2, 64, 16, [20, 3000], [4, 6])
    c, s = cache_of(dev), dev["starts"]
    for bad in (dev["q"].float(), dev["q"][0], dev["q"].cpu()):
        with pytest.raises(TypeError):
            swm.tree_attention(c, bad, s)
    with pytest.raises(ValueError):
        swm.tree_attention(c, dev["q"][..., :32], s)
    for bad in (s.long(), s.cpu()):
        with pytest.raises(TypeError):
            swm.tree_attention(c, dev["q"], bad)
    for bad in (s[:2], ints([0, 0, 4, 4, 10, 10])[::2]):
        with pytest.raises(ValueError):
            swm.tree_attention(c, dev["q"], bad)
    with pytest.raises(TypeError):
        swm.tree_attention(c, dev["q"], s, dev["parents"].long())
    with pytest.raises(ValueError):
        swm.tree_attention(c, dev["q"], s, dev["parents"][:5])
    with pytest.raises(ValueError):
        swm.tree_attention(c, dev["q"], s, mask=torch.ones((2, 3), dtype=torch.bool, device="cuda"))
    with pytest.raises(ValueError):
        swm.tree_attention(c, dev["q"], s, out=torch.empty_like(dev["q"])[:4])
    with pytest.raises(swm.SwmError, match="UNSUPPORTED"):
        swm.tree_attention(c, dev["q"], s, max_tokens=65)
    with pytest.raises(swm.SwmError, match="INVALID"):
        swm.tree_attention(c, dev["q"], s, max_tokens=-1)
    with pytest.raises(swm.SwmError, match="INVALID"):  # three heads over two
        swm.tree_attention(c, dev["q"][:, :3], s)
    with pytest.raises(swm.SwmError, match="INVALID"):  # rows of out that share memory
        swm.tree_attention(c, dev["q"], s, out=torch.empty_like(dev["q"][:1]).expand(10, 4, 64))
    with pytest.raises(swm.SwmError, match="INVALID"):  # a workspace too small
        assert c.tree_workspace_bytes(4, 6) > 16
        swm.tree_attention(c, dev["q"], s, max_tokens=6, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))


@gpu
@pytest.mark.parametrize("bad", [[1, 2], 3, np.zeros((2, 64), np.int32)])
def test_what_is_no_tensor_is_a_type_error(gpu_lib, bad):
    q, k, v, table, parents, dev = make(4, 2, 64, 16, [20, 30], [4, 6])
    c = cache_of(dev)
    for name in ("parents", "mask", "out", "workspace"):
        with pytest.raises(TypeError):
            swm.tree_attention(c, dev["q"], dev["starts"], **{name: bad})
    with pytest.raises(TypeError):
        swm.tree_attention(c, dev["q"], bad)
    with pytest.raises(TypeError):
        swm.tree_attention(c, bad, dev["starts"])
    for name in ("mask", "weights", "workspace"):
        with pytest.raises(TypeError):
            swm.paged_attention(c, dev["q"][:2], **{name: bad})
    import torch
    slots, at = torch.zeros(2, dtype=torch.int64, device="cuda"), ints([0, 1])
    rows = dev["q"][:2, :2]
    for kw in (dict(weights=bad), dict(positions=bad, at=at), dict(positions=ints(np.zeros((dev["k"].shape[0], 2, 16))),
                                                                   at=bad)):
        with pytest.raises(TypeError):
            swm.kv_append(c, rows, rows, slots, **kw)
    with pytest.raises(TypeError):
        swm.kv_append(c, rows, rows, bad)


def cache_struct(**kw):
    f = dict(k=4096, v=4096, table=4096, lengths=4096, k_page=1024, k_slot=64, k_head=64, v_page=1024, v_slot=64,
             v_head=64, table_ld=4, pages=8, page_size=16, heads=1, dim=64, batch=2, pages_per_seq=4)
    f.update(kw)
    return swm.KvCache(**f)


def call(cache, **change):
    a = dict(q=4096, q_token=64, q_head=64, q_heads=1, tokens=8, starts=4096, parents=None, max_tokens=4, scale=0.125,
             mask=None, mask_ld=0, out=8192, out_token=64, out_head=64, ws=None, ws_bytes=0, stream=None)
    a.update(change)
    return swm.load().swm_tree_attention(cache and ctypes.addressof(cache), *a.values())


@pytest.mark.parametrize("fields,code", [
    (dict(k=None), 1), (dict(lengths=None), 1), (dict(table=None), 1), (dict(batch=-1), 1), (dict(pages=0), 1),
    (dict(k_slot=-64), 1), (dict(dim=60), 8), (dict(batch=65536), 8), (dict(page_size=1 << 30), 8), (dict(k=4104), 3),
    (dict(v_head=4), 3), (dict(k_slot=1 << 26), 8), (dict(v_slot=1 << 26), 8),
])
def test_cache_refusals(fields, code):
    assert call(cache_struct(**fields)) == code


@pytest.mark.parametrize("change,code", [
    (dict(q=None), 1), (dict(out=None), 1), (dict(starts=None), 1), (dict(q_heads=0), 1), (dict(scale=float("nan")), 1),
    (dict(tokens=-1), 1), (dict(max_tokens=-1), 1), (dict(q_token=-8), 1), (dict(out_head=-8), 1),
    (dict(mask=4096, mask_ld=63), 1), (dict(out_token=0), 1), (dict(out_token=63), 1), (dict(q=4104), 3),
    (dict(q_head=4), 3), (dict(max_tokens=65), 8), (dict(q_heads=65536), 8), (dict(tokens=(1 << 31) - 65536), 8),
    (dict(tokens=0, q=None), 0), (dict(max_tokens=0, q=None), 0),
])
def test_call_refusals(change, code):
    assert call(cache_struct(), **change) == code
    assert call(None, **change) == 1


def test_workspace_of_refused_sizes():
    lib = swm.load()
    for fields, heads, most in ((dict(heads=4), 6, 4), (dict(), 1, 65), (dict(), 1, 0), (dict(dim=60), 1, 4),
                                (dict(batch=0), 1, 4)):
        assert lib.swm_tree_attention_workspace_bytes(ctypes.addressof(cache_struct(**fields)), heads, most) == 0
