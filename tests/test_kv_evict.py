"""kv_evict against its definition on the host: everything it returns is a whole number or a copy, so all of it
is compared exactly."""
import ctypes

import numpy as np
import pytest

import sparse_weight_matmul_amd as swm

gpu = pytest.mark.gpu


def keep_of(w, pos, budget, recent):
    """Slots that stay, ascending, by the definition."""
    if not len(w):
        return np.zeros(0, int)
    first = (pos.astype(np.int64) > int(pos.max()) - recent) | np.isnan(w) | (w == np.inf)
    order = sorted(range(len(w)), key=lambda t: (0 if first[t] else 1, 0.0 if first[t] else -float(w[t]), t))
    return np.array(sorted(order[:budget]), int)


def reference(k, v, w, pos, table, lengths, budget, recent):
    """Host arrays after the call: (k, v, w, pos, lengths, kept)."""
    k, v, w, pos = k.copy(), v.copy(), w.copy(), pos.copy()
    S, H = k.shape[1], k.shape[2]
    B = len(lengths)
    kept = np.full((B, H, budget), -1, np.int32)
    for b in range(B):
        n = min(max(int(lengths[b]), 0), table.shape[1] * S)
        t = np.arange(n)
        page, slot = table[b][t // S], t % S
        for h in range(H):
            stay = keep_of(w[page, h, slot], pos[page, h, slot], budget, recent)
            place = np.arange(min(n, budget))
            free = np.setdiff1d(place, stay)
            place[free] = stay[stay >= budget]
            kept[b, h, :len(place)] = place
            for to, src in zip(free, place[free]):
                for x in (k, v):
                    x[page[to], slot[to], h] = x[page[src], slot[src], h]
                for x in (w, pos):
                    x[page[to], h, slot[to]] = x[page[src], h, slot[src]]
    return k, v, w, pos, np.minimum(np.maximum(lengths, 0), budget).astype(np.int32), kept


def make(B, H, D, S, lengths, kind, seed=0):
    r = np.random.default_rng([seed, B, H, D, S])
    need = [-(-max(n, 0) // S) for n in lengths]
    per, P = max(max(need), 1) + 1, sum(need) + 2
    k, v = (r.standard_normal((P, S, H, D)).astype(np.float16) for _ in range(2))
    table = np.full((B, per), -1, np.int32)
    pages, at = r.permutation(P), 0
    for b in range(B):
        table[b, :need[b]] = pages[at:at + need[b]]
        at += need[b]
    if kind == "ties":
        w = r.integers(0, 3, (P, H, S)).astype(np.float32)
        w[w == 1] = -0.0
    elif kind == "equal":
        w = np.full((P, H, S), 0.25, np.float32)
    elif kind == "wild":  # NaN of both signs, infinities, subnormals, negative weights
        w = r.choice(np.array([np.nan, -np.nan, np.inf, -np.inf, 1e-42, -1e-42, 0.0, -0.0, -1.5, 3.0, 1e30],
                              np.float32), (P, H, S))
    elif kind == "close":  # thousands of keys that share their top bits, some all of them
        w = (1 + r.integers(0, 1500, (P, H, S)) * 2.0**-23).astype(np.float32)
    else:
        w = (r.random((P, H, S)) ** 6 * 4).astype(np.float32)
    pos = r.permuted(np.tile(np.arange(P * S, dtype=np.int32), (H, 1)), axis=1).reshape(H, P, S).transpose(1, 0, 2)
    return k, v, w, np.ascontiguousarray(pos), table


def same(a, b):
    """Equal bits."""
    a = np.ascontiguousarray(a)
    return np.array_equal(a.view(np.uint8), np.ascontiguousarray(b).astype(a.dtype, copy=False).view(np.uint8))


def dev(x, layout="token"):
    import torch
    if layout == "head":
        return torch.from_numpy(np.ascontiguousarray(x.transpose(0, 2, 1, 3))).cuda().transpose(1, 2)
    return torch.from_numpy(x).cuda()


CASES = [
    # B, H, D, S, lengths, budget, recent, kind, layout
    (1, 1, 64, 16, [1], 1, 0, "long", "token"),
    (2, 3, 128, 16, [17, 16], 16, 4, "long", "token"),
    (4, 2, 128, 16, [0, 1, 64, 200], 64, 16, "long", "head"),
    (2, 2, 64, 8, [300, 299], 1, 0, "ties", "token"),
    (2, 2, 64, 8, [300, 299], 299, 5, "ties", "token"),
    (2, 2, 80, 24, [1000, 700], 333, 100, "equal", "head"),
    (2, 4, 256, 5, [513, 130], 100, 100, "wild", "token"),
    (2, 4, 8, 32, [513, 130], 100, 400, "wild", "token"),
    (1, 8, 128, 16, [4096], 1024, 128, "long", "token"),
    (1, 2, 128, 64, [5000], 4999, 1024, "long", "head"),
    (3, 2, 64, 16, [2500, 2049, 40], 2048, 0, "ties", "token"),
    (1, 2, 8, 128, [40000], 9000, 500, "long", "token"),     # more tokens than the keys that fit on chip
    (1, 1, 8, 256, [33000], 32990, 500, "ties", "token"),
    (1, 1, 8, 100, [20000], 150, 20, "equal", "token"),
    (4, 2, 8, 64, [33000, 1025, 32768, 300], 1000, 200, "long", "token"),   # short sequences in a table for long ones
    (3, 1, 8, 64, [40000, 32700, 21000], 16500, 100, "close", "head"),
    (2, 2, 64, 16, [2000, 1900], 1100, 10, "close", "token"),
    (1, 2, 64, 16, [8192], 8191, 0, "close", "head"),
    (1, 2, 8, 32, [32768], 16384, 300, "long", "token"),
    (1, 1, 8, 32, [32700], 10, 5, "close", "token"),
    (300, 1, 8, 8, [21] * 300, 20, 4, "long", "token"),
    (1, 2, 128, 16, [3000], 1000, 100, "long", "head"),       # few heads, many rows: a second launch moves them
    (2, 2, 64, 16, [100, 50], 0, 3, "long", "token"),
    (2, 2, 64, 16, [100, 50], 1000, 3, "long", "token"),     # a budget beyond the capacity
]


@gpu
@pytest.mark.parametrize("B,H,D,S,lengths,budget,recent,kind,layout", CASES)
@pytest.mark.parametrize("inplace", [True, False])
def test_against_the_definition(gpu_lib, B, H, D, S, lengths, budget, recent, kind, layout, inplace):
    import torch
    k, v, w, pos, table = make(B, H, D, S, lengths, kind)
    want = reference(k, v, w, pos, table, np.array(lengths), budget, recent)
    K, V, W, Q = dev(k, layout), dev(v, layout), dev(w), dev(pos)
    cache = swm.PagedCache(K, V, dev(table), torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    if inplace:
        n, kept = swm.kv_evict(cache, W, Q, budget, recent)
        got_w, got_q = W, Q
    else:
        got_w, got_q = torch.full_like(W, -7.0), torch.full_like(Q, -7)
        n, kept = swm.kv_evict(cache, W, Q, budget, recent, weights_out=got_w, positions_out=got_q)
        assert same(W.cpu().numpy(), w) and same(Q.cpu().numpy(), pos)  # the inputs stay
        inside = np.zeros((k.shape[0], S), bool)  # and the outputs are written below the new lengths only
        for b in range(B):
            t = np.arange(min(lengths[b], budget))
            inside[table[b][t // S], t % S] = True
        for x in want[2:4]:
            x[~np.broadcast_to(inside[:, None], x.shape)] = -7
    for name, x, y in zip("k v weights positions lengths kept".split(), (K, V, got_w, got_q, n, kept), want):
        assert same(x.cpu().numpy(), y), name
    assert cache.lengths.tolist() == lengths


@gpu
def test_attention_after_eviction(gpu_lib):
    """Evicting tokens whose weight is zero and attending over the rest gives the masked attention."""
    import torch
    B, H, D, S, n, budget = 2, 4, 128, 16, 200, 120
    k, v, w, pos, table = make(B, H, D, S, [n, n], "long")
    r = np.random.default_rng(5)
    drop = np.stack([r.permutation(n)[:n - budget] for _ in range(B)])
    mask = np.ones((B, table.shape[1] * S), bool)
    w[:] = 1.0
    for b in range(B):
        mask[b, drop[b]] = False
        w[table[b][drop[b] // S], :, drop[b] % S] = 0.0
    q = torch.from_numpy((2 * r.standard_normal((B, H, D))).astype(np.float16)).cuda()
    cache = swm.PagedCache(dev(k), dev(v), dev(table), torch.tensor([n, n], dtype=torch.int32, device="cuda"))
    before = swm.paged_attention(cache, q, mask=torch.from_numpy(mask).cuda())
    lengths, _ = swm.kv_evict(cache, dev(w), dev(pos), budget, 0)
    cache.lengths.copy_(lengths)
    after = swm.paged_attention(cache, q)
    # the same sums in another order: both are within one rounding to fp16 of the same value
    assert float((after.float() - before.float()).abs().max()) <= 2.0**-9


@gpu
def test_graph_and_stream(gpu_lib):
    import torch
    B, H, D, S = 2, 3, 64, 16
    k, v, w, pos, table = make(B, H, D, S, [300, 180], "long")
    K, V, W, Q = dev(k), dev(v), dev(w), dev(pos)
    cache = swm.PagedCache(K, V, dev(table), torch.tensor([300, 180], dtype=torch.int32, device="cuda"))
    wo, po = torch.zeros_like(W), torch.zeros_like(Q)
    n, kept = swm.kv_evict(cache, W, Q, 150, 10, weights_out=wo, positions_out=po)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        swm.kv_evict(cache, W, Q, 150, 10, weights_out=wo, positions_out=po, lengths_out=n, kept=kept)
    for lengths in ([300, 180], [151, 150], [0, 299 - 120], [300, 1]):
        K.copy_(dev(k)), V.copy_(dev(v)), wo.zero_(), po.zero_()
        cache.lengths.copy_(torch.tensor(lengths, dtype=torch.int32))
        want = reference(k, v, w, pos, table, np.array(lengths), 150, 10)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip((K, V, n, kept), (want[0], want[1], want[4], want[5])):
            assert same(x.cpu().numpy(), y), lengths
    K.copy_(dev(k)), V.copy_(dev(v))
    cache.lengths.copy_(torch.tensor([300, 180], dtype=torch.int32))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    n2, kept2 = swm.kv_evict(cache, W, Q, 150, 10, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    want = reference(k, v, w, pos, table, np.array([300, 180]), 150, 10)
    for x, y in zip((K, V, W, Q, n2, kept2), want):
        assert same(x.cpu().numpy(), y)


@gpu
def test_largest_budget(gpu_lib):
    import torch
    S, D, n = 16, 64, 37
    k = torch.zeros((4, S, 1, D), dtype=torch.float16, device="cuda")
    cache = swm.PagedCache(k, k.clone(), torch.tensor([[2, 0, 3]], dtype=torch.int32, device="cuda"),
                           torch.tensor([n], dtype=torch.int32, device="cuda"))
    w = torch.rand((4, 1, S), device="cuda")
    pos = torch.arange(4 * S, dtype=torch.int32, device="cuda").view(4, 1, S)
    lengths, kept = swm.kv_evict(cache, w, pos, (1 << 31) - 1, 4)
    assert lengths.tolist() == [n]
    assert torch.equal(kept[0, 0, :n], torch.arange(n, dtype=torch.int32, device="cuda"))
    assert int(kept[0, 0, n:].max()) == -1 and int(kept[0, 0, n:].min()) == -1


@gpu
def test_missing_pages_are_never_touched(gpu_lib):
    import torch
    k, v, w, pos, table = make(1, 2, 64, 16, [100], "long")
    table[0, 2], table[0, 5] = 1 << 20, -3
    cache = swm.PagedCache(dev(k), dev(v), dev(table), torch.tensor([100], dtype=torch.int32, device="cuda"))
    n, kept = swm.kv_evict(cache, dev(w), dev(pos), 60, 8)
    assert n.tolist() == [60]
    kept = kept.cpu().numpy()
    page = table[0][kept // 16]
    # 68 tokens are there for 60 places: none of the 32 that are not is taken from above the budget
    assert np.all((kept < 60) | ((page >= 0) & (page < k.shape[0])))


def reference_with_holes(k, v, w, pos, table, lengths, budget, recent, w_out, pos_out):
    """reference where the table may name no page: such tokens come after all others, and neither they nor what
    would move into their slots is copied.  w_out, pos_out: contents before the call (copies of w, pos: in place)."""
    P, S, H = k.shape[:3]
    k, v = k.copy(), v.copy()
    kept = np.full((len(lengths), H, budget), -1, np.int32)
    for b, n in enumerate(lengths):
        t = np.arange(n)
        page, slot = table[b][t // S], t % S
        there = (page >= 0) & (page < P)
        at = np.where(there, page, 0)
        for h in range(H):
            wt, pt = w[at, h, slot], pos[at, h, slot]
            newest = int(pt[there].max()) if there.any() else 0
            first = (pt.astype(np.int64) > newest - recent) | np.isnan(wt) | (wt == np.inf)
            order = sorted(t, key=lambda i: (2, 0.0, i) if not there[i] else
                           (0 if first[i] else 1, 0.0 if first[i] else -float(wt[i]), i))
            stay = np.array(sorted(order[:budget]), int)
            place = np.arange(min(n, budget))
            free = np.setdiff1d(place, stay)
            place[free] = stay[stay >= budget]
            kept[b, h, :len(place)] = place
            for to, src in enumerate(place):
                if there[to] and there[src]:
                    w_out[page[to], h, slot[to]], pos_out[page[to], h, slot[to]] = wt[src], pt[src]
                    for x in (k, v):
                        x[page[to], slot[to], h] = x[page[src], slot[src], h]
    return k, v, w_out, pos_out, np.minimum(lengths, budget).astype(np.int32), kept


HOLES = [
    # B, H, D, S, lengths, budget, recent, every how many-th page is missing
    (1, 2, 64, 16, [100], 60, 8, 3),
    (2, 2, 64, 5, [513, 130], 100, 10, 2),
    (2, 2, 128, 16, [2000, 700], 1990, 50, 4),       # more slots than tokens that are there
    (1, 2, 64, 16, [3000], 1200, 100, 3),            # a second launch moves the rows
    (1, 1, 8, 64, [40000], 15000, 500, 3),           # more tokens than the keys that fit on chip
    (1, 1, 8, 64, [40000], 39000, 500, 3),
    (300, 1, 8, 8, [21] * 300, 16, 4, 3),
    (2, 1, 64, 16, [90, 40], 100, 4, 3),             # within the budget
    (2, 1, 64, 16, [90, 40], 20, 4, 1),              # nothing there at all
]


@gpu
@pytest.mark.parametrize("B,H,D,S,lengths,budget,recent,every", HOLES)
@pytest.mark.parametrize("inplace", [True, False])
def test_everything_around_missing_pages(gpu_lib, B, H, D, S, lengths, budget, recent, every, inplace):
    """Bits of the pools, weights and positions where table entries name no page, page 0 and pages that no table
    names among them."""
    import torch
    k, v, w, pos, table = make(B, H, D, S, lengths, "long")
    wrong = np.array([-1, -(1 << 31), k.shape[0], 1 << 30], np.int32)
    for b in range(B):
        gone = np.arange(b % every, table.shape[1], every)
        table[b, gone] = wrong[gone % 4]
    assert not (np.unique(table[(table >= 0) & (table < k.shape[0])], return_counts=True)[1] > 1).any()
    K, V, W, Q = dev(k), dev(v), dev(w), dev(pos)
    cache = swm.PagedCache(K, V, dev(table), torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    if inplace:
        want = reference_with_holes(k, v, w, pos, table, lengths, budget, recent, w.copy(), pos.copy())
        n, kept = swm.kv_evict(cache, W, Q, budget, recent)
        got_w, got_q = W, Q
    else:
        want = reference_with_holes(k, v, w, pos, table, lengths, budget, recent, np.full_like(w, -7.0),
                                    np.full_like(pos, -7))
        got_w, got_q = torch.full_like(W, -7.0), torch.full_like(Q, -7)
        n, kept = swm.kv_evict(cache, W, Q, budget, recent, weights_out=got_w, positions_out=got_q)
        assert same(W.cpu().numpy(), w) and same(Q.cpu().numpy(), pos)
    for name, x, y in zip("lengths kept k v weights positions".split(), (n, kept, K, V, got_w, got_q),
                          (want[4], want[5], *want[:4])):
        assert same(x.cpu().numpy(), y), name


@gpu
def test_binding_refuses(gpu_lib):
    import torch
    k, v, w, pos, table = make(1, 2, 64, 16, [100], "long")
    c = swm.PagedCache(dev(k), dev(v), dev(table), torch.tensor([100], dtype=torch.int32, device="cuda"))
    W, Q = dev(w), dev(pos)
    with pytest.raises(TypeError):
        swm.kv_evict(c, W.double(), Q, 50)
    with pytest.raises(TypeError):
        swm.kv_evict(c, W, Q.long(), 50)
    with pytest.raises(ValueError):
        swm.kv_evict(c, W[:, :1], Q, 50)
    with pytest.raises(ValueError):
        swm.kv_evict(c, W, Q, -1)
    with pytest.raises(TypeError):
        swm.kv_evict(c, W, Q, 50, kept=torch.zeros((1, 2, 49), dtype=torch.int32, device="cuda"))
    with pytest.raises(swm.SwmError):
        swm.kv_evict(c, W, Q, 50, recent=-1)
    with pytest.raises(swm.SwmError):  # the lengths are read by every head while one writes the new ones
        swm.kv_evict(c, W, Q, 50, lengths_out=c.lengths)


@pytest.mark.parametrize("change", [
    dict(weights_out=8192, w_head=0, wo_head=0), dict(positions_out=12288, p_head=0, po_head=0),  # in place, expanded
    dict(wo_head=0), dict(po_head=15), dict(wo_page=0), dict(po_page=8), dict(wo_page=16, wo_head=16),
])
def test_entries_shared_by_heads_or_pages_are_not_written(change):
    """Heads of one sequence keep different tokens: entries that two of them wrote would be either's."""
    lib = swm.load()
    c = swm.KvCache(4096, 4096, 4096, 4096, 1024, 64, 64, 1024, 64, 64, 4, 8, 16, 3, 64, 2, 4)
    a = dict(weights=8192, w_page=48, w_head=16, positions=12288, p_page=48, p_head=16, budget=20, recent=4,
             weights_out=16384, wo_page=48, wo_head=16, positions_out=20480, po_page=48, po_head=16,
             lengths_out=24576, kept=28672, stream=None)
    a.update(change)
    assert lib.swm_kv_evict(ctypes.addressof(c), *a.values()) == 1


@pytest.mark.parametrize("stride", ["k_head", "v_head", "k_page", "v_page"])
def test_rows_shared_by_heads_or_pages_do_not_move(stride):
    lib = swm.load()
    f = dict(k=4096, v=4096, table=4096, lengths=4096, k_page=3072, k_slot=192, k_head=64, v_page=3072, v_slot=192,
             v_head=64, table_ld=4, pages=8, page_size=16, heads=3, dim=64, batch=2, pages_per_seq=4)
    f[stride] = 0
    c = swm.KvCache(**f)
    assert lib.swm_kv_evict(ctypes.addressof(c), 8192, 48, 16, 12288, 48, 16, 20, 4, 16384, 48, 16, 20480, 48, 16,
                            24576, 28672, None) == 1


@gpu
def test_heads_share_their_inputs(gpu_lib):
    """Positions and weights of a cache that nothing has been evicted from yet, the same for every head: expanded
    tensors as inputs alone; in place they are refused."""
    import torch
    B, H, D, S = 2, 3, 64, 16
    k, v, w, pos, table = make(B, H, D, S, [300, 180], "long")
    w[:], pos[:] = w[:, :1], pos[:, :1]
    want = reference(k, v, w, pos, table, np.array([300, 180]), 150, 10)
    K, V = dev(k), dev(v)
    W, Q = dev(np.ascontiguousarray(w[:, :1])).expand(-1, H, -1), dev(np.ascontiguousarray(pos[:, :1])).expand(-1, H, -1)
    cache = swm.PagedCache(K, V, dev(table), torch.tensor([300, 180], dtype=torch.int32, device="cuda"))
    with pytest.raises(swm.SwmError):
        swm.kv_evict(cache, W, Q, 150, 10)
    wo, po = W.contiguous(), Q.contiguous()
    n, kept = swm.kv_evict(cache, W, Q, 150, 10, weights_out=wo, positions_out=po)
    for x, y in zip((K, V, wo, po, n, kept), want):
        assert same(x.cpu().numpy(), y)


@pytest.mark.parametrize("change,code", [
    (dict(weights=None), 1), (dict(positions=None), 1), (dict(weights_out=None), 1), (dict(positions_out=None), 1),
    (dict(lengths_out=None), 1), (dict(kept=None), 1), (dict(budget=-1), 1), (dict(recent=-1), 1),
    (dict(budget=1 << 31), 1), (dict(recent=1 << 31), 1), (dict(w_page=-1), 1), (dict(po_head=-1), 1),
    (dict(lengths_out=4096), 1), (dict(weights_out=8192, wo_page=8), 1), (dict(positions_out=12288, po_head=8), 1),
])
def test_call_refusals(change, code):
    lib = swm.load()
    c = swm.KvCache(4096, 4096, 4096, 4096, 1024, 64, 64, 1024, 64, 64, 4, 8, 16, 1, 64, 2, 4)
    a = dict(weights=8192, w_page=16, w_head=16, positions=12288, p_page=16, p_head=16, budget=20, recent=4,
             weights_out=16384, wo_page=16, wo_head=16, positions_out=20480, po_page=16, po_head=16,
             lengths_out=24576, kept=28672, stream=None)
    a.update(change)
    assert lib.swm_kv_evict(ctypes.addressof(c), *a.values()) == code
    assert lib.swm_kv_evict(None, *a.values()) == 1
