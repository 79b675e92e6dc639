"""paged_attention against softmax attention in 64 bits, and its refusals.

Tolerances follow from the arithmetic: products of fp16 values are exact in
fp32, so a score is off by at most E = scale * D * 2^-24 * sum |q_d k_d| (the
fp32 sum) plus 2^-22 |x| (scaling and the subtraction of the maximum).  A
weight e^(x - m) / sum is then relatively off by at most 2 E plus 2^-19 (the
exponential, the running rescale and the sums), so an output by that times
sum p |v|, plus its one rounding to fp16 (2^-11 relative, 2^-25 below the
normal range).
"""
import ctypes

import numpy as np
import pytest

import sparse_weight_matmul_amd as swm

gpu = pytest.mark.gpu


def reference(q, k, v, table, lengths, scale, mask=None):
    """(out, bound on its error, weights per token, bound) in 64 bits; table/lengths/mask host arrays."""
    B, Hq, D = q.shape
    P, S, Hkv, _ = k.shape
    G = Hq // Hkv
    cap = table.shape[1] * S
    out, tol = np.zeros((B, Hq, D)), np.zeros((B, Hq, D))
    w, wtol = np.zeros((B, Hkv, cap)), np.zeros((B, Hkv, cap))
    for b in range(B):
        t = np.arange(min(max(int(lengths[b]), 0), cap))
        page = table[b][t // S] if len(t) else t
        t = t[(page >= 0) & (page < P)]
        if mask is not None:
            t = t[mask[b][t] != 0]
        if not len(t):
            continue
        page, slot = table[b][t // S], t % S
        for h in range(Hq):
            K, V = (np.asarray(x[page, slot, h // G], np.float64) for x in (k, v))
            qh = np.asarray(q[b, h], np.float64)
            x = scale * (K @ qh)
            e = np.exp(x - x.max())
            p = e / e.sum()
            err = np.max(abs(scale) * D * 2.0**-24 * (np.abs(K) @ np.abs(qh)) + 2.0**-22 * np.abs(x))
            eps = 2 * err + 2.0**-19
            out[b, h] = p @ V
            tol[b, h] = eps * (p @ np.abs(V)) + 2.0**-11 * np.abs(out[b, h]) + 2.0**-25
            w[b, h // G, t] += p
            wtol[b, h // G, t] += p * eps
    return out, tol, w, wtol


def make(B, Hq, Hkv, D, S, lengths, layout="token", seed=0, extra=3, slack=0):
    """Tensors of a case; every page has one owner and the spare ones hold NaN."""
    import torch
    r = np.random.default_rng([seed, B, Hq, D, S])
    need = [-(-max(n, 0) // S) for n in lengths]
    per, P = max(max(need), 1) + slack, sum(need) + extra
    k, v = (r.standard_normal((P, S, Hkv, D)).astype(np.float16) for _ in range(2))
    q = (2 * r.standard_normal((B, Hq, D))).astype(np.float16)
    pages = r.permutation(P)
    table = np.full((B, per), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :need[b]] = pages[at:at + need[b]]
        at += need[b]
        if need[b]:  # slots past the length hold stale values of the worst kind
            last = table[b, need[b] - 1]
            k[last, lengths[b] - (need[b] - 1) * S:] = np.nan
            v[last, lengths[b] - (need[b] - 1) * S:] = np.inf
    k[pages[at:]], v[pages[at:]] = np.nan, np.nan

    def pool(x):
        if layout == "token":
            return torch.from_numpy(x).cuda()
        return torch.from_numpy(np.ascontiguousarray(x.transpose(0, 2, 1, 3))).cuda().transpose(1, 2)

    dev = {"q": torch.from_numpy(q).cuda(), "k": pool(k), "v": pool(v), "table": torch.from_numpy(table).cuda(),
           "lengths": torch.tensor(lengths, dtype=torch.int32, device="cuda")}
    return q, k, v, table, dev


def check(out, ref, tol, what=""):
    got = out.double().cpu().numpy()
    assert np.all(np.isfinite(got)), what
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (what, int(bad.sum()), float(np.max(np.abs(got - ref) - tol)))


def ragged(B, most, seed=0):
    r = np.random.default_rng([seed, B, most])
    n = r.integers(0, most + 1, B)
    n[r.integers(0, B, 1 + B // 8)] = 0
    n[r.integers(0, B)] = most
    return n.tolist()


CASES = [
    # B, Hq, Hkv, D, S, lengths, layout
    (1, 1, 1, 64, 16, [1], "token"),
    (1, 32, 32, 128, 16, [137], "token"),
    (3, 4, 4, 128, 16, [0, 1, 33], "head"),
    (4, 8, 2, 128, 32, [31, 32, 127, 129], "token"),
    (2, 6, 2, 80, 24, [100, 257], "head"),
    (2, 5, 1, 96, 8, [640, 77], "token"),
    (2, 16, 1, 64, 64, [1000, 5], "head"),
    (1, 17, 1, 128, 16, [300], "token"),
    (1, 40, 1, 64, 16, [1500], "token"),
    (2, 6, 3, 256, 16, [513, 40], "token"),
    (2, 4, 2, 136, 40, [90, 200], "head"),
    (3, 3, 3, 8, 16, [50, 64, 200], "token"),
    (2, 4, 4, 40, 1, [19, 260], "token"),
    (2, 4, 2, 128, 5, [131, 12], "head"),
    (1, 2, 2, 200, 100, [350], "token"),
    (1, 8, 1, 128, 128, [20001], "head"),
    (2, 2, 2, 64, 20, [9000, 4097], "token"),
    (1, 16, 1, 256, 16, [700], "token"),                    # the most shared memory
    (1, 32, 2, 248, 24, [5000], "head"),
    (40, 8, 8, 64, 16, ragged(40, 1500), "token"),          # more units than CUs: sorted
    (128, 4, 4, 64, 8, ragged(128, 1300), "head"),
    (129, 3, 3, 64, 16, ragged(129, 1400), "token"),        # too many sequences to sort
    (100, 2, 1, 128, 32, ragged(100, 1600), "token"),       # cut by the lengths
    (21, 16, 8, 64, 16, ragged(21, 4300), "head"),
    (9, 34, 2, 256, 16, ragged(9, 5000), "token"),
    (20, 8, 8, 64, 16, [4200] * 20, "token"),               # of one length: whole
]


@gpu
@pytest.mark.parametrize("B,Hq,Hkv,D,S,lengths,layout", CASES)
@pytest.mark.parametrize("masked", [False, True])
def test_against_64_bits(gpu_lib, B, Hq, Hkv, D, S, lengths, layout, masked):
    import torch
    q, k, v, table, dev = make(B, Hq, Hkv, D, S, lengths, layout)
    P, cap = k.shape[0], table.shape[1] * S
    r = np.random.default_rng(7)
    mask = None
    if masked:
        mask = r.random((B, cap + 3)) < 0.7  # rows longer than the capacity
        mask[0] = False                      # a row that the mask leaves empty
        for b in range(1, B):                # masked rows hold infinities and NaN
            for t in np.nonzero(~mask[b][:lengths[b]])[0][:20]:
                dev["k"][int(table[b][t // S]), int(t % S)] = float("nan")
                dev["v"][int(table[b][t // S]), int(t % S)] = float("-inf")
    w0 = r.random((P, Hkv, S)).astype(np.float32)
    w = torch.from_numpy(w0).cuda()
    cache = swm.PagedCache(dev["k"], dev["v"], dev["table"], dev["lengths"])
    m = None if mask is None else torch.from_numpy(mask).cuda()
    out = swm.paged_attention(cache, dev["q"], mask=m, weights=w)
    plain = swm.paged_attention(cache, dev["q"], mask=m)
    ref, tol, add, addtol = reference(q, k, v, table, lengths, D ** -0.5, mask)
    check(out, ref, tol)
    assert torch.equal(out, plain)  # the accumulator changes nothing, and a second call gives the same bits
    want, wt = w0.astype(np.float64), np.zeros_like(w0, dtype=np.float64)
    for b in range(B):
        for t in range(lengths[b]):
            want[table[b][t // S], :, t % S] += add[b, :, t]
            wt[table[b][t // S], :, t % S] += addtol[b, :, t]
    got = w.double().cpu().numpy()
    assert np.all(np.abs(got - want) <= wt + 2.0**-23 * np.abs(want))
    assert np.array_equal(got[want == w0], w0[want == w0])  # nothing is added anywhere else


@gpu
@pytest.mark.parametrize("B,Hq,Hkv,D,lengths", [
    (2, 4, 2, 64, [1000, 517]),           # whole sequences
    (130, 1, 1, 128, [1500] * 130),       # longer ones
    (1, 2, 1, 128, [131072]),             # cut into pieces
    (5, 6, 3, 256, [4000, 9000, 1, 2, 40]),
])
@pytest.mark.parametrize("gap", [4, 8, 12, 16, 18])
def test_one_token_far_above_the_others(gpu_lib, B, Hq, Hkv, D, lengths, gap):
    """A token `gap` nats above all others whose value row is zero: the output is the others' small share."""
    import torch
    S = 16
    q, k, v, table, dev = make(B, Hq, Hkv, D, S, lengths)
    r = np.random.default_rng(gap)
    q[:] = 0
    q[:, :, 0] = 8
    k[:, :, :, 0] = 0
    v[:] = np.where(np.isnan(v), v, 1 + v / 8)
    for b, n in enumerate(lengths):
        t = 0 if b % 2 == 0 else int(r.integers(0, n))
        k[table[b][t // S], t % S, :, 0] = gap / (8 * D ** -0.5)
        v[table[b][t // S], t % S] = 0
    cache = swm.PagedCache(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), dev["table"], dev["lengths"])
    w = torch.zeros((k.shape[0], Hkv, S), device="cuda")
    out = swm.paged_attention(cache, torch.from_numpy(q).cuda(), weights=w)
    ref, tol, add, addtol = reference(q, k, v, table, lengths, D ** -0.5)
    check(out, ref, tol)
    got = w.double().cpu().numpy()
    for b, n in enumerate(lengths):
        t = np.arange(n)
        at = got[table[b][t // S], :, t % S].T
        assert np.all(np.abs(at - add[b, :, :n]) <= addtol[b, :, :n])


@gpu
def test_strided_operands_stream_and_scale(gpu_lib):
    import torch
    B, H, D, S = 3, 4, 128, 16
    lengths = [70, 300, 5]
    q, k, v, table, dev = make(B, H, H, D, S, lengths, slack=2)
    ref, tol, _, _ = reference(q, k, v, table, lengths, 0.05)
    stacked = torch.zeros((B, 3 * H * D), dtype=torch.float16, device="cuda")
    stacked[:, H * D:2 * H * D] = dev["q"].reshape(B, -1)
    qs = stacked[:, H * D:2 * H * D].view(B, H, D)
    wide = torch.full((B, 9 + table.shape[1]), -7, dtype=torch.int32, device="cuda")
    wide[:, 4:4 + table.shape[1]] = dev["table"]
    kv = torch.stack([dev["k"], dev["v"]], dim=2)  # keys and values side by side in one pool
    cache = swm.PagedCache(kv[:, :, 0], kv[:, :, 1], wide[:, 4:4 + table.shape[1]], dev["lengths"])
    out = torch.full((B, 2 * H, D), 9.0, dtype=torch.float16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    swm.paged_attention(cache, qs, scale=0.05, out=out[:, ::2], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    check(out[:, ::2], ref, tol)
    assert bool((out[:, 1::2] == 9).all())


@gpu
def test_entries_outside_the_pool_and_lengths_past_the_capacity(gpu_lib):
    import torch
    B, H, D, S = 3, 2, 64, 16
    lengths = [90, 64, 48]
    q, k, v, table, dev = make(B, H, H, D, S, lengths)
    table = table.copy()
    table[0, 2] = 1 << 30
    table[1, 0] = -5
    table[2, :] = k.shape[0]
    dev["table"].copy_(torch.from_numpy(table))
    dev["lengths"].copy_(torch.tensor([90, 1 << 30, -3], dtype=torch.int32))
    dev["k"][:] = torch.nan_to_num(dev["k"], nan=0.5)
    dev["v"][:] = torch.nan_to_num(dev["v"], nan=0.5, posinf=1.0)
    k, v = dev["k"].cpu().numpy(), dev["v"].cpu().numpy()
    cache = swm.PagedCache(dev["k"], dev["v"], dev["table"], dev["lengths"])
    ref, tol, _, _ = reference(q, k, v, table, [90, 1 << 30, -3], D ** -0.5)
    check(swm.paged_attention(cache, dev["q"]), ref, tol)


@gpu
def test_shared_pages_add_up(gpu_lib):
    import torch
    B, H, D, S = 2, 2, 64, 16
    q, k, v, table, dev = make(B, H, H, D, S, [64, 80])
    dev["table"][1, :4] = dev["table"][0, :4]
    table = dev["table"].cpu().numpy()
    cache = swm.PagedCache(dev["k"], dev["v"], dev["table"], dev["lengths"])
    w = torch.zeros((k.shape[0], H, S), device="cuda")
    out = swm.paged_attention(cache, dev["q"], weights=w)
    ref, tol, add, addtol = reference(q, k, v, table, [64, 80], D ** -0.5)
    check(out, ref, tol)
    got = w.double().cpu().numpy()
    for t in range(64):
        want = add[0, :, t] + add[1, :, t]
        at = got[table[0][t // S], :, t % S]
        assert np.all(np.abs(at - want) <= addtol[0, :, t] + addtol[1, :, t] + 2.0**-22 * want)


@gpu
def test_offsets_past_32_bits(gpu_lib):
    import torch
    # a pool of 2^32 + elements (8.6 GB); the sequences' pages are its last ones
    S, H, D = 64, 32, 128
    P = (1 << 32) // (S * H * D) + 3
    pool = torch.empty((P, S, H, D), dtype=torch.float16, device="cuda")
    r = np.random.default_rng(3)
    rows = r.standard_normal((3, S, H, D)).astype(np.float16)
    pool[P - 3:] = torch.from_numpy(rows).cuda()
    table = np.array([[P - 1, P - 3, P - 2]], np.int32)
    q = r.standard_normal((1, H, D)).astype(np.float16)
    cache = swm.PagedCache(pool, pool, torch.from_numpy(table).cuda(), torch.tensor([150], dtype=torch.int32).cuda())
    ref, tol, _, _ = reference(q, rows, rows, table - (P - 3), [150], D ** -0.5)
    check(swm.paged_attention(cache, torch.from_numpy(q).cuda()), ref, tol)


@gpu
@pytest.mark.parametrize("tokens", [2047 * 1049056, 2047 * 1049056 - 1000000])
def test_capacities_next_to_2_31(gpu_lib, tokens):
    import torch
    # 2046 times a page of zeros, then a page of 2047: exact sums, a mean of 2047 * (its share)
    S, D, n = 1049056, 8, 2047
    k = torch.zeros((2, S, 1, D), dtype=torch.float16, device="cuda")
    v = torch.zeros_like(k)
    v[1] = 2047
    table = torch.zeros((1, n), dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    cache = swm.PagedCache(k, v, table, torch.tensor([tokens], dtype=torch.int32, device="cuda"))
    out = swm.paged_attention(cache, torch.ones((1, 1, D), dtype=torch.float16, device="cuda"))
    want = 2047 * (tokens - (n - 1) * S) / tokens
    # sums of up to 2^31 in fp32, one rounding per split and two: far below one rounding to fp16
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= 2.0**-10 * want)


@gpu
def test_graph_follows_lengths_and_table(gpu_lib):
    import torch
    B, H, D, S = 2, 4, 128, 16
    q, k, v, table, dev = make(B, H, H, D, S, [3000, 2500])
    cache = swm.PagedCache(dev["k"], dev["v"], dev["table"], dev["lengths"])
    ws = torch.empty(cache.attention_workspace_bytes(H, True), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(dev["q"])
    w = torch.zeros((k.shape[0], H, S), device="cuda")
    swm.paged_attention(cache, dev["q"], weights=w, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        swm.paged_attention(cache, dev["q"], weights=w, out=out, workspace=ws)
    for n in ([1, 2500], [3000, 0], [1234, 777], [3000, 2500]):
        dev["lengths"].copy_(torch.tensor(n, dtype=torch.int32))
        want = torch.zeros_like(w)
        eager = swm.paged_attention(cache, dev["q"], weights=want)
        w.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and torch.equal(w, want)
        ref, tol, _, _ = reference(q, k, v, table, n, D ** -0.5)
        check(out, ref, tol, str(n))


@gpu
def test_infinite_scores_and_no_sequences(gpu_lib):
    import torch
    q, k, v, table, dev = make(1, 1, 1, 64, 16, [32])
    cache = swm.PagedCache(dev["k"], dev["v"], dev["table"], dev["lengths"])
    dev["k"][int(table[0, 0]), 3] = float("nan")  # a live NaN is the caller's own
    assert bool(torch.isnan(swm.paged_attention(cache, dev["q"])).all())
    none = swm.PagedCache(dev["k"], dev["v"], dev["table"][:0], dev["lengths"][:0])
    assert swm.paged_attention(none, dev["q"][:0]).shape == (0, 1, 64)
    nowhere = swm.PagedCache(dev["k"], dev["v"], dev["table"][:, :0], dev["lengths"])
    assert bool((swm.paged_attention(nowhere, dev["q"]) == 0).all())


@gpu
@pytest.mark.parametrize("lengths", [[200, 90], [5000, 3000]])
def test_infinite_values_stay_in_their_dimension(gpu_lib, lengths):
    import torch
    q, k, v, table, dev = make(2, 4, 2, 64, 16, lengths)
    dev["v"][int(table[0, 1]), 3, 1, 17] = float("inf")  # sequence 0, query heads 2 and 3
    cache = swm.PagedCache(dev["k"], dev["v"], dev["table"], dev["lengths"])
    out = swm.paged_attention(cache, dev["q"])
    hit = np.zeros((2, 4, 64), bool)
    hit[0, 2:, 17] = True
    assert np.array_equal(~np.isfinite(out.float().cpu().numpy()), hit)
    ref, tol, _, _ = reference(q, k, v, table, lengths, 64 ** -0.5)
    check(torch.where(torch.from_numpy(hit).cuda(), torch.zeros_like(out), out), np.where(hit, 0, ref), tol)


@gpu
@pytest.mark.parametrize("B,Hq,Hkv,lengths", [(2, 4, 2, [200, 90]),       # weights added by the first launch
                                              (2, 4, 2, [5000, 3000]),    # cut into pieces
                                              (2, 40, 2, [300, 170])])    # scores through the workspace
@pytest.mark.parametrize("where", ["key", "query"])
def test_nan_among_live_tokens_adds_nothing_elsewhere(gpu_lib, B, Hq, Hkv, lengths, where):
    import torch
    D, S = 64, 16
    q, k, v, table, dev = make(B, Hq, Hkv, D, S, lengths)
    r = np.random.default_rng(11)
    mask = r.random((B, table.shape[1] * S)) < 0.6
    mask[0, 5] = True
    table[0, 2] = -1  # tokens on no page
    dev["table"].copy_(torch.from_numpy(table))
    if where == "key":
        dev["k"][int(table[0, 0]), 5, 0] = float("nan")
    else:
        dev["q"][0, 1] = float("nan")
    cache = swm.PagedCache(dev["k"], dev["v"], dev["table"], dev["lengths"])
    w0 = r.random((k.shape[0], Hkv, S)).astype(np.float32)
    w = torch.from_numpy(w0).cuda()
    out = swm.paged_attention(cache, dev["q"], mask=torch.from_numpy(mask).cuda(), weights=w)
    hit = np.zeros((B, Hq), bool)  # the first sequence: the heads of key-value head 0, or the one query head
    hit[0, slice(0, Hq // Hkv) if where == "key" else 1] = True
    assert np.array_equal(np.isnan(out.float().cpu().numpy()).any(-1), hit)
    got = w.cpu().numpy()
    live = np.zeros((k.shape[0], S), bool)
    for b, n in enumerate(lengths):
        t = np.arange(n)[mask[b, :n]]
        t = t[table[b][t // S] >= 0]
        live[table[b][t // S], t % S] = True
        at = got[table[b][t // S], :, t % S]
        assert np.array_equal(np.isnan(at), np.broadcast_to(np.arange(Hkv) == 0, at.shape) & (b == 0))
    live = np.broadcast_to(live[:, None], got.shape)
    assert np.array_equal(got[~live], w0[~live])


@gpu
def test_binding_refuses(gpu_lib):
    import torch
    q, k, v, table, dev = make(2, 4, 2, 64, 16, [20, 30])
    c = swm.PagedCache(dev["k"], dev["v"], dev["table"], dev["lengths"])
    with pytest.raises(TypeError):
        swm.PagedCache(dev["k"].float(), dev["v"], dev["table"], dev["lengths"])
    with pytest.raises(TypeError):
        swm.PagedCache(dev["k"], dev["v"], dev["table"].long(), dev["lengths"])
    with pytest.raises(ValueError):
        swm.PagedCache(dev["k"], dev["v"][:1], dev["table"], dev["lengths"])
    with pytest.raises(TypeError):
        swm.paged_attention(c, dev["q"].float())
    with pytest.raises(ValueError):
        swm.paged_attention(c, dev["q"][:1])
    with pytest.raises(ValueError):
        swm.paged_attention(c, dev["q"], mask=torch.ones((2, 3), dtype=torch.bool, device="cuda"))
    with pytest.raises(ValueError):
        swm.paged_attention(c, dev["q"], weights=torch.zeros((1, 2, 16), device="cuda"))
    with pytest.raises(swm.SwmError):  # three heads over two
        swm.paged_attention(c, torch.zeros((2, 3, 64), dtype=torch.float16, device="cuda"))
    with pytest.raises(swm.SwmError):  # eight-byte alignment
        odd = torch.zeros(2 * 4 * 64 + 4, dtype=torch.float16, device="cuda")[4:].view(2, 4, 64)
        swm.paged_attention(c, odd)
    with pytest.raises(swm.SwmError):
        # more query heads to a key-value head than one workgroup takes: the scores go through the workspace
        many = torch.zeros((2, 34, 64), dtype=torch.float16, device="cuda")
        assert c.attention_workspace_bytes(34, True) > 16
        swm.paged_attention(c, many, weights=torch.zeros((k.shape[0], 2, 16), device="cuda"),
                            workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))


def cache_struct(**kw):
    f = dict(k=4096, v=4096, table=4096, lengths=4096, k_page=1024, k_slot=64, k_head=64, v_page=1024, v_slot=64,
             v_head=64, table_ld=4, pages=8, page_size=16, heads=1, dim=64, batch=2, pages_per_seq=4)
    f.update(kw)
    return swm.KvCache(**f)


# Sizes and addresses that are refused before anything touches a device.
REFUSED = [
    (dict(k=None), 1), (dict(lengths=None), 1), (dict(table=None), 1), (dict(batch=-1), 1), (dict(pages=0), 1),
    (dict(page_size=0), 1), (dict(heads=0), 1), (dict(k_slot=-64), 1), (dict(table_ld=-1), 1), (dict(dim=0), 1),
    (dict(dim=60), 8), (dict(dim=264), 8), (dict(batch=65536), 8), (dict(page_size=1 << 30), 8),
    (dict(k=4104), 3), (dict(v_head=4), 3), (dict(k_page=1028), 3),
]


@pytest.mark.parametrize("fields,code", REFUSED)
def test_cache_refusals(fields, code):
    lib = swm.load()
    c = cache_struct(**fields)
    p = ctypes.addressof(c)
    assert lib.swm_paged_attention(p, 4096, 64, 64, 1, 0.125, None, 0, None, 0, 0, 8192, 64, 64, None, 0,
                                   None) == code
    if "k" not in fields and "v_head" not in fields and "k_page" not in fields and code != 1:
        assert lib.swm_paged_attention_workspace_bytes(p, 1, 1) == 0


@pytest.mark.parametrize("change,code", [
    (dict(q=None), 1), (dict(out=None), 1), (dict(heads=0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(q_batch=-8), 1), (dict(mask=4096, mask_ld=63), 1),
    (dict(weights=4096, w_page=-1), 1), (dict(q=4104), 3), (dict(q_head=4), 3), (dict(heads=65536), 8),
])
def test_call_refusals(change, code):
    lib = swm.load()
    c = cache_struct()
    a = dict(q=4096, q_batch=64, q_head=64, heads=1, scale=0.125, mask=None, mask_ld=0, weights=None, w_page=0,
             w_head=0, out=8192, out_batch=64, out_head=64, ws=None, ws_bytes=0, stream=None)
    a.update(change)
    assert lib.swm_paged_attention(ctypes.addressof(c), *a.values()) == code
    assert lib.swm_paged_attention(None, *a.values()) == 1


@pytest.mark.parametrize("strides", [(0, 64), (63, 64), (256, 0), (256, 32), (64, 64)])
def test_outputs_that_share_memory_are_refused(strides):
    lib = swm.load()
    c = cache_struct(heads=4)
    assert lib.swm_paged_attention(ctypes.addressof(c), 4096, 256, 64, 4, 0.125, None, 0, None, 0, 0, 8192, *strides,
                                   None, 0, None) == 1


def test_query_heads_are_a_multiple():
    lib = swm.load()
    c = cache_struct(heads=4)
    assert lib.swm_paged_attention_workspace_bytes(ctypes.addressof(c), 6, 0) == 0
    assert lib.swm_paged_attention(ctypes.addressof(c), 4096, 64, 64, 6, 0.125, None, 0, None, 0, 0, 8192, 64, 64,
                                   None, 0, None) == 1
