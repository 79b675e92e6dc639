"""prompt_attention against softmax attention in 64 bits, and its refusals.

Tolerances follow from the arithmetic: products of fp16 values are exact in
fp32, so a score is off by at most E = scale * D * 2^-24 * sum |q_d k_d| (the
fp32 sum) plus 2^-22 |x| (scaling and the subtraction of the maximum).  A
weight is then relatively off by at most 2 E plus 2^-19 (the exponential, the
rescales and the sum).  Its one rounding to fp16, d_j = 2^-11 p_j at most, or
2^-35 of the largest weight where it is far below it, is in the numerator and in
the sum that divides: sum (p_j + d_j) v_j / sum (p_j + d_j) is off by sum d_j
(v_j - o), to first order, so by at most 2^-11 (sum p |v| + |o|) and n 2^-34 max
|v|.  The output's sum over n tokens, sixteen at a time, adds n / 16 + 64
roundings of 2^-24, its own rounding 2^-11 of itself (2^-25 below the normal
range).
"""
import ctypes

import numpy as np
import pytest

import sparse_weight_matmul_amd as swm

gpu = pytest.mark.gpu


def attend(q, K, V, scale, sees):
    """(out, bound) of rows q over tokens K, V in 64 bits; sees (rows, tokens) bool."""
    q, K, V = (np.asarray(x, np.float64) for x in (q, K, V))
    x = scale * (q @ K.T)
    err = np.abs(scale) * q.shape[1] * 2.0**-24 * (np.abs(q) @ np.abs(K).T) + 2.0**-22 * np.abs(x)
    err = np.where(sees, err, 0).max(1, initial=0.0, keepdims=True)
    x = np.where(sees, x, -np.inf)
    top = x.max(1, initial=-np.inf, keepdims=True)
    e = np.exp(x - np.where(np.isfinite(top), top, 0))
    total = e.sum(1, keepdims=True)
    p = e / np.where(total > 0, total, 1)
    n = sees.sum(1)[:, None]
    eps = 2 * err + 2.0**-19 + 2.0**-11 + (n / 16 + 64) * 2.0**-24
    out = p @ V
    tol = eps * (p @ np.abs(V)) + 2.0**-34 * n * np.abs(V).max(initial=0) + 2.0**-10 * np.abs(out) + 2.0**-25
    return out, tol


def reference(q, k, v, starts, scale, causal):
    """(out, bound, rows of a sequence) for host arrays."""
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    out, tol, rows = np.zeros((T, Hq, D)), np.zeros((T, Hq, D)), np.zeros(T, bool)
    for a, b in zip(starts[:-1], starts[1:]):
        sees = np.tril(np.ones((b - a, b - a), bool)) if causal else np.ones((b - a, b - a), bool)
        rows[a:b] = True
        for h in range(Hq if b > a else 0):
            out[a:b, h], tol[a:b, h] = attend(q[a:b, h], k[a:b, h // G], v[a:b, h // G], scale, sees)
    return out, tol, rows


def make(T, Hq, Hkv, D, layout="separate", seed=0):
    """Host arrays and device tensors of T rows."""
    import torch
    r = np.random.default_rng([seed, T, Hq, Hkv, D])
    q, k, v = (r.standard_normal((T, h, D)).astype(np.float16) for h in (Hq, Hkv, Hkv))
    q *= np.float16(2)
    if layout == "stacked":
        y = torch.from_numpy(np.concatenate([q, k, v], 1)).cuda()
        return q, k, v, y[:, :Hq], y[:, Hq:Hq + Hkv], y[:, Hq + Hkv:]
    if layout == "head":
        return q, k, v, *(torch.from_numpy(np.ascontiguousarray(x.transpose(1, 0, 2))).cuda().transpose(0, 1)
                          for x in (q, k, v))
    return q, k, v, *(torch.from_numpy(x).cuda() for x in (q, k, v))


def bounds(lengths, first=0):
    return (first + np.concatenate([[0], np.cumsum(lengths)])).astype(np.int32)


def ints(x):
    import torch
    return torch.from_numpy(np.asarray(x, np.int32)).cuda()


def check(out, ref, tol, what=""):
    got = out.double().cpu().numpy()
    assert np.all(np.isfinite(got)), what
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (what, int(bad.sum()), float(np.max(np.abs(got - ref) - tol)))


CASES = [
    # Hq, Hkv, D, lengths, layout
    (1, 1, 64, [1], "separate"),
    (4, 4, 128, [137], "stacked"),
    (4, 2, 128, [31, 32, 33, 63, 64, 65], "separate"),
    (2, 1, 128, [127, 128, 129, 0, 1, 2], "head"),
    (3, 1, 80, [300, 0, 191], "head"),
    (5, 5, 96, [97, 255], "stacked"),
    (2, 2, 72, [130], "separate"),
    (2, 1, 8, [70, 200], "separate"),
    (2, 2, 40, [66, 1], "stacked"),
    (2, 1, 136, [129, 65], "separate"),
    (2, 2, 192, [257], "head"),
    (4, 1, 200, [100, 90], "separate"),
    (2, 1, 248, [140], "stacked"),
    (8, 1, 256, [193, 64], "separate"),
    (16, 2, 64, [0, 0, 385, 0], "separate"),
    (40, 8, 16, [65, 130], "stacked"),
    (8, 8, 64, [3] * 70 + [150] + [0] * 60 + [129, 1], "separate"),  # more sequences than lanes
    (1, 1, 128, [2100], "separate"),
    (16, 4, 64, [9, 1, 0, 33, 70, 31, 32, 64] * 8, "stacked"),       # a wave a block
    (24, 3, 128, [20] * 30 + [0, 100, 65], "head"),
    (32, 32, 80, [1, 2, 40] * 20, "separate"),
    (36, 4, 256, [17, 35, 5, 0] * 16, "separate"),
    (2, 1, 64, [(7 * b) % 5 for b in range(3000)] + [140], "separate"),
    (48, 4, 128, [100] * 70, "separate"),                            # small tiles
    (48, 4, 96, [90, 0, 300, 128, 129, 1] * 12, "stacked"),
    (8, 2, 128, [1111, 640], "separate"),
]


@gpu
@pytest.mark.parametrize("Hq,Hkv,D,lengths,layout", CASES)
@pytest.mark.parametrize("causal", [True, False])
def test_against_64_bits(gpu_lib, Hq, Hkv, D, lengths, layout, causal):
    import torch
    T = sum(lengths) + 7  # rows before and behind the sequences
    q, k, v, dq, dk, dv = make(T, Hq, Hkv, D, layout)
    for x in (dk, dv):  # stale rows of the worst kind
        x[:3] = float("nan")
        x[T - 4:] = float("inf")
    starts = bounds(lengths, 3)
    out = torch.full((T, Hq, D), 7.0, dtype=torch.float16, device="cuda")
    got = swm.prompt_attention(dq, dk, dv, ints(starts), causal=causal, out=out)
    assert got is out
    ref, tol, rows = reference(q, k, v, starts, D ** -0.5, causal)
    check(out[torch.from_numpy(rows).cuda()], ref[rows], tol[rows])
    assert bool((out[torch.from_numpy(~rows).cuda()] == 7.0).all())
    again = swm.prompt_attention(dq, dk, dv, ints(starts), causal=causal)
    assert torch.equal(again[3:T - 4], out[3:T - 4])


@gpu
@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("gap", [2.0, 17.0, 40.0])
def test_one_token_far_above_the_others(gpu_lib, D, gap):
    """A first token of value zero takes almost all of the weight: the others' share is the whole output."""
    q, k, v, dq, dk, dv = make(700, 2, 1, D, seed=3)
    u = np.ones(D, np.float16)
    q[:], k[:] = u, 0
    k[0, 0] = np.float16(gap) / np.float16(D ** 0.5) * u  # scores: gap, then zeros
    v[0] = 0
    v[1:] = np.abs(v[1:]) + np.float16(0.25)
    for x, y in ((dq, q), (dk, k), (dv, v)):
        import torch
        x.copy_(torch.from_numpy(y))
    starts = bounds([700])
    out = swm.prompt_attention(dq, dk, dv, ints(starts))
    ref, tol, _ = reference(q, k, v, starts, D ** -0.5, True)
    check(out, ref, tol)


@gpu
@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0, 1e-4])
def test_scales(gpu_lib, scale):
    q, k, v, dq, dk, dv = make(200, 4, 2, 64)
    starts = bounds([150, 50])
    out = swm.prompt_attention(dq, dk, dv, ints(starts), scale=scale)
    ref, tol, _ = reference(q, k, v, starts, scale, True)
    check(out, ref, tol)


@gpu
def test_scores_of_any_size(gpu_lib):
    """Scores of thousands of either sign: a row's largest alone counts, wherever it stands."""
    q, k, v, dq, dk, dv = make(400, 2, 2, 128, seed=9)
    starts = bounds([400])
    out = swm.prompt_attention(dq, dk, dv, ints(starts), scale=30.0)
    ref, tol, _ = reference(q, k, v, starts, 30.0, True)
    check(out, ref, tol)


@gpu
def test_heads_share_keys_and_rows_share_queries(gpu_lib):
    """Expanded inputs: one key-value head for all, one query row for all tokens."""
    import torch
    q, k, v, dq, dk, dv = make(150, 4, 1, 64)
    starts = bounds([100, 50])
    ref, tol, _ = reference(q, k, v, starts, 0.125, True)
    wide = [x.expand(150, 4, 64) for x in (dk, dv)]
    check(swm.prompt_attention(dq, *wide, ints(starts)), ref, tol)
    one = dq[:1].expand(150, 4, 64)
    ref, tol, _ = reference(np.broadcast_to(q[:1], q.shape), k, v, starts, 0.125, True)
    check(swm.prompt_attention(one, dk, dv, ints(starts)), ref, tol)
    assert swm.prompt_attention(dq[:1], dk[:1].expand(1, 2, 64), dv[:1].expand(1, 2, 64),
                                ints([0, 1])).allclose(dv[:1].expand(1, 4, 64))


@gpu
@pytest.mark.parametrize("D", [64, 80, 128, 256])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("at", [0, 70, 127, 128, 200, 299])
def test_what_is_not_finite_stays_with_its_readers(gpu_lib, D, bad, at):
    """A value that is no number reaches its dimension of the rows that see its token, a key all of those rows."""
    import torch
    q, k, v, dq, dk, dv = make(360, 2, 1, D)
    starts = bounds([300, 60])
    ref, tol, _ = reference(q, k, v, starts, D ** -0.5, True)
    hit = np.zeros((360, 2, D), bool)
    hit[at:300, :, D - 3] = True
    dv[at, 0, D - 3] = bad
    out = swm.prompt_attention(dq, dk, dv, ints(starts)).double().cpu().numpy()
    assert np.array_equal(~np.isfinite(out), hit)
    assert np.all(np.abs(out - ref)[~hit] <= tol[~hit])
    dv[at, 0, D - 3] = 0.0
    dk[at, 0, 1] = float("nan")
    hit[:] = False
    hit[at:300] = True
    out = swm.prompt_attention(dq, dk, dv, ints(starts)).double().cpu().numpy()
    assert np.array_equal(np.isnan(out), hit)


LONG = [
    # Hq, Hkv, D, lengths: short in the mean, some far above it
    (8, 2, 128, [1] * 30 + [513] + [0] * 30 + [512, 9]),
    (12, 4, 64, [3, 0, 700, 1, 641, 640, 40] + [2] * 57),
    (8, 1, 256, [0] * 63 + [1500]),
    (9, 3, 80, [1300] + [0, 1] * 40),                          # more sequences than lanes
    (4, 4, 128, [5] * 100 + [2049] + [31, 33, 0] * 60 + [514]),
    (2, 1, 96, [0] * 700 + [513, 511, 1025] + [1, 0, 64] * 100 + [1100]),
    (4, 2, 40, [(7 * b) % 5 for b in range(3000)] + [900, 140, 600]),
    (16, 16, 192, [10] * 60 + [600]),
]


@gpu
@pytest.mark.parametrize("Hq,Hkv,D,lengths", LONG)
@pytest.mark.parametrize("causal", [True, False])
def test_long_prompts_among_short_and_empty_ones(gpu_lib, Hq, Hkv, D, lengths, causal):
    """Short ones are dealt out by 32 rows, long ones by 128, in one call: each row is done once."""
    import torch
    T = sum(lengths) + 2
    assert T // len(lengths) < 80 and (T // 128 + min(T, len(lengths))) * Hq >= 512
    q, k, v, dq, dk, dv = make(T, Hq, Hkv, D, "stacked")
    starts = bounds(lengths, 1)
    out = torch.full((T, Hq, D), 7.0, dtype=torch.float16, device="cuda")
    swm.prompt_attention(dq, dk, dv, ints(starts), causal=causal, out=out)
    ref, tol, rows = reference(q, k, v, starts, D ** -0.5, causal)
    check(out[torch.from_numpy(rows).cuda()], ref[rows], tol[rows])
    assert bool((out[0] == 7.0).all()) and bool((out[T - 1] == 7.0).all())
    n, at = max(lengths), int(starts[int(np.argmax(lengths))])
    dv[at + n - 70, 0, 1] = float("inf")  # of the long one, seen by its last rows or by all of it
    out = swm.prompt_attention(dq, dk, dv, ints(starts), causal=causal).double().cpu().numpy()
    hit = np.zeros((T, Hq, D), bool)
    hit[at + n - 70 if causal else at:at + n, :Hq // Hkv, 1] = True
    assert np.array_equal(~np.isfinite(out[rows]), hit[rows])
    assert np.all((np.abs(out - ref) <= tol)[rows[:, None, None] & ~hit])


@gpu
def test_starts_that_fall_among_many(gpu_lib):
    """Bounds that are not in order: rows of a sequence may be another's too, and nothing else is read or written."""
    import torch
    q, k, v, dq, dk, dv = make(900, 8, 2, 64)
    starts = np.array(([0, 700, 100] * 40) + [900], np.int32)  # 40 of 700 tokens, 39 of none, one of 800
    out = torch.full_like(dq, 3.0)
    swm.prompt_attention(dq, dk, dv, ints(starts), out=out)
    ref, tol, _ = reference(q, k, v, [0, 700], 0.125, True)
    check(out[:100], ref[:100], tol[:100])
    assert bool(torch.isfinite(out).all())


@gpu
@pytest.mark.parametrize("Hq,lengths,at", [(32, [40, 9] * 20, 25), (32, [40, 9] * 20, 39), (64, [150] * 30, 70),
                                           (64, [150] * 30, 149)])
@pytest.mark.parametrize("D", [64, 128])
def test_what_is_not_finite_in_large_batches(gpu_lib, Hq, lengths, at, D):
    """The same where blocks are a wave's and where tiles are small."""
    q, k, v, dq, dk, dv = make(sum(lengths), Hq, 2, D)
    starts = bounds(lengths)
    ref, tol, _ = reference(q, k, v, starts, D ** -0.5, True)
    dv[int(starts[2]) + at, 1, 5] = float("nan")
    hit = np.zeros(ref.shape, bool)
    hit[starts[2] + at:starts[3], Hq // 2:, 5] = True
    out = swm.prompt_attention(dq, dk, dv, ints(starts)).double().cpu().numpy()
    assert np.array_equal(np.isnan(out), hit)
    assert np.all(np.abs(out - ref)[~hit] <= tol[~hit])


@gpu
def test_a_key_that_no_row_can_score(gpu_lib):
    """A score of -inf has no weight; a row with nothing else gives zeros."""
    import torch
    q, k, v, dq, dk, dv = make(100, 1, 1, 64)
    dq.copy_(dq.abs() + 0.5)
    dk[0], dk[40] = -float("inf"), -float("inf")
    starts = ints([0, 100])
    out = swm.prompt_attention(dq, dk, dv, starts)
    q = dq.cpu().numpy()
    sees = np.tril(np.ones((100, 100), bool))
    sees[:, [0, 40]] = False
    k[[0, 40]] = 0
    ref, tol = attend(q[:, 0], k[:, 0], v[:, 0], 0.125, sees)
    check(out[:, 0], ref, tol)
    assert bool((out[0] == 0).all())


@gpu
def test_starts_outside_the_rows(gpu_lib):
    """Bounds that fall or lie outside are clamped; nothing else is read or written."""
    import torch
    q, k, v, dq, dk, dv = make(90, 2, 2, 64)
    out = torch.full_like(dq, 3.0)
    swm.prompt_attention(dq, dk, dv, ints([-5, 40, 20, 1000]), out=out)
    ref, tol, _ = reference(q, k, v, [0, 40, 40], 0.125, True)
    check(out[:20], ref[:20], tol[:20])  # rows 20 to 39 belong to two sequences
    ref, tol, _ = reference(q[20:], k[20:], v[20:], [0, 70], 0.125, True)
    check(out[40:], ref[20:], tol[20:])


@gpu
def test_graph_follows_starts_on_a_stream(gpu_lib):
    import torch
    q, k, v, dq, dk, dv = make(640, 4, 2, 128)
    starts, out = ints([0, 640, 640]), torch.zeros_like(dq)
    swm.prompt_attention(dq, dk, dv, starts, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        swm.prompt_attention(dq, dk, dv, starts, out=out)
    side = torch.cuda.Stream()
    for n in ([100, 540], [640, 0], [0, 1], [333, 300]):
        starts.copy_(ints(bounds(n)))
        out.zero_()
        graph.replay()
        want = torch.zeros_like(dq)
        side.wait_stream(torch.cuda.current_stream())
        swm.prompt_attention(dq, dk, dv, starts, out=want, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        ref, tol, rows = reference(q, k, v, bounds(n), 128 ** -0.5, True)
        check(out[: sum(n)], ref[: sum(n)], tol[: sum(n)], str(n))


@gpu
def test_offsets_past_32_bits(gpu_lib):
    """Rows a megabyte of elements apart: 4 GiB lie between tokens of one sequence."""
    import torch
    T, step = 2300, 1 << 20
    q, k, v, dq, dk, dv = make(T, 2, 1, 64)
    pool = torch.empty(T * step, dtype=torch.float16, device="cuda")
    wide = [pool[i * 64:].as_strided((T, 1, 64), (step, 64, 1)) for i in range(2)]
    wide[0].copy_(dk)
    wide[1].copy_(dv)
    starts = bounds([2250, 50])
    ref, tol, _ = reference(q, k, v, starts, 0.125, True)
    check(swm.prompt_attention(dq, *wide, ints(starts)), ref, tol)


@gpu
@pytest.mark.parametrize("Hq", [1, 3])
def test_as_many_sequences_as_there_may_be(gpu_lib, Hq):
    """65535 of them, of one token and none, two of three tokens and one of 600 at the end."""
    import torch
    n = np.arange(65535) % 2
    n[[5, 40000]], n[-1] = 3, 600
    T, starts = int(n.sum()), bounds(n)
    q, k, v, dq, dk, dv = make(T, Hq, 1, 8)
    out = swm.prompt_attention(dq, dk, dv, ints(starts))
    one = np.repeat(n == 1, n)
    assert np.array_equal(out.cpu().numpy()[one], np.broadcast_to(v, q.shape)[one])
    for b in (5, 40000, 65534):
        ref, tol, _ = reference(*(x[starts[b]:starts[b + 1]] for x in (q, k, v)), [0, n[b]], 8 ** -0.5, True)
        check(out[starts[b]:starts[b + 1]], ref, tol)
    with pytest.raises(swm.SwmError, match="UNSUPPORTED"):
        swm.prompt_attention(dq, dk, dv, ints(np.zeros(65537)))


@gpu
def test_no_tokens_and_no_sequences(gpu_lib):
    import torch
    q, k, v, dq, dk, dv = make(5, 2, 1, 64)
    assert swm.prompt_attention(dq[:0], dk[:0], dv[:0], ints([0, 0])).shape == (0, 2, 64)
    out = torch.full_like(dq, 2.0)
    swm.prompt_attention(dq, dk, dv, ints([0]), out=out)
    swm.prompt_attention(dq, dk, dv, ints([2, 2, 2]), out=out)
    assert bool((out == 2.0).all())


@gpu
@pytest.mark.parametrize("n", [9, 40])
def test_a_prompt_is_its_tokens_one_by_one(gpu_lib, n):
    """The decoding example: a prompt at once, and the same tokens as steps of another session."""
    import importlib.util
    import os
    import torch
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "pruned_decode.py")
    spec = importlib.util.spec_from_file_location("pruned_decode", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    y = m.Layer(hidden=256, ffn=520, heads=4, kv_heads=2, vocab=1003, seed=3)
    a, b = (m.Session(y, batch=3, budget=60, slack=4, recent=4, page_size=8) for _ in range(2))
    tokens = (torch.arange(3 * n, device="cuda") * 37 % 1003).view(3, n)
    ids, logp, entropy = a.prompt(tokens)
    for i in range(n):
        ids_b, logp_b, entropy_b = b.step(tokens[:, i])
    # both round every product's outputs to fp16; logits of rms 1 differ by 2^-7 at most, as against plain torch
    assert float((entropy - entropy_b).abs().max()) < 2.0**-6 and float((logp - logp_b).abs().max()) < 2.0**-6
    assert a.lengths.tolist() == b.lengths.tolist() == [n] * 3
    t = torch.arange(n, device="cuda")
    for x, z in ((a.k, b.k), (a.v, b.v), (a.positions.transpose(1, 2), b.positions.transpose(1, 2))):
        x, z = (c[s.table[:, t // 8].long(), t % 8] for c, s in ((x, a), (z, b)))
        assert float((x.float() - z.float()).abs().max()) < 2.0**-6
    # and on from there: the next step reads the prompt's rows
    (ids, logp, entropy), (ids_b, logp_b, entropy_b) = a.step(ids), b.step(ids)
    assert float((entropy - entropy_b).abs().max()) < 2.0**-6 and float((logp - logp_b).abs().max()) < 2.0**-6


@gpu
def test_binding_refuses(gpu_lib):
    import torch
    q, k, v, dq, dk, dv = make(8, 4, 2, 64)
    s = ints([0, 8])
    for bad in (dq.float(), dq[0], dq.cpu(), None):
        with pytest.raises(TypeError):
            swm.prompt_attention(bad, dk, dv, s)
    for a, b in ((dk[:4], dv[:4]), (dk, dv[:, :1]), (dk[..., :32], dv[..., :32])):
        with pytest.raises(ValueError):
            swm.prompt_attention(dq, a, b, s)
    for bad in (s.long(), s.cpu(), [0, 8]):
        with pytest.raises(TypeError):
            swm.prompt_attention(dq, dk, dv, bad)
    for bad in (s[:0], s.view(2, 1), ints([0, 0, 8, 8])[::2]):
        with pytest.raises(ValueError):
            swm.prompt_attention(dq, dk, dv, bad)
    with pytest.raises(ValueError):
        swm.prompt_attention(dq, dk, dv, s, out=torch.empty_like(dq)[:4])
    with pytest.raises(ValueError):
        swm.prompt_attention(dq.transpose(1, 2).contiguous().transpose(1, 2), dk, dv, s)
    for kw in (dict(out=torch.empty_like(dq[:1]).expand(8, 4, 64)), dict(scale=float("nan"))):
        with pytest.raises(swm.SwmError, match="INVALID"):
            swm.prompt_attention(dq, dk, dv, s, **kw)
    with pytest.raises(swm.SwmError, match="INVALID"):  # rows of keys that overlap
        swm.prompt_attention(dq, dk[:1].expand(8, 2, 64), dv, s)
    with pytest.raises(swm.SwmError, match="INVALID"):  # four heads over three
        swm.prompt_attention(dq, dk[:, :1].expand(8, 3, 64), dv[:, :1].expand(8, 3, 64), s)
    with pytest.raises(swm.SwmError, match="ALIGN"):
        odd = torch.zeros(8 * 4 * 64 + 4, dtype=torch.float16, device="cuda")[4:].view(8, 4, 64)
        swm.prompt_attention(odd, dk, dv, s)


@pytest.mark.parametrize("change,code", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(out=None), 1), (dict(starts=None), 1),
    (dict(tokens=-1), 1), (dict(batch=-1), 1), (dict(heads=0), 1), (dict(q_heads=0), 1), (dict(q_heads=3), 1),
    (dict(dim=0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("-inf")), 1), (dict(q_token=-8), 1),
    (dict(k_head=-8), 1), (dict(out_head=-64), 1), (dict(k_token=56), 1), (dict(v_token=0), 1),
    (dict(out_token=128, out_head=32), 1), (dict(out_token=64, out_head=64), 1), (dict(out_token=0), 1),
    (dict(q=4104), 3), (dict(k=4104), 3), (dict(v=4100), 3), (dict(q_token=260), 3), (dict(v_head=4), 3),
    (dict(dim=60), 8), (dict(dim=264, k_token=1024, v_token=1024, out_token=2048, out_head=512), 8),
    (dict(batch=65536), 8), (dict(q_heads=65536), 8), (dict(tokens=(1 << 31) - 65536), 8),
    (dict(k_token=1 << 23), 8), (dict(tokens=1 << 30, q_heads=4), 8),
    (dict(tokens=0, q=None), 0), (dict(batch=0, starts=None), 0),
])
def test_call_refusals(change, code):
    lib = swm.load()
    a = dict(q=4096, q_token=256, q_head=64, k=8192, k_token=128, k_head=64, v=12288, v_token=128, v_head=64,
             tokens=16, q_heads=4, heads=2, dim=64, starts=4096, batch=2, scale=0.125, causal=1, out=16384,
             out_token=256, out_head=64, stream=None)
    a.update(change)
    assert lib.swm_prompt_attention(*a.values()) == code
