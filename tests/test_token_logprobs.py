"""token_logprobs against log softmax in 64 bits.

Tolerances: log p = (x - m) - log l.  The exponent x log2(e) - m log2(e) is one
fused multiply-add of fp32 numbers: off by 2^-24 of itself and, in common with
every other logit of the row, by the rounding of the base (2^-24 |m|, which
cancels between the two terms) and of log2(e) (2^-25 of x - m).  An exponential
is off by 2^-22 of itself and l, whose rounding grows with the running sum, by
2^-18 at most for the lengths here.  With d the larger of 1 and |log p|, an
error of 2^-18 + 2^-21 d (the entropy, a sum of p log p, the same with d = 1 +
its own log range).
"""
import numpy as np
import pytest

import sparse_weight_matmul_amd as swm

gpu = pytest.mark.gpu


def reference(x, top):
    x = x.astype(np.float64)
    with np.errstate(invalid="ignore", divide="ignore"):
        m = x.max(-1, keepdims=True)
        m0 = np.where(np.isfinite(m), m, 0)
        z = np.exp(x - m0).sum(-1, keepdims=True)
        lp = np.where(z > 0, x - m0 - np.log(np.where(z > 0, z, 1)), -np.inf)
        p = np.exp(lp)
        h = -np.where(p > 0, p * lp, 0).sum(-1)
    ids = np.argsort(-x, axis=-1, kind="stable")[:, :top]
    return lp, h, ids


def rows(kind, N, V, dtype, seed=0):
    r = np.random.default_rng([seed, N, V])
    x = 2.5 * r.standard_normal((N, V))
    if kind == "masked":
        x[r.random((N, V)) < 0.6] = -np.inf
        x[::3] = -np.inf                      # nothing left
        x[1::3, : V - 1] = -np.inf            # one token left, the last
    elif kind == "ties":
        x = r.integers(-2, 3, (N, V)).astype(float)
        x[x == 0] *= r.choice([-1.0, 1.0], int((x == 0).sum()))  # zeros of both signs are equal
    elif kind == "constant":
        x[:] = 1.5
        x[::2] = -3.0
    elif kind == "large":
        x = x * 4000
    elif kind == "descending":
        x = np.tile(np.linspace(30, -30, V), (N, 1))
    elif kind == "stripes":                   # one place of each 8192 holds all the large ones: one thread's
        x[:, ::8192] = 20 + r.random((N, len(range(0, V, 8192))))
    return x.astype(dtype)


CASES = [
    (1, 1, 1, "plain"), (3, 7, 64, "plain"), (5, 100, 20, "plain"), (1, 32000, 5, "plain"), (4, 32001, 0, "plain"),
    (7, 1029, 64, "plain"), (2, 131071, 32, "plain"), (33, 4099, 1, "plain"), (300, 517, 3, "plain"),
    (6, 50021, 20, "masked"), (6, 300, 64, "masked"), (4, 20000, 64, "ties"), (4, 900, 40, "ties"),
    (4, 50000, 33, "constant"), (4, 1500, 64, "constant"), (3, 9999, 10, "large"), (3, 40000, 64, "descending"),
    (2, 131072, 17, "stripes"), (2, 1100, 64, "constant"), (2, 1030, 64, "plain"),
]


@gpu
@pytest.mark.parametrize("N,V,top,kind", CASES)
@pytest.mark.parametrize("dtype", [np.float16, np.float32])
def test_against_64_bits(gpu_lib, N, V, top, kind, dtype):
    import torch
    x = rows(kind, N, V, dtype)
    t = np.random.default_rng(1).integers(0, V, N)
    X, T = torch.from_numpy(x).cuda(), torch.from_numpy(t).cuda()
    logp, ent, ids, lps = swm.token_logprobs(X, T, top=top)
    lp, h, want_ids = reference(x, top)
    want = lp[np.arange(N), t]
    close(logp.cpu().numpy(), want, np.maximum(1, np.abs(want)))
    spread = 1 + np.log(V) + np.where(np.isfinite(lp), np.exp(lp) * np.abs(np.where(np.isfinite(lp), lp, 0)), 0).sum(-1)
    close(ent.cpu().numpy(), h, spread)
    if top:
        k = min(top, V)
        assert np.array_equal(ids.cpu().numpy()[:, :k], want_ids)
        want = np.take_along_axis(lp, want_ids, -1)
        close(lps.cpu().numpy()[:, :k], want, np.maximum(1, np.abs(want)))
        assert bool((ids[:, k:] == -1).all()) and bool((lps[:, k:] == -float("inf")).all())
    else:
        assert ids is None and lps is None
    again = swm.token_logprobs(X, T.int(), top=top)  # the same bits, whatever the targets' type
    for a, b in zip((logp, ent, ids, lps), again):
        assert a is None or torch.equal(a, b)


def close(got, want, d):
    fin = np.isfinite(want)
    assert np.array_equal(got[~fin], want[~fin].astype(np.float32), equal_nan=True)
    with np.errstate(invalid="ignore"):
        bad = (np.abs(got - want) > 2.0**-18 + 2.0**-21 * d) & fin
    assert not bad.any(), (int(bad.sum()), float(np.abs(got - want)[fin].max()))


@gpu
def test_strides_alignment_and_targets(gpu_lib):
    import torch
    x = rows("plain", 6, 1000, np.float16)
    lp, h, ids = reference(x, 9)
    wide = torch.full((6, 1017), float("nan"), dtype=torch.float16, device="cuda")
    t = torch.tensor([0, 999, -1, -100, 1000, 5], device="cuda")
    for off in range(9):  # every alignment of a row's start
        wide.fill_(float("nan"))
        wide[:, off:off + 1000] = torch.from_numpy(x).cuda()
        logp, ent, got, _ = swm.token_logprobs(wide[:, off:off + 1000], t, top=9)
        assert np.array_equal(got.cpu().numpy(), ids)
        logp = logp.cpu().numpy()
        assert np.all(logp[2:4] == 0) and np.isnan(logp[4])
        close(logp[[0, 1, 5]], lp[[0, 1, 5], [0, 999, 5]], 8.0)
        close(ent.cpu().numpy(), h, 8.0)
    none, ent, _, _ = swm.token_logprobs(wide[:, 8:1008])
    assert none is None
    close(ent.cpu().numpy(), h, 8.0)
    a = swm.token_logprobs(wide[:0, :1000], t[:0], top=2)
    assert a[0].shape == (0,) and a[2].shape == (0, 2)


@gpu
def test_infinities_and_nan(gpu_lib):
    import torch
    x = np.zeros((4, 3000), np.float32)
    x[0, 77], x[1, 2999] = np.nan, np.inf
    x[2, 5] = -np.nan
    x[3] = np.linspace(-1, 1, 3000)
    logp, ent, ids, lps = swm.token_logprobs(torch.from_numpy(x).cuda(), torch.tensor([3, 3, 3, 3]).cuda(), top=3)
    assert bool(torch.isnan(logp[:3]).logical_or(logp[:3] == -float("inf")).all())
    assert bool(torch.isnan(ent[:3]).all())
    assert bool(((ids >= 0) & (ids < 3000)).all())
    lp, h, want = reference(x[3:], 3)
    assert np.array_equal(ids[3:].cpu().numpy(), want)
    close(ent[3:].cpu().numpy(), h, 8.0)


def closer(got, want, d):
    """close, and a number wherever one is wanted."""
    assert np.isfinite(got[np.isfinite(want)]).all()
    close(got, want, d)


@gpu
@pytest.mark.parametrize("N,V,top,kind", CASES)
@pytest.mark.parametrize("dtype", [np.float16, np.float32])
def test_numbers_where_the_definition_has_them(gpu_lib, N, V, top, kind, dtype):
    import torch
    x = rows(kind, N, V, dtype)
    t = np.random.default_rng(1).integers(0, V, N)
    logp, ent, ids, lps = swm.token_logprobs(torch.from_numpy(x).cuda(), torch.from_numpy(t).cuda(), top=top)
    lp, h, want_ids = reference(x, top)
    got = [(logp, lp[np.arange(N), t]), (ent, h)]
    if top:
        got.append((lps[:, :min(top, V)], np.take_along_axis(lp, want_ids, -1)))
    for a, b in got:
        assert np.array_equal(np.isfinite(a.cpu().numpy()), np.isfinite(b))


@gpu
@pytest.mark.parametrize("N,V,top", [(5, 3, 1), (5, 7, 20), (5, 300, 5), (5, 900, 64), (5, 1500, 1), (5, 50021, 20),
                                     (5, 131072, 64), (300, 517, 3), (300, 9000, 20)])
@pytest.mark.parametrize("dtype", [np.float16, np.float32])
def test_rows_of_nan(gpu_lib, N, V, top, dtype):
    """Rows of nothing but NaN, of a few numbers among NaN, half and one: NaN throughout, the top tokens in the
    order NaN first, then by size, equal ones by the lower index."""
    import torch
    x = rows("plain", N, V, dtype)
    r = np.random.default_rng(V)
    x[0::5] = np.nan
    some = x[1::5]
    some[:, r.permutation(V)[min(3, V // 2):]] = np.nan
    half = x[2::5]
    half[r.random(half.shape) < 0.5] = np.nan
    half[:, 0] = np.nan
    x[3::5] = -np.inf
    x[3::5, V // 2] = np.nan
    t = np.where(np.arange(N) % 2, V - 1, 0)
    logp, ent, ids, lps = swm.token_logprobs(torch.from_numpy(x).cuda(), torch.from_numpy(t).cuda(), top=top)
    k = min(top, V)
    key = np.where(np.isnan(x), np.inf, x).astype(np.float64)  # no +inf among them
    assert np.array_equal(ids.cpu().numpy()[:, :k], np.argsort(-key, axis=-1, kind="stable")[:, :k])
    bad = np.isnan(x).any(-1)
    assert bad[np.arange(N) % 5 < 4].all() and not bad[4::5].any()
    for got in (logp, ent, lps[:, :k]):
        assert np.isnan(got.cpu().numpy()[bad]).all()
    lp, h, _ = reference(x[4::5], k)
    closer(logp.cpu().numpy()[4::5], lp[np.arange(len(lp)), t[4::5]], 16.0)
    closer(ent.cpu().numpy()[4::5], h, 1 + np.log(V) + h)


@gpu
@pytest.mark.parametrize("dtype,V,threads,top", [(np.float16, 2040, 64, 32), (np.float32, 1020, 64, 32),
                                                 (np.float32, 1 << 20, 1024, 3)])
@pytest.mark.parametrize("fill", [np.nan, 60.0])
def test_more_above_the_bound_than_the_list_holds(gpu_lib, dtype, V, threads, top, fill):
    """Fewer than `top` threads of a row hold hundreds of logits above all others, the first logit among them:
    found in rounds over the row."""
    import torch
    x = rows("plain", 1, V, dtype)
    vec = 16 // np.dtype(dtype).itemsize
    x[0, np.arange(V) // vec % threads < top - 1] = fill
    assert np.count_nonzero(x[0] != x[0]) + np.count_nonzero(x[0] == 60) > 448
    x[0, 1::5] += dtype(0.5)  # unlike sizes among the numbers
    _, ent, ids, lps = swm.token_logprobs(torch.from_numpy(x).cuda(), top=top)
    key = np.where(np.isnan(x), np.inf, x).astype(np.float64)
    want = np.argsort(-key, axis=-1, kind="stable")[:, :top]
    assert np.array_equal(ids.cpu().numpy(), want)
    if np.isnan(fill):
        assert bool(torch.isnan(lps).all()) and bool(torch.isnan(ent).all())
    else:
        lp, h, _ = reference(x, top)
        closer(lps.cpu().numpy(), np.take_along_axis(lp, want, -1), 16.0)
        closer(ent.cpu().numpy(), h, 1 + np.log(V) + h)


@gpu
@pytest.mark.parametrize("N,V,top", [(8, 300, 5), (8, 5001, 20), (8, 50021, 0), (8, 140000, 64), (2100, 700, 0),
                                     (300, 3001, 3)])
@pytest.mark.parametrize("dtype,fill", [(np.float16, x) for x in (-1e4, -65504.0, 6e4)] + [
    (np.float32, x) for x in (-1e4, -1.6777e7, -1.6778e7, -1e9, -1e10, -1e12, -1e20, -1e30, -1e37, -2.4e38,
                              float(np.finfo(np.float32).min), 1.6777e7, 1.6778e7, 1e10, 3e38)])
def test_finite_masks(gpu_lib, fill, N, V, top, dtype):
    """Tokens ruled out by a large finite number: single ones, ranges, all but one token, all of a row; and single
    logits as large the other way.  The definition gives finite numbers wherever they fit 32 bits."""
    import torch
    x = rows("plain", N, V, dtype)
    r = np.random.default_rng(V)
    part = x[0::8]
    part[r.random(part.shape) < 0.5] = fill
    x[1::8, :V // 3] = fill           # whole vectors, threads and waves of them, first
    x[2::8, V // 2:] = fill           # and last: a padded vocabulary
    x[3::8] = fill                    # the whole row
    x[4::8, 1:] = fill                # all but one
    x[5::8, V // 2] = -fill           # one token that takes all
    x[6::8] = fill
    x[6::8, ::7] = fill / 2           # two sizes of them
    t = np.where(np.arange(N) % 2, V - 1, 0)
    logp, ent, ids, lps = swm.token_logprobs(torch.from_numpy(x).cuda(), torch.from_numpy(t).cuda(), top=top)
    lp, h, want_ids = reference(x, top)
    lp = np.where(np.abs(lp) > np.finfo(np.float32).max, -np.inf, lp)
    want = lp[np.arange(N), t]
    closer(logp.cpu().numpy(), want, np.maximum(1, np.abs(want)))
    spread = 1 + np.log(V) + np.where(np.isfinite(lp), np.exp(lp) * np.abs(np.where(np.isfinite(lp), lp, 0)), 0).sum(-1)
    closer(ent.cpu().numpy(), h, spread)
    if top:
        assert np.array_equal(ids.cpu().numpy(), want_ids)
        want = np.take_along_axis(lp, want_ids, -1)
        closer(lps.cpu().numpy(), want, np.maximum(1, np.abs(want)))


@gpu
def test_graph_and_stream(gpu_lib):
    import torch
    X, T = torch.from_numpy(rows("plain", 9, 3333, np.float16)).cuda(), torch.arange(9, device="cuda")
    swm.token_logprobs(X, T, top=4)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = swm.token_logprobs(X, T, top=4)
    for seed in (1, 2, 3):
        X.copy_(torch.from_numpy(rows("plain", 9, 3333, np.float16, seed)))
        eager = swm.token_logprobs(X, T, top=4)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = swm.token_logprobs(X, T, top=4, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(out, other))


@gpu
def test_binding_refuses(gpu_lib):
    import torch
    X = torch.zeros((4, 100), dtype=torch.float16, device="cuda")
    T = torch.zeros(4, dtype=torch.int64, device="cuda")
    with pytest.raises(TypeError):
        swm.token_logprobs(X.double(), T)
    with pytest.raises(TypeError):
        swm.token_logprobs(X, T.float())
    with pytest.raises(ValueError):
        swm.token_logprobs(X, T[:3])
    with pytest.raises(ValueError):
        swm.token_logprobs(X.t(), torch.zeros(100, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):  # rows that overlap
        swm.token_logprobs(X.view(-1).as_strided((4, 100), (50, 1)), T)
    with pytest.raises(swm.SwmError):
        swm.token_logprobs(X, T, top=65)
    with pytest.raises(swm.SwmError):
        swm.token_logprobs(X, T, top=-1)


@pytest.mark.parametrize("change,code", [
    (dict(logits=None), 1), (dict(N=-1), 1), (dict(V=0), 1), (dict(ld=99), 1), (dict(top=-1), 1),
    (dict(logp=None), 1), (dict(top_ids=None), 1), (dict(top_logp=None), 1), (dict(logits=4097), 3),
    (dict(fp32=1, logits=4098), 3), (dict(top=65), 8), (dict(V=1 << 31, ld=1 << 31), 8), (dict(N=1 << 22), 8),
])
def test_call_refusals(change, code):
    a = dict(logits=4096, fp32=0, N=4, V=100, ld=100, targets=8192, wide=1, logp=12288, entropy=16384, top=5,
             top_ids=20480, top_logp=24576, stream=None)
    a.update(change)
    assert swm.load().swm_token_logprobs(*a.values()) == code


def test_nothing_to_do():
    assert swm.load().swm_token_logprobs(None, 0, 0, 100, 100, None, 0, None, None, 0, None, None, None) == 0
