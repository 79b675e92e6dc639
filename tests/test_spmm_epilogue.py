"""spmm_epilogue against act(W X + b) + R in 64 bits on every route of the product.

Tolerance: the products of fp16 numbers are exact in fp32 and their sum, in any order, is off by at most
K 2^-24 sum |w x| =: E; adding the bias by 2^-24 more of the result.  The activations have slopes below 1.13 and are
themselves off by at most 2^-18 of their value; the result is rounded once to fp16 (2^-11 relative, 2^-25 below the
normal range).
"""
import ctypes

import numpy as np
import pytest

import sparse_weight_matmul_amd as swm
import swm_workloads as wl

gpu = pytest.mark.gpu

ACTS = ["none", "relu", "silu", "gelu"]


def act64(act, y):
    from scipy.special import erfc
    return {"none": lambda: y, "relu": lambda: np.maximum(y, 0), "silu": lambda: y / (1 + np.exp(-y)),
            "gelu": lambda: y * 0.5 * erfc(-y / np.sqrt(2))}[act]()


def check(Y, W, X, bias, act, residual):
    W64, X64 = W.astype(np.float64), X.astype(np.float64)
    y = X64 @ W64.T
    E = W.shape[1] * 2.0**-24 * (np.abs(X64) @ np.abs(W64).T)
    if bias is not None:
        y = y + bias.astype(np.float64)
    a = act64(act, y)
    want = a if residual is None else a + residual.astype(np.float64)
    tol = 1.13 * (E + 2.0**-24 * np.abs(y)) + 2.0**-18 * np.abs(a) + 2.0**-11 * np.abs(want) + 2.0**-25
    got = Y.double().cpu().numpy()
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), float(np.max(np.abs(got - want) - tol)), np.argwhere(bad)[:3].tolist())


def case(M, K, N, seed=0, mask=None, scale=0.08):
    r = np.random.default_rng([seed, M, K, N])
    W = (scale * r.standard_normal((M, K))).astype(np.float16)
    W[~(r.random((M, K)) < 0.5 if mask is None else mask(W))] = 0
    X = r.standard_normal((N, K)).astype(np.float16)
    return W, X, r.standard_normal(M).astype(np.float16), r.standard_normal((N, M)).astype(np.float16)


def t(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def workspace(f, N):
    import torch
    need = swm.spmm_epilogue_workspace_bytes(f, N)
    assert need >= swm.spmm_workspace_bytes(f, N)
    return torch.empty(need, dtype=torch.uint8, device="cuda") if need else None


SHAPES = [
    # M, K, N
    (300, 520, 1), (300, 520, 4), (17, 64, 7), (300, 520, 16), (4096, 1024, 13),     # straight-line decode
    (300, 520, 17), (300, 520, 32),                                                  # two groups of 16 tokens
    (33, 77, 1), (33, 77, 20), (33, 77, 40), (1, 1, 1),                              # unaligned: looped, in slices
    (300, 520, 33), (300, 520, 200), (1001, 264, 130),                               # slices, on-chip, expanded
    (4096, 1024, 100), (2000, 4096, 255), (130, 64, 64), (5000, 200, 37),
    (1001, 2056, 130), (391, 3440, 60), (130, 8200, 513), (17, 1096, 1023), (2049, 1928, 300),  # K split
    (300, 520, 257), (260, 136, 1027),                                               # expanded, 128 x 128 blocks
    (4096, 256, 2048), (4099, 128, 3000), (8192, 64, 4096),                          # larger blocks
    (707, 480, 304), (885, 72, 174), (4096, 4096, 73), (132, 2048, 1000),            # rows not aligned for 8 or 16 bytes
    (8203, 64, 2050), (4200, 72, 4100),                                              # and a launch for the last rows
]


@pytest.mark.parametrize("where", ["bias", "residual", "Y"])
def test_operands_on_another_device_are_refused(where):
    import torch

    class OnGpu(torch.Tensor):
        is_cuda = property(lambda self: True)
        device = property(lambda self: torch.device("cuda", self.at))

        def get_device(self):
            return self.at

    class Fmt:
        M, K, _h = 24, 16, None

    def made(at, *shape):
        x = torch.zeros(shape, dtype=torch.float16).as_subclass(OnGpu)
        x.at = at
        return x

    a = {"bias": made(0, 24), "residual": made(0, 4, 24), "Y": made(0, 4, 24)}
    a[where] = made(1, *a[where].shape)
    with pytest.raises(ValueError, match=f"{where} must be on cuda:0"):
        swm.spmm_epilogue(Fmt, made(0, 4, 16), **a)


@gpu
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_routes(gpu_lib, M, K, N):
    import torch
    W, X, b, R = case(M, K, N)
    f = swm.sparse_compress(W)
    ws, Xd, bd, Rd = workspace(f, N), t(X), t(b), t(R)
    for act in ACTS:
        for bias, res in ((True, True), (True, False), (False, True)):
            Y = torch.full((N, M), float("nan"), dtype=torch.float16, device="cuda")
            swm.spmm_epilogue(f, Xd, bd if bias else None, act, Rd if res else None, ws, Y)
            check(Y, W, X, b if bias else None, act, R if res else None)
    a = swm.spmm_epilogue(f, Xd, workspace=ws)
    check(a, W, X, None, "none", None)
    if not 32 < N < 1024:
        assert torch.equal(a, swm.spmm_ws(f, Xd, ws))
    check(swm.spmm_epilogue(f, Xd, bd, "silu", Rd), W, X, b, "silu", R)  # a workspace of its own
    if 32 < N < 256:  # one that is too small takes the expansion off the choice
        small = torch.empty(16, dtype=torch.uint8, device="cuda")
        check(swm.spmm_epilogue(f, Xd, bd, "silu", Rd, small), W, X, b, "silu", R)
    c = swm.spmm_epilogue(f, Xd, bd, "gelu", Rd, ws)
    assert torch.equal(c, swm.spmm_epilogue(f, Xd, bd, "gelu", Rd, ws))
    inplace = Rd.clone()  # the residual stream updated in place
    swm.spmm_epilogue(f, Xd, bd, "gelu", inplace, ws, inplace)
    assert torch.equal(c, inplace)


@gpu
@pytest.mark.parametrize("M,K,N", [(512, 64, 60), (512, 512, 512), (1000, 264, 400), (512, 72, 1500)])
@pytest.mark.parametrize("aligned", ["residual", "output", "neither"])
def test_rows_of_unlike_alignment(gpu_lib, M, K, N, aligned):
    import torch
    W, X, b, R = case(M, K, N)
    f = swm.sparse_compress(W)
    res = torch.zeros((N, M + 24), dtype=torch.float16, device="cuda")
    at = 0 if aligned == "residual" else 3
    res = res[:, at:at + M]
    res.copy_(t(R))
    out = torch.full((N, M + 24), 7.0, dtype=torch.float16, device="cuda")
    at = 8 if aligned == "output" else 5
    swm.spmm_epilogue(f, t(X), t(b), "silu", res, None, out[:, at:at + M])
    check(out[:, at:at + M], W, X, b, "silu", R)
    assert bool((out[:, :at] == 7).all()) and bool((out[:, at + M:] == 7).all())


@gpu
@pytest.mark.parametrize("M,K,N", [(1001, 2056, 130), (130, 8200, 513)])
def test_split_of_k(gpu_lib, M, K, N):
    import torch
    W, X, b, R = case(M, K, N)
    f = swm.sparse_compress(W)
    need = swm.spmm_epilogue_workspace_bytes(f, N)
    assert 0 < need and need != M * K * 2  # the sums of the splits, not W
    guard = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    Y = swm.spmm_epilogue(f, t(X), t(b), "silu", t(R), guard[:need])
    check(Y, W, X, b, "silu", R)
    assert bool((guard[need:] == 0xA5).all())  # nothing past what was asked for
    assert torch.equal(Y, swm.spmm_epilogue(f, t(X), t(b), "silu", t(R), guard[:need]))
    less = swm.spmm_epilogue(f, t(X), t(b), "silu", t(R), guard[:need - 16])  # one split fewer, or another route
    check(less, W, X, b, "silu", R)


@gpu
@pytest.mark.parametrize("N", [1, 8, 16, 32])
def test_looped_decode(gpu_lib, N, monkeypatch):
    W, X, b, R = case(500, 1032, N)
    monkeypatch.setenv("SWM_DECODE_PATH", "loop")
    f = swm.sparse_compress(W)
    for act in ACTS:
        check(swm.spmm_epilogue(f, t(X), t(b), act, t(R)), W, X, b, act, R)


@gpu
@pytest.mark.parametrize("kept", ["2:4", "half"])
@pytest.mark.parametrize("M,N", [(4096, 1024), (1000, 1100), (8192, 4096)])
def test_sparse_matrix_cores(gpu_lib, kept, M, N):
    W, X, b, R = case(M, 256, N, mask=wl.prune_2_4_mask if kept == "2:4" else None)
    f = swm.sparse_compress(W, smfmac=True)
    assert swm.spmm_workspace_bytes(f, N) == 0
    for act, bias, res in (("gelu", b, R), ("silu", None, R), ("relu", b, None), ("none", b, R)):
        Y = swm.spmm_epilogue(f, t(X), None if bias is None else t(bias), act, None if res is None else t(res))
        check(Y, W, X, bias, act, res)


@gpu
@pytest.mark.parametrize("N", [3, 20, 100, 1200])
def test_strides_and_alignment(gpu_lib, N):
    import torch
    M, K = 301, 264
    W, X, b, R = case(M, K, N)
    f = swm.sparse_compress(W)
    ws = workspace(f, N)
    for off, pad in ((0, 3), (1, 6), (2, 5), (3, 4), (4, 11)):
        bias = torch.zeros(M + off, dtype=torch.float16, device="cuda")[off:]
        bias.copy_(t(b))
        res = torch.full((N, M + pad + off), float("nan"), dtype=torch.float16, device="cuda")
        res[:, off:off + M] = t(R)
        out = torch.full((N, M + pad), 7.0, dtype=torch.float16, device="cuda")
        swm.spmm_epilogue(f, t(X), bias, "silu", res[:, off:off + M], ws, out[:, :M])
        check(out[:, :M], W, X, b, "silu", R)
        assert bool((out[:, M:] == 7).all())


@gpu
def test_activations_past_4_gib(gpu_lib):
    import torch
    # token rows 8.4 million elements apart: beyond the 32-bit offsets of the LDS-direct kernel
    M, K, N, ld = 384, 64, 260, 8400000
    W, X, b, R = case(M, K, N)
    big = torch.empty((N - 1) * ld + K, dtype=torch.float16, device="cuda").as_strided((N, K), (ld, 1))
    big.copy_(t(X))
    f = swm.sparse_compress(W)
    ws = workspace(f, N)
    assert ws is not None
    for act in ACTS:
        check(swm.spmm_epilogue(f, big, t(b), act, t(R), ws), W, X, b, act, R)


@gpu
def test_extreme_sums(gpu_lib):
    import torch
    W = np.zeros((16, 64), np.float16)
    W[:, 0] = 1
    X = np.zeros((12, 64), np.float16)
    X[:, 0] = [-60000, -1000, -20, -9, -6, -3, -1e-4, 0, 1e-4, 3, 20, 60000]
    f = swm.sparse_compress(W)
    for act in ACTS:
        check(swm.spmm_epilogue(f, t(X), act=act), W, X, None, act, None)
    # the tail of GELU keeps its relative accuracy down to the subnormal numbers
    X[:, 0] = -np.array([2, 2.5, 3, 3.5, 4, 4.25, 4.5, 4.75, 5, 5.25, 5.5, 5.75])
    check(swm.spmm_epilogue(f, t(X), act="gelu"), W, X, None, "gelu", None)
    X[0, 0] = np.nan
    for act in ACTS:
        assert bool(torch.isnan(swm.spmm_epilogue(f, t(X[:1]), act=act, bias=t(np.ones(16, np.float16)))).all())
    X[0, 0] = np.inf
    Y = swm.spmm_epilogue(f, t(X[:1]), act="gelu", bias=t(np.ones(16, np.float16)))
    assert bool((Y == float("inf")).all())


@gpu
def test_graph_and_stream(gpu_lib):
    import torch
    W, X, b, R = case(2048, 512, 16)
    f = swm.sparse_compress(W)
    Xd, bd, Rd, Y = t(X), t(b), t(R), torch.empty((16, 2048), dtype=torch.float16, device="cuda")
    swm.spmm_epilogue(f, Xd, bd, "silu", Rd, None, Y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        swm.spmm_epilogue(f, Xd, bd, "silu", Rd, None, Y)
    for k in range(3):
        Rd.mul_(0.5)
        eager = swm.spmm_epilogue(f, Xd, bd, "silu", Rd)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, eager)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    swm.spmm_epilogue(f, Xd, bd, "silu", Rd, None, Y, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(Y, eager)


@gpu
def test_refusals(gpu_lib):
    import torch
    W, X, b, R = case(64, 64, 4)
    f = swm.sparse_compress(W)
    Xd, bd, Rd = t(X), t(b), t(R)
    with pytest.raises(ValueError):
        swm.spmm_epilogue(f, Xd, act="tanh")
    with pytest.raises(TypeError):
        swm.spmm_epilogue(f, Xd, bias=bd.float())
    with pytest.raises(TypeError):
        swm.spmm_epilogue(f, Xd, bias=bd[:5])
    with pytest.raises(ValueError):
        swm.spmm_epilogue(f, Xd, residual=Rd[:3])
    lib, p, q = swm.load(), Xd.data_ptr(), Rd.data_ptr()
    y = torch.zeros((4, 64), dtype=torch.float16, device="cuda").data_ptr()
    s = torch.cuda.current_stream().cuda_stream
    assert lib.swm_spmm_epilogue(f._h, p, 64, y, 64, 4, None, 4, None, 0, None, 0, s) == 1
    assert lib.swm_spmm_epilogue(f._h, p, 64, y, 64, 4, None, -1, None, 0, None, 0, s) == 1
    assert lib.swm_spmm_epilogue(f._h, p, 64, y, 64, 4, None, 0, q, 63, None, 0, s) == 1
    assert lib.swm_spmm_epilogue(f._h, p, 64, y, 64, 4, None, 0, y, 65, None, 0, s) == 1
    assert lib.swm_spmm_epilogue(f._h, p, 63, y, 64, 4, None, 1, q, 64, None, 0, s) == 1
    assert lib.swm_spmm_epilogue(f._h, p, 64, y, 64, 0, None, 1, q, 64, None, 0, s) == 1
    long = torch.zeros((40, 64), dtype=torch.float16, device="cuda")
    out = torch.zeros_like(long)
    p, y = long.data_ptr(), out.data_ptr()
    assert lib.swm_spmm_epilogue(f._h, p, 64, y, 64, 40, None, 1, None, 0, None, 4096, s) == 1
    assert lib.swm_spmm_epilogue(f._h, p, 64, y, 64, 40, None, 1, None, 0, q + 2, 4096, s) == 3
    assert lib.swm_spmm_epilogue(f._h, p, 63, y, 64, 40, None, 1, None, 0, None, 0, s) == 1
    assert lib.swm_spmm_epilogue(f._h, p, 64, y, 63, 40, None, 1, None, 0, None, 0, s) == 1


def test_null_handle():
    lib = swm.load()
    assert lib.swm_spmm_epilogue_workspace_bytes(None, 100) == 0
    assert lib.swm_spmm_epilogue(None, 4096, 64, 8192, 64, 4, None, 0, None, 0, None, 0, None) == 1
