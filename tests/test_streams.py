"""The serving operators on a stream that is not the current one: whose memory their new tensors are."""
import contextlib

import numpy as np
import pytest

import sparse_weight_matmul_amd as swm

gpu = pytest.mark.gpu


@pytest.mark.parametrize("make", ["_empty", "_empty_like", "_workspace"])
def test_new_tensors_are_made_on_the_stream(monkeypatch, make):
    import torch
    now, made, kept = ["current"], [], []

    @contextlib.contextmanager
    def stream(s):
        now.append(s)
        yield
        now.pop()

    real_empty, real_like = torch.empty, torch.empty_like
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now[-1])
    monkeypatch.setattr(torch, "empty", lambda *a, **k: made.append(now[-1]) or real_empty(*a, **k))
    monkeypatch.setattr(torch, "empty_like", lambda *a, **k: made.append(now[-1]) or real_like(*a, **k))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: kept.append(s))
    cpu, like = torch.device("cpu"), torch.zeros(4)
    call = {"_empty": lambda s: swm._empty((2, 3), torch.float16, cpu, s), "_empty_like": lambda s: swm._empty_like(like, s),
            "_workspace": lambda s: swm._workspace(None, 64, cpu, s)[0]}[make]
    call("side")
    assert made == ["side"]       # not a block that the current stream may still be reading
    assert kept == ["current"]    # and not given to another call while the current stream reads it
    for same in (None, "current"):
        made.clear(), kept.clear()
        call(same)
        assert made == ["current"] and not kept


def calls():
    """(name, call(stream) -> tensors made by it) of every operator."""
    import torch
    r = np.random.default_rng(0)
    dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    k = dev(r.standard_normal((12, 16, 2, 64)).astype(np.float16))
    cache = swm.PagedCache(k, k.clone(), dev(np.arange(12, dtype=np.int32).reshape(2, 6)),
                           dev(np.array([90, 50], np.int32)))
    q = dev(r.standard_normal((2, 4, 64)).astype(np.float16))
    w, pos = dev(r.random((12, 2, 16)).astype(np.float32)), dev(np.arange(384, dtype=np.int32).reshape(12, 2, 16))
    wo, po = torch.zeros_like(w), torch.zeros_like(pos)
    f = swm.sparse_compress((r.standard_normal((256, 512)) * (r.random((256, 512)) < 0.5)).astype(np.float16))
    x, bias = dev(r.standard_normal((80, 512)).astype(np.float16)), dev(r.standard_normal(256).astype(np.float16))
    logits, target = dev(r.standard_normal((5, 3000)).astype(np.float16)), dev(np.arange(5))
    return [("attention", lambda s: [swm.paged_attention(cache, q, stream=s)]),
            ("attention, q strided", lambda s: [swm.paged_attention(cache, q.transpose(0, 1)[:2].transpose(0, 1)[:, :2],
                                                                    stream=s)]),
            ("evict", lambda s: list(swm.kv_evict(cache, w, pos, 40, 4, wo, po, stream=s))),
            ("product", lambda s: [swm.spmm_epilogue(f, x, bias, "silu", stream=s)]),
            ("logprobs", lambda s: list(swm.token_logprobs(logits, target, top=3, stream=s)))]


@gpu
def test_outputs_are_not_the_current_streams_memory(gpu_lib):
    import torch
    for name, call in calls():
        want = call(None)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        # blocks of the outputs' sizes that the current stream has just given back
        given = [torch.empty_like(t) for t in want for _ in range(4)]
        free = {t.data_ptr() for t in given}
        del given
        side.wait_stream(torch.cuda.current_stream())
        got = call(side)
        assert not free & {t.data_ptr() for t in got}, name
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name
