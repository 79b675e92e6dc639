"""The decoding example against the same steps written plainly in torch, 32 bits on the CPU."""
import importlib.util
import os

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load():
    spec = importlib.util.spec_from_file_location("pruned_decode", os.path.join(ROOT, "examples", "pruned_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


class Plain:
    """One sequence's cache as lists per head; the arithmetic in fp32, rounded where the library stores fp16."""

    def __init__(self, layer, budget, slack, recent):
        import torch
        self.y, self.budget, self.slack, self.recent = layer, budget, slack, recent
        self.w = {n: torch.from_numpy(w.astype(np.float32)) for n, w in layer.dense.items()}
        self.cache = [[] for _ in range(layer.kv_heads)]  # [position, weight, k, v]
        self.seen = 0

    def step(self, token, margin):
        import torch
        y, w = self.y, self.w
        half = lambda t: t.half().float()
        norm = lambda t: half(t * torch.rsqrt(t.square().mean() + 1e-5))
        x = y.embed[token].float().cpu()
        qkv = half(w["qkv"] @ norm(x))
        kv, D = y.kv_heads * y.dim, y.dim
        q = qkv[:y.hidden].view(y.heads, D)
        k, v = (qkv[i:i + kv].view(y.kv_heads, D) for i in (y.hidden, y.hidden + kv))
        out = torch.zeros(y.heads, D)
        for h in range(y.kv_heads):
            self.cache[h].append([self.seen, 0.0, k[h], v[h]])
            K, V = (torch.stack([c[i] for c in self.cache[h]]) for i in (2, 3))
            for g in range(h * (y.heads // y.kv_heads), (h + 1) * (y.heads // y.kv_heads)):
                p = torch.softmax(K @ q[g] * D ** -0.5, 0)
                out[g] = p @ V
                for c, pi in zip(self.cache[h], p):
                    c[1] += float(pi)
        self.seen += 1
        x = half(x + w["o"] @ half(out).view(-1))
        u = norm(x)
        g = w["gate"] @ u
        x = half(x + w["down"] @ half(g * torch.sigmoid(g) * (w["up"] @ u)))
        if len(self.cache[0]) == self.budget + self.slack:
            for h in range(y.kv_heads):
                c = self.cache[h]
                old = sorted((e for e in c if e[0] <= self.seen - 1 - self.recent), key=lambda e: -e[1])
                new = [e for e in c if e[0] > self.seen - 1 - self.recent]
                n = self.budget - len(new)
                margin.append((old[n - 1][1] - old[n][1]) / old[n - 1][1])  # how clear the cut was
                self.cache[h] = new + old[:n]
        return torch.log_softmax(half(w["head"] @ norm(x)), -1)


def test_steps_match_plain_torch(gpu_lib):
    import torch
    m = load()
    y = m.Layer(hidden=256, ffn=520, heads=4, kv_heads=2, vocab=1003, seed=3)
    s = m.Session(y, batch=2, budget=12, slack=4, recent=4, page_size=8)
    plain = [Plain(y, 12, 4, 4) for _ in range(2)]
    tokens, margin = torch.tensor([5, 77], device="cuda"), []
    for step in range(40):  # seven evictions
        ids, logp, entropy = s.step(tokens)
        for b in range(2):
            want = plain[b].step(int(tokens[b]), margin)
            # logits of a few units in fp16 behind eight products whose outputs are rounded to fp16: each
            # rounding is 2^-11 relative, so the residual stream and the logits (rms about 1) differ by 2^-7 at most
            assert abs(float(logp[b]) - float(want[int(ids[b])])) < 2.0**-7
            assert float(want.max()) - float(want[int(ids[b])]) < 2.0**-6
            assert abs(float(entropy[b]) + float((want.exp() * want).sum())) < 2.0**-6
            for h in range(2):  # the same tokens survive every eviction
                t = np.arange(s.used)
                page = s.table[b].cpu().numpy()[t // 8]
                got = s.positions.cpu().numpy()[page, h, t % 8]
                assert sorted(got.tolist()) == sorted(e[0] for e in plain[b].cache[h]), (step, b, h)
        tokens = ids  # both sides go on from the library's choice
    # the cuts were clear of the rounding of the attention weights, so equal survivors were due
    assert min(margin) > 1e-3
    assert s.seen == 40 and s.used < 16


def test_command_line(gpu_lib, capsys):
    load().main(["--hidden", "256", "--ffn", "512", "--heads", "4", "--kv-heads", "4", "--vocab", "500", "--batch", "3",
                 "--steps", "30", "--budget", "16", "--slack", "4"])
    assert "30 steps of 3 sequences" in capsys.readouterr().out
