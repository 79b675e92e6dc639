"""Cases, inputs and plain forms of the serving operators beside the pruned products.

Four operators, measured on the same inputs in their plain form (elementary
torch operations in 32 bits) and, where ``own`` is true, as calls of the
package:

* ``attention``: one new token per sequence over a paged key-value cache,
  optionally adding each position's attention weight to an accumulator;
* ``evict``: a cache cut back to a budget of tokens per head, by that
  accumulated weight and a window of recent tokens;
* ``product``: a pruned product with bias, activation and residual;
* ``logprobs``: log probabilities of given tokens, the entropy of every row
  and its most likely tokens.

``prepare`` makes a case's inputs from the seed; ``run`` is one pass;
``exact`` is the definition in 64 bits, written apart from the plain forms.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ the cases

def _attention(name, B, Hq, Hkv, D, S, L, layout="token", ragged=False, mask=False, weights=False):
    return {"name": name, "op": "attention", "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "S": S, "L": L,
            "layout": layout, "ragged": ragged, "mask": mask, "weights": weights}


def _evict(name, B, Hkv, D, S, L, budget, recent, layout="token", ragged=False):
    return {"name": name, "op": "evict", "B": B, "Hkv": Hkv, "D": D, "S": S, "L": L, "budget": budget,
            "recent": recent, "layout": layout, "ragged": ragged}


def _product(name, M, K, N, sparsity, act, bias, residual):
    return {"name": name, "op": "product", "M": M, "K": K, "N": N, "sparsity": sparsity, "act": act,
            "bias": bias, "residual": residual}


def _logprobs(name, N, V, top, dtype, masked):
    return {"name": name, "op": "logprobs", "N": N, "V": V, "top": top, "dtype": dtype, "masked": masked}


def listed():
    return [
        # a chat's first answers: one sequence of the 4096-wide layer, a cache of a few pages; latency counts
        _attention("attention 1 x 137", 1, 32, 32, 128, 16, 137),
        # a serving batch of that layer, every sequence of another length, weights kept for the eviction
        _attention("attention 16 x 4096 weights", 16, 32, 32, 128, 16, 4096, ragged=True, weights=True),
        # long documents with eight query heads to a key-value head, pages of 64 tokens kept head by head
        _attention("attention 2 x 131072 grouped", 2, 64, 8, 128, 64, 131072, layout="head"),
        # the step after a token was appended to a full cache: one token of each head goes
        _evict("evict 1 x 1025 to 1024", 1, 32, 128, 16, 1025, 1024, 256),
        # a batch that lets 128 tokens pile up between evictions
        _evict("evict 16 x 2176 to 2048", 16, 8, 128, 32, 2176, 2048, 512),
        # prompts of a batch cut to a quarter after they were read
        _evict("evict 8 x 4096 to 1024", 8, 32, 128, 16, 4096, 1024, 128, ragged=True),
        # the attention's output projection with the residual stream, one token
        _product("product 4096x4096 n1", 4096, 4096, 1, 0.5, "none", False, True),
        # the feed-forward block's second projection, a decode batch
        _product("product 4096x11008 n16", 4096, 11008, 16, 0.5, "none", True, True),
        # a feed-forward block's first projection over a prompt
        _product("product 11008x4096 n2048", 11008, 4096, 2048, 0.5, "gelu", True, False),
        # the token just sampled, with five alternatives for the caller
        _logprobs("logprobs 1 x 32000", 1, 32000, 5, "float16", False),
        # a batch under a grammar that rules tokens out, 32-bit logits of an odd vocabulary
        _logprobs("logprobs 61 x 50021 masked", 61, 50021, 20, "float32", True),
        # the perplexity of a window of 4096 tokens
        _logprobs("logprobs 4096 x 32000", 4096, 32000, 0, "float16", False),
    ]


def _log(rng, lo, hi):
    """A whole number spread over [lo, hi] by its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["attention", "evict", "product", "logprobs"])
    if op == "attention":
        hkv, g = rng.choice([1, 2, 4, 8, 12, 32]), rng.choice([1, 1, 2, 4, 5, 8, 16])
        d = rng.choice([64, 80, 96, 128, 128, 128, 256])
        b = _log(rng, 1, 64)
        most = (1 << 29) // (hkv * d * b)  # key values of the largest listed case, shared out
        length = _log(rng, 1, max(1, min(131072, most // 2, (1 << 24) * 2 // (hkv * g * b))))
        c = _attention("", b, hkv * g, hkv, d, rng.choice([8, 16, 16, 24, 32, 64, 128]), length,
                       rng.choice(["token", "head"]), rng.random() < 0.6, rng.random() < 0.3, rng.random() < 0.5)
    elif op == "evict":
        b, hkv = _log(rng, 1, 32), rng.choice([1, 2, 8, 8, 32])
        d = rng.choice([64, 80, 128, 128, 256])
        length = _log(rng, 17, max(17, min(32768, (1 << 27) // (b * hkv * d))))
        gone = rng.choice([1, 1, max(1, length // 16), max(1, length // 2), max(1, (3 * length) // 4)])
        budget = max(1, length - gone)
        c = _evict("", b, hkv, d, rng.choice([8, 16, 16, 24, 32, 64]), length, budget,
                   rng.randint(0, budget), rng.choice(["token", "head"]), rng.random() < 0.5)
    elif op == "product":
        m, k = rng.choice([(4096, 4096), (11008, 4096), (4096, 11008), (None, None)])
        if m is None:
            m, k = _log(rng, 100, 8192), 8 * _log(rng, 8, 512)
        n = rng.choice([_log(rng, 1, 32), _log(rng, 1, 2048)])
        c = _product("", m, k, n, rng.choice([0.5, 0.6, 0.7]), rng.choice(["none", "relu", "silu", "gelu"]),
                     rng.random() < 0.6, rng.random() < 0.6)
    else:
        n = _log(rng, 1, 4096)
        v = _log(rng, 200, max(200, min(131072, (1 << 26) // n)))
        c = _logprobs("", n, v, rng.choice([0, 1, 5, 20, 32]), rng.choice(["float16", "float16", "float32"]),
                      rng.random() < 0.4)
    del c["name"]
    return c


def _lengths(case):
    """Tokens of each sequence: all L, or spread from L/B to L with an idle place in larger batches."""
    B, L = case["B"], case["L"]
    n = [L] * B
    if case["ragged"]:
        n = [max(1, L * (1 + (7 * b) % B) // B) for b in range(B)]
        if B >= 8:
            n[3] = 0
    return n


def work(case):
    op = case["op"]
    if op == "attention":
        B, Hq, Hkv, D, S = (case[k] for k in ("B", "Hq", "Hkv", "D", "S"))
        n = sum(_lengths(case))
        b = 4 * n * Hkv * D + 4 * B * Hq * D + 4 * B * -(-case["L"] // S)
        b += 8 * n * Hkv * case["weights"] + n * case["mask"]
        return {"bytes": b, "flops": 4 * n * Hq * D}
    if op == "evict":
        Hkv, D, budget = case["Hkv"], case["D"], case["budget"]
        n = [x for x in _lengths(case)]
        kept = sum(min(x, budget) for x in n)
        # weights and positions read, those of the kept tokens and the map written; the rows that change
        # their place are at most the tail's and at least those of the recent window
        moved = sum(min(case["recent"], x - budget) for x in n if x > budget)
        return {"bytes": Hkv * (8 * sum(n) + 12 * kept + 8 * D * moved), "flops": Hkv * sum(n)}
    if op == "product":
        M, K, N = case["M"], case["K"], case["N"]
        nnz = M * K * (1 - case["sparsity"])
        b = 2 * nnz + M * K / 8 + 2 * N * K + 2 * N * M * (1 + case["residual"]) + 2 * M * case["bias"]
        return {"bytes": b, "flops": 2 * nnz * N}
    N, V, top = case["N"], case["V"], case["top"]
    size = 2 if case["dtype"] == "float16" else 4
    return {"bytes": N * V * size + N * (16 + 12 * top), "flops": 4 * N * V}


# ------------------------------------------------------------------ the inputs

def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float16)


def _cache(case, g):
    """Pools of keys and values (P, S, Hkv, D), the page table and the lengths."""
    B, Hkv, D, S, L = (case[k] for k in ("B", "Hkv", "D", "S", "L"))
    n = _lengths(case)
    per = -(-L // S)
    P = sum(-(-x // S) for x in n) + 3
    shape = (P, S, Hkv, D) if case["layout"] == "token" else (P, Hkv, S, D)
    k, v = _randn(g, *shape), _randn(g, *shape)
    if case["layout"] == "head":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    free = torch.randperm(P, generator=g, device=DEV).to(torch.int32)
    table = torch.full((B, per), -1, dtype=torch.int32, device=DEV)  # -1: no page there
    at = 0
    for b in range(B):
        pages = -(-n[b] // S)
        table[b, :pages] = free[at:at + pages]
        at += pages
    s = {"k": k, "v": v, "table": table, "lengths": torch.tensor(n, dtype=torch.int32, device=DEV)}
    if own:  # a serving program describes its pools once; table and lengths change in place
        import sparse_weight_matmul_amd as swm
        s["cache"] = swm.PagedCache(k, v, table, s["lengths"])
    return s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op = case["op"]
    s = {"case": case}
    if op == "attention":
        s.update(_cache(case, g))
        B, Hq, Hkv, D, S = (case[k] for k in ("B", "Hq", "Hkv", "D", "S"))
        s["q"] = _randn(g, B, Hq, D) * 2.0  # scores with a deviation of 2: some tokens stand out
        cap = s["table"].shape[1] * S
        s["mask"] = None
        if case["mask"]:  # true where a token counts; a left padding and some single tokens do not
            pad = torch.randint(0, max(1, case["L"] // 8) + 1, (B, 1), generator=g, device=DEV)
            s["mask"] = (torch.rand((B, cap), generator=g, device=DEV) > 0.1) & (torch.arange(cap, device=DEV) >= pad)
        s["weights"] = None
        if case["weights"]:
            s["weights"] = torch.rand((s["k"].shape[0], Hkv, S), generator=g, device=DEV)
    elif op == "evict":
        s.update(_cache(case, g))
        B, Hkv, S, L = (case[k] for k in ("B", "Hkv", "S", "L"))
        P = s["k"].shape[0]
        # accumulated weights have a long tail, and tokens that nothing looked at yet have none
        w = torch.rand((P, Hkv, S), generator=g, device=DEV) ** 6 * 4
        s["weights"] = torch.where(w < 1e-5, torch.zeros_like(w), w)
        # an earlier eviction left the tokens out of order: a shuffled half, then the order they came in
        cap = s["table"].shape[1] * S
        order = torch.arange(cap, device=DEV, dtype=torch.int32).repeat(B, Hkv, 1)
        half = max(1, min(case["budget"], L) // 2)
        order[:, :, :half] = torch.rand((B, Hkv, half), generator=g, device=DEV).argsort(-1).to(torch.int32)
        s["positions"] = torch.zeros((P, Hkv, S), dtype=torch.int32, device=DEV)
        b, p = (s["table"] >= 0).nonzero(as_tuple=True)
        s["positions"][s["table"][b, p].long()] = order.view(B, Hkv, -1, S).transpose(1, 2)[b, p]
        s["weights_out"], s["positions_out"] = torch.zeros_like(s["weights"]), torch.zeros_like(s["positions"])
    elif op == "product":
        M, K, N = case["M"], case["K"], case["N"]
        W = torch.randn((M, K), generator=g, device=DEV) * 0.02
        cut = 0.02 * math.sqrt(2) * torch.erfinv(torch.tensor(case["sparsity"])).item()
        s["W"] = torch.where(W.abs() > cut, W, torch.zeros_like(W)).half()  # the smaller magnitudes pruned
        s["X"] = _randn(g, N, K)
        s["bias"] = _randn(g, M) if case["bias"] else None
        s["residual"] = _randn(g, N, M) if case["residual"] else None
        if own:  # a pruned weight is compressed once, when the model is loaded
            import sparse_weight_matmul_amd as swm
            s["fmt"] = swm.sparse_compress(s["W"].cpu().numpy())
            need = swm.spmm_workspace_bytes(s["fmt"], N)
            s["ws"] = torch.empty(need, dtype=torch.uint8, device=DEV) if need else None
    else:
        N, V = case["N"], case["V"]
        x = torch.randn((N, V), generator=g, device=DEV) * 2.5
        if case["masked"]:
            x.masked_fill_(torch.rand((N, V), generator=g, device=DEV) < 0.3, -math.inf)
            if N > 1:
                x[N // 2] = -math.inf  # the grammar has no way on
        s["logits"] = x.to(getattr(torch, case["dtype"]))
        s["targets"] = torch.randint(0, V, (N,), generator=g, device=DEV)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import sparse_weight_matmul_amd as swm
    case = s["case"]
    op = case["op"]
    if op == "attention":
        out = swm.paged_attention(s["cache"], s["q"], mask=s["mask"], weights=s["weights"])
        return [out] if s["weights"] is None else [out, s["weights"]]
    if op == "evict":
        n, kept = swm.kv_evict(s["cache"], s["weights"], s["positions"], case["budget"], case["recent"],
                               weights_out=s["weights_out"], positions_out=s["positions_out"])
        return [n, kept, s["weights_out"], s["positions_out"], s["k"], s["v"]]
    if op == "product":
        return [swm.spmm_epilogue(s["fmt"], s["X"], bias=s["bias"], act=case["act"], residual=s["residual"],
                                  workspace=s["ws"])]
    r = swm.token_logprobs(s["logits"], s["targets"], top=case["top"])
    return list(r) if case["top"] else list(r[:2])


def _run_plain(s):
    return {"attention": _attention_plain, "evict": _evict_plain, "product": _product_plain,
            "logprobs": _logprobs_plain}[s["case"]["op"]](s)


def _attention_plain(s):
    q, table, mask = s["q"], s["table"], s["mask"]
    P, S, Hkv, D = s["k"].shape
    B, Hq, _ = q.shape
    cap = table.shape[1] * S
    page = table.long().clamp(0, P - 1)
    k = s["k"][page].reshape(B, cap, Hkv, D).permute(0, 2, 3, 1).float()
    v = s["v"][page].reshape(B, cap, Hkv, D).transpose(1, 2).float()
    live = torch.arange(cap, device=q.device) < s["lengths"][:, None]
    if mask is not None:
        live = live & mask
    score = (q.float().reshape(B, Hkv, Hq // Hkv, D) @ k) * (1.0 / math.sqrt(D))
    score = score.masked_fill(~live[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, torch.ones_like(total))  # a row with no token left gives zeros
    out = (p @ v.masked_fill(~live[:, None, :, None], 0.0)).reshape(B, Hq, D).half()
    if s["weights"] is None:
        return [out]
    add = p.sum(2).reshape(B, Hkv, -1, S).transpose(1, 2).reshape(-1, Hkv, S)
    s["weights"].index_add_(0, page.reshape(-1), add)
    return [out, s["weights"]]


def _evict_plain(s):
    case, table = s["case"], s["table"]
    budget, recent = case["budget"], case["recent"]
    P, S, Hkv, D = s["k"].shape
    B, cap = table.shape[0], table.shape[1] * S
    page = table.long().clamp(0, P - 1)
    slot = torch.arange(cap, device=table.device)
    n = s["lengths"][:, None, None]
    live = (slot < n).expand(B, Hkv, cap)
    w = s["weights"][page].transpose(1, 2).reshape(B, Hkv, cap)
    pos = s["positions"][page].transpose(1, 2).reshape(B, Hkv, cap)
    newest = pos.masked_fill(~live, -1).amax(-1, keepdim=True)
    key = torch.where((pos > newest - recent) | torch.isnan(w), torch.full_like(w, math.inf), w)
    key = key.masked_fill(~live, -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, slot.expand_as(order))
    keep = (rank < budget) & live
    new_lengths = s["lengths"].clamp(max=budget)
    stay = live & (slot < budget)
    # the tail's kept tokens fill, in order, the places that were freed below the budget
    hb, hh, hs = (stay & ~keep).nonzero(as_tuple=True)
    mb, mh, ms = (keep & (slot >= budget)).nonzero(as_tuple=True)
    kept = torch.full((B, Hkv, budget), -1, dtype=torch.int32, device=table.device)
    b, h, j = stay.nonzero(as_tuple=True)
    kept[b, h, j] = j.int()
    kept[hb, hh, hs] = ms.int()
    src = kept[b, h, j].long()
    s["weights_out"][page[b, j // S], h, j % S] = w[b, h, src]
    s["positions_out"][page[b, j // S], h, j % S] = pos[b, h, src]
    for c in (s["k"], s["v"]):
        c[page[hb, hs // S], hs % S, hh] = c[page[mb, ms // S], ms % S, mh]
    return [new_lengths, kept, s["weights_out"], s["positions_out"], s["k"], s["v"]]


def _product_plain(s):
    y = s["X"].float() @ s["W"].float().t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    act = s["case"]["act"]
    if act == "relu":
        y = torch.where(y > 0, y, torch.zeros_like(y))
    elif act == "silu":
        y = y / (1 + torch.exp(-y))
    elif act == "gelu":
        y = 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return [y.half()]


def _logprobs_plain(s):
    x, t, top = s["logits"].float(), s["targets"], s["case"]["top"]
    m = x.amax(-1, keepdim=True)
    d = x - torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = torch.exp(d)
    z = e.sum(-1, keepdim=True)
    log_z = torch.log(torch.where(z > 0, z, torch.ones_like(z)))  # no token left: log probabilities of -inf
    mean = (e * torch.where(e > 0, d, torch.zeros_like(d))).sum(-1, keepdim=True) / torch.where(z > 0, z, 1.0)
    logp = d.gather(-1, t[:, None]) - log_z
    out = [logp[:, 0], (log_z - mean)[:, 0]]
    if top:
        v, i = torch.sort(d, dim=-1, descending=True, stable=True)
        out += [i[:, :top].contiguous(), v[:, :top] - log_z]
    return out


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"attention": _attention_exact, "evict": _evict_exact, "product": _product_exact,
            "logprobs": _logprobs_exact}[case["op"]](case, s)


def _tokens(s, pool, b):
    """A sequence's rows of a pool, in slot order."""
    n, S = int(s["lengths"][b]), pool.shape[1]
    t = torch.arange(n, device=pool.device)
    return pool[s["table"][b].long()[t // S], t % S]


def _attention_exact(case, s):
    B, Hq, D = s["q"].shape
    Hkv, S = case["Hkv"], case["S"]
    out = torch.zeros((B, Hq, D), dtype=torch.float64, device=DEV)
    weights = None if s["weights"] is None else s["weights"].double()
    for b in range(B):
        n = int(s["lengths"][b])
        t = torch.arange(n, device=DEV)
        if s["mask"] is not None:
            t = t[s["mask"][b, :n]]
        if len(t) == 0:
            continue
        K, V = _tokens(s, s["k"], b), _tokens(s, s["v"], b)
        for h in range(Hkv):
            heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            x = s["q"][b, heads].double() @ K[t, h].double().t().contiguous() / D ** 0.5
            p = torch.softmax(x, -1)
            out[b, heads] = p @ V[t, h].double()
            if weights is not None:
                weights[s["table"][b].long()[t // S], h, t % S] += p.sum(0)
    return [out.cpu().numpy()] + ([] if weights is None else [weights.cpu().numpy()])


def _evict_exact(case, s):
    B, Hkv, S, budget = case["B"], case["Hkv"], case["S"], case["budget"]
    n, table = s["lengths"].cpu().numpy(), s["table"].cpu().numpy()
    w, pos = s["weights"].cpu().numpy().astype(np.float64), s["positions"].cpu().numpy()
    w_out, pos_out = np.zeros_like(w), np.zeros_like(pos)
    kept = np.full((B, Hkv, budget), -1, np.int32)
    for b in range(B):
        t = np.arange(n[b])
        if not len(t):
            continue
        page, slot = table[b, t // S], t % S
        for h in range(Hkv):
            wt, pt = w[page, h, slot], pos[page, h, slot]
            worth = np.where(pt > pt.max() - case["recent"], np.inf, wt)
            good = np.sort(np.lexsort((t, -worth))[:budget])
            place = np.arange(min(n[b], budget))
            place[np.setdiff1d(place, good)] = good[good >= budget]
            kept[b, h, :len(place)] = place
            to = t[:len(place)]
            w_out[page[to], h, slot[to]] = wt[place]
            pos_out[page[to], h, slot[to]] = pt[place]
    return [np.minimum(n, budget), kept, w_out, pos_out, None, None]  # the pools are copies, not computed


def _product_exact(case, s):
    y = s["X"].double() @ s["W"].double().t().contiguous()
    if s["bias"] is not None:
        y = y + s["bias"].double()
    act = {"none": lambda z: z, "relu": lambda z: z.clamp(min=0), "silu": lambda z: z * torch.sigmoid(z),
           "gelu": lambda z: z * torch.special.ndtr(z)}[case["act"]]
    y = act(y)
    return [(y if s["residual"] is None else y + s["residual"].double()).cpu().numpy()]


def _logprobs_exact(case, s):
    N, top = case["N"], case["top"]
    logp, ent = np.empty(N), np.empty(N)
    top_ids, top_logp = np.empty((N, top), np.int64), np.empty((N, top))
    for i0 in range(0, N, 256):
        x = s["logits"][i0:i0 + 256].double()
        lse = torch.logsumexp(x, -1, keepdim=True)
        lp = torch.where(lse == -math.inf, x, x - lse)
        at = slice(i0, i0 + x.shape[0])
        logp[at] = lp.gather(-1, s["targets"][at, None])[:, 0].cpu().numpy()
        ent[at] = torch.special.entr(lp.exp()).sum(-1).cpu().numpy()
        if top:
            i = torch.sort(-lp, dim=-1, stable=True).indices[:, :top]
            top_ids[at], top_logp[at] = i.cpu().numpy(), lp.gather(-1, i).cpu().numpy()
    return [logp, ent] + ([top_ids, top_logp] if top else [])
