"""Cases, inputs and plain forms of the operators that bring prompts and drafted tokens into a paged cache.

Four operators, measured on the same inputs in their plain form (elementary
torch operations in 32 bits) and, where ``own`` is true, as calls of the
package:

* ``prompt``: attention over whole prompts, packed one behind the other;
* ``tree``: attention of drafted tokens, a tree per sequence, over a paged
  cache that holds their keys and values behind the sequence's own;
* ``reserve``: pages for the tokens that a step adds to every sequence, pages
  back from those that it drops, and the slot of every added token;
* ``append``: key and value rows of new tokens written into their slots.

``prepare`` makes a case's inputs from the seed; ``run`` is one pass;
``exact`` is the definition in 64 bits, written apart from the plain forms.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ the cases

def _prompt(name, B, Hq, Hkv, D, L, layout="stacked", ragged=False, causal=True):
    return {"name": name, "op": "prompt", "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "L": L, "layout": layout,
            "ragged": ragged, "causal": causal}


def _tree(name, B, Hq, Hkv, D, S, L, T, layout="token", ragged=False, shape="tree", mask=False):
    return {"name": name, "op": "tree", "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "S": S, "L": L, "T": T,
            "layout": layout, "ragged": ragged, "shape": shape, "mask": mask}


def _reserve(name, B, S, L, step, short=False):
    return {"name": name, "op": "reserve", "B": B, "S": S, "L": L, "step": step, "short": short}


def _append(name, B, Hq, Hkv, D, S, L, T, layout="token", sums=False):
    return {"name": name, "op": "append", "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "S": S, "L": L, "T": T,
            "layout": layout, "sums": sums}


def listed():
    return [
        # a chat's first question in the 4096-wide layer: one short prompt; latency counts
        _prompt("prompt 1 x 137", 1, 32, 32, 128, 137),
        # a step that takes in sixteen prompts of all lengths up to 2048
        _prompt("prompt 16 ragged x 2048", 16, 32, 32, 128, 2048, ragged=True),
        # a long document with four query heads to a key-value head
        _prompt("prompt 1 x 16384 grouped", 1, 32, 8, 128, 16384),
        # an odd model's encoder: every token looks at all, head-major rows of 80
        _prompt("prompt 5 ragged x 613 of 80", 5, 12, 4, 80, 613, layout="head", ragged=True, causal=False),
        # one sequence verifies a small tree of drafts over a cache of 1024 tokens; latency counts
        _tree("tree 1 x 1024, 25 drafted", 1, 32, 32, 128, 16, 1024, 25),
        # a serving batch of that layer, every sequence of another length, eight drafted tokens in a row
        _tree("tree 16 ragged x 4096, 8 in a row", 16, 32, 32, 128, 16, 4096, 8, ragged=True, shape="chain"),
        # long documents with eight query heads to a key-value head, pages of 64 tokens, trees of 64
        _tree("tree 2 x 131072 grouped, 64", 2, 64, 8, 128, 64, 131072, 64, layout="head"),
        # the pages of a decode step: one token for each of sixteen sequences
        _reserve("reserve 16 x 1", 16, 16, 2000, "one"),
        # continuous batching: of 256 sequences a quarter ends, a quarter begins, the others take a token
        _reserve("reserve 256, turnover", 256, 16, 2048, "turnover"),
        # the new tokens of a decode step into the cache, with their accumulated weights and positions
        _append("append 16 x 1", 16, 32, 32, 128, 16, 2000, 1, sums=True),
        # the prompts of a step into the cache
        _append("append 8 x 2048", 8, 32, 8, 128, 32, 2048, 2048),
    ]


def _log(rng, lo, hi):
    """A whole number spread over [lo, hi] by its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "tree", "tree", "reserve", "append"])
    hkv, g = rng.choice([1, 2, 4, 8, 12, 32]), rng.choice([1, 1, 2, 4, 5, 8])
    d = rng.choice([64, 80, 96, 128, 128, 128, 256])
    layout, s = rng.choice(["token", "head"]), rng.choice([8, 16, 16, 24, 32, 64, 128])
    if op == "prompt":
        b = _log(rng, 1, 64)
        most = math.isqrt((1 << 32) // (hkv * g * b * max(1, d // 128)))  # the scores of the largest listed case
        c = _prompt("", b, hkv * g, hkv, d, _log(rng, 1, max(1, min(16384, most))),
                    rng.choice(["stacked", "stacked", "token", "head"]), rng.random() < 0.6, rng.random() < 0.8)
    elif op == "tree":
        b, t = _log(rng, 1, 32), _log(rng, 1, 64)
        most = (1 << 28) // (b * max(hkv * d, hkv * g * t // 4))
        c = _tree("", b, hkv * g, hkv, d, s, _log(rng, t, max(t, min(131072, most))), t, layout,
                  rng.random() < 0.6, rng.choice(["tree", "tree", "chain"]), rng.random() < 0.3)
    elif op == "reserve":
        b = _log(rng, 1, 512)
        c = _reserve("", b, s, _log(rng, 64, max(64, min(32768, (1 << 19) // b))),
                     rng.choice(["one", "draft", "turnover"]), rng.random() < 0.3)
    else:
        b = _log(rng, 1, 64)
        length = _log(rng, 1, max(1, min(32768, (1 << 25) // (b * hkv * d))))
        c = _append("", b, hkv * g, hkv, d, s, length, rng.choice([1, 1, max(1, length // 7), length]), layout,
                    rng.random() < 0.5)
    del c["name"]
    return c


def _lengths(case):
    """Tokens of each sequence: all L, or spread from L/B to L, in larger batches with an empty and a single one."""
    B, L = case["B"], case["L"]
    n = [L] * B
    if case.get("ragged"):
        n = [max(1, L * (1 + (7 * b) % B) // B) for b in range(B)]
        if B >= 8:
            n[3], n[5] = 0, 1
    return n


def _drafted(case):
    """Drafted tokens of each sequence, which its length counts: T, fewer for some where batches are ragged."""
    t = [case["T"]] * case["B"]
    if case["ragged"]:
        t = [max(1, x - b % 3) for b, x in enumerate(t)]
    return [min(x, n) for x, n in zip(t, _lengths(case))]


def _counts(case):
    """Lengths before a step and what it adds to each sequence (negative: drops)."""
    B, L = case["B"], case["L"]
    old = [max(1, L - (13 * b) % max(1, L // 2)) for b in range(B)]
    if case["step"] == "one":
        return old, [1] * B
    if case["step"] == "draft":  # drafted tokens, and what an earlier step drafted in vain
        return old, [5 + b % 20 if b % 4 else -min(old[b], 7) for b in range(B)]
    add = [1] * B
    for b in range(B):
        if b % 4 == 1:
            add[b] = -old[b]
        elif b % 4 == 3:
            add[b], old[b] = old[b], 0
    return old, add


def work(case):
    op = case["op"]
    if op == "prompt":
        Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
        n = _lengths(case)
        pairs = sum(x * (x + 1) // 2 if case["causal"] else x * x for x in n)
        return {"bytes": sum(n) * 4 * D * (Hq + Hkv) + 4 * (len(n) + 1), "flops": 4 * D * Hq * pairs}
    if op == "tree":
        Hq, Hkv, D, S = case["Hq"], case["Hkv"], case["D"], case["S"]
        n, t = _lengths(case), _drafted(case)
        b = sum(n) * 4 * Hkv * D + sum(t) * (4 * Hq * D + 4) + 4 * sum(-(-x // S) for x in n) + sum(n) * case["mask"]
        return {"bytes": b, "flops": 4 * D * Hq * sum(x * y for x, y in zip(n, t))}
    if op == "reserve":
        S = case["S"]
        old, add = _counts(case)
        pages = sum(abs(-(-(o + a) // S) - -(-o // S)) for o, a in zip(old, add))
        # both ways: lengths, counts, starts and grants, the pages that change hands, the slots of added tokens
        return {"bytes": 2 * (20 * case["B"] + 8 * pages) + 8 * sum(abs(a) for a in add),
                "flops": sum(abs(a) for a in add)}
    T, Hkv, D = case["B"] * min(case["T"], case["L"]), case["Hkv"], case["D"]
    return {"bytes": T * (8 * Hkv * D + 8 + case["sums"] * (8 * Hkv + 4)), "flops": T}


# ------------------------------------------------------------------ the inputs

def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float16)


def _int(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _packed(case, g, T):
    """Queries, keys and values of T tokens: views of a stacked product's rows, or tensors of their own."""
    Hq, Hkv, D, layout = case["Hq"], case["Hkv"], case["D"], case.get("layout")
    if layout == "head":
        q, k, v = (_randn(g, h, T, D).transpose(0, 1) for h in (Hq, Hkv, Hkv))
    elif layout == "stacked" or case["op"] == "append":
        y = _randn(g, T, (Hq + 2 * Hkv) * D).view(T, Hq + 2 * Hkv, D)
        q, k, v = y[:, :Hq], y[:, Hq:Hq + Hkv], y[:, Hq + Hkv:]
    else:
        q, k, v = (_randn(g, T, h, D) for h in (Hq, Hkv, Hkv))
    q.mul_(2.0)  # scores with a deviation of 2: some tokens stand out
    return {"q": q, "k": k, "v": v}


def _pages(n, S, g, more=3):
    """A page table for sequences of n tokens, in random order: (pages of the pool, table)."""
    per = max(1, -(-max(n) // S))
    P = sum(-(-x // S) for x in n) + more
    free = torch.randperm(P, generator=g, device=DEV).to(torch.int32)
    used = torch.arange(per, device=DEV) < -(-_int(n)[:, None] // S)
    table = torch.full((len(n), per), -1, dtype=torch.int32, device=DEV)  # -1: no page there
    table[used] = free[:P - more]
    return P, table


def _pools(case, g, P):
    Hkv, D, S = case["Hkv"], case["D"], case["S"]
    shape = (P, S, Hkv, D) if case["layout"] == "token" else (P, Hkv, S, D)
    k, v = _randn(g, *shape), _randn(g, *shape)
    return (k, v) if case["layout"] == "token" else (k.transpose(1, 2), v.transpose(1, 2))


def _describe(s):
    """A serving program describes its pools once; table and lengths change in place."""
    if own:
        import sparse_weight_matmul_amd as swm
        s["cache"] = swm.PagedCache(s["pool_k"], s["pool_v"], s["table"], s["lengths"])


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op = case["op"]
    s = {"case": case}
    if op == "prompt":
        n = _lengths(case)
        s.update(_packed(case, g, sum(n)))
        s["starts"] = _int(np.concatenate([[0], np.cumsum(n)]).tolist())
    elif op == "tree":
        n, t = _lengths(case), _drafted(case)
        P, s["table"] = _pages(n, case["S"], g)
        s["pool_k"], s["pool_v"] = _pools(case, g, P)
        s["lengths"] = _int(n)
        T = sum(t)
        s["q"] = _randn(g, T, case["Hq"], case["D"]) * 2.0
        s["starts"] = _int(np.concatenate([[0], np.cumsum(t)]).tolist())
        i = torch.cat([torch.arange(x, device=DEV) for x in t])
        if case["shape"] == "tree":  # a parent among the four drafted last, or the sequence itself
            back = torch.randint(1, 5, (T,), generator=g, device=DEV)
            s["parents"] = (i - back).clamp(min=-1).to(torch.int32)
        else:
            s["parents"] = (i - 1).to(torch.int32)
        s["mask"] = None
        if case["mask"]:  # true where a token counts; a left padding and some single tokens do not
            cap = s["table"].shape[1] * case["S"]
            pad = torch.randint(0, max(1, case["L"] // 8) + 1, (case["B"], 1), generator=g, device=DEV)
            s["mask"] = torch.rand((case["B"], cap), generator=g, device=DEV) > 0.1
            s["mask"] &= torch.arange(cap, device=DEV) >= pad
        _describe(s)
    elif op == "reserve":
        S = case["S"]
        old, add = _counts(case)
        need = sum(max(0, -(-(o + a) // S) - -(-o // S)) for o, a in zip(old, add))
        back = sum(max(0, -(-o // S) - -(-(o + a) // S)) for o, a in zip(old, add))
        more = max(0, need - back) + 5
        if case["short"]:  # not all of them can be had
            more = max(1, (need - back) // 2) if need > back else 1
        P, table = _pages(old, S, g, more)
        s["table"] = torch.full((case["B"], -(-max(o + max(a, 0) for o, a in zip(old, add)) // S) + 1), -1,
                                dtype=torch.int32, device=DEV)
        s["table"][:, :table.shape[1]] = table
        taken = torch.zeros(P, dtype=torch.bool, device=DEV)
        taken[table[table >= 0].long()] = True
        s["free"] = torch.full((P,), -1, dtype=torch.int32, device=DEV)
        s["free"][:more] = (~taken).nonzero()[:, 0][torch.randperm(more, generator=g, device=DEV)]
        s["free_count"] = _int([more])
        s["lengths"], s["counts"] = _int(old), _int(add)
        s["tokens"] = [sum(max(0, a) for a in add), sum(max(0, -a) for a in add)]  # of the step, and of its undoing
        s["pool_k"] = s["pool_v"] = torch.zeros((P, S, 1, 8), dtype=torch.float16, device=DEV)
        _describe(s)
    else:
        B, S, L, T = (case[k] for k in ("B", "S", "L", "T"))
        P, s["table"] = _pages([L] * B, S, g)
        s["pool_k"], s["pool_v"] = _pools(case, g, P)
        s["lengths"] = _int([L] * B)
        s.update(_packed(case, g, B * T))
        at = torch.arange(L - T, L, device=DEV)
        page = s["table"][:, at // S].long()
        s["slots"] = (page * S + at % S).view(-1)
        s["sums"] = None
        if case["sums"]:
            s["sums"] = torch.rand((P, case["Hkv"], S), generator=g, device=DEV)
            s["positions"] = torch.zeros((P, case["Hkv"], S), dtype=torch.int32, device=DEV)
            s["at"] = (at.repeat(B) + torch.randint(0, 1000, (1,), generator=g, device=DEV)).to(torch.int32)
        _describe(s)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import sparse_weight_matmul_amd as swm
    op = s["case"]["op"]
    if op == "prompt":
        return [swm.prompt_attention(s["q"], s["k"], s["v"], s["starts"], causal=s["case"]["causal"])]
    if op == "tree":
        return [swm.tree_attention(s["cache"], s["q"], s["starts"], s["parents"], max_tokens=s["case"]["T"],
                                   mask=s["mask"])]
    if op == "reserve":  # a step's pages, and back
        c, free, count = s["cache"], s["free"], s["free_count"]
        a = swm.kv_reserve(c, s["counts"], free, count, s["tokens"][0])
        b = swm.kv_reserve(c, -a[2], free, count, s["tokens"][1])
        return [*a, *b, s["table"], s["lengths"], free, count]
    if s["sums"] is None:
        swm.kv_append(s["cache"], s["k"], s["v"], s["slots"])
        return [s["pool_k"], s["pool_v"]]
    swm.kv_append(s["cache"], s["k"], s["v"], s["slots"], weights=s["sums"], positions=s["positions"], at=s["at"])
    return [s["pool_k"], s["pool_v"], s["sums"], s["positions"]]


def _run_plain(s):
    op = s["case"]["op"]
    if op == "reserve":
        a = _reserve_plain(s, s["counts"], s["tokens"][0])
        b = _reserve_plain(s, -a[2], s["tokens"][1])
        return [*a, *b, s["table"], s["lengths"], s["free"], s["free_count"]]
    return {"prompt": _prompt_plain, "tree": _tree_plain, "append": _append_plain}[op](s)


def _softmax(score):
    """Over the last dimension, in place; a row of -inf gives zeros."""
    top = score.amax(-1, keepdim=True)
    score.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = score.sum(-1, keepdim=True)
    return score.div_(torch.where(total > 0, total, torch.ones_like(total)))


def _rows_of(starts, T):
    """The sequence of each of T packed rows, and its place there."""
    i = torch.arange(T, device=starts.device)
    b = torch.searchsorted(starts[1:].contiguous(), i.to(torch.int32), right=True)
    return b, i - starts[b]


def _prompt_plain(s):
    q, k, v, starts, case = s["q"], s["k"], s["v"], s["starts"], s["case"]
    T, Hq, D = q.shape
    B, Hkv, L = case["B"], case["Hkv"], case["L"]
    b, i = _rows_of(starts, T)
    pq = torch.zeros((B, L, Hq, D), device=q.device)
    pk, pv = torch.zeros((B, L, Hkv, D), device=q.device), torch.zeros((B, L, Hkv, D), device=q.device)
    pq[b, i], pk[b, i], pv[b, i] = q.float(), k.float(), v.float()
    score = pq.view(B, L, Hkv, -1, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D) @ pk.permute(0, 2, 3, 1)
    score.mul_(1.0 / math.sqrt(D))
    at = torch.arange(L, device=q.device)
    dead = (at >= (starts[1:] - starts[:-1])[:, None])[:, None].expand(B, L, L)
    if case["causal"]:
        dead = dead | (at > at[:, None])
    score.view(B, Hkv, -1, L, L).masked_fill_(dead[:, None, None], -math.inf)
    out = _softmax(score) @ pv.transpose(1, 2)
    return [out.view(B, Hq, L, D).transpose(1, 2)[b, i].half()]


def _tree_plain(s):
    q, table, starts, case = s["q"], s["table"], s["starts"], s["case"]
    n, mask = s["lengths"][:, None], s["mask"]
    T, Hq, D = q.shape
    P, S, Hkv, _ = s["pool_k"].shape
    B, most = table.shape[0], case["T"]
    cap = table.shape[1] * S
    page = table.long().clamp(0, P - 1)
    k = s["pool_k"][page].reshape(B, cap, Hkv, D).permute(0, 2, 3, 1).float()
    v = s["pool_v"][page].reshape(B, cap, Hkv, D).transpose(1, 2).float()
    b, i = _rows_of(starts, T)
    pq = torch.zeros((B, most, Hq, D), device=q.device)
    pq[b, i] = q.float()
    # which drafted tokens each of them sees: itself, its parent and so on, by squaring
    sees = torch.eye(most, device=q.device).repeat(B, 1, 1)
    child = s["parents"] >= 0
    sees[b[child], i[child], s["parents"][child].long()] = 1.0
    sees = ((sees @ sees) > 0).float()
    sees = ((sees @ sees) > 0).float()
    sees = ((sees @ sees) > 0).float()
    sees = ((sees @ sees) > 0).float()
    sees = ((sees @ sees) > 0).float()
    sees = (sees @ sees) > 0
    slot = torch.arange(cap, device=q.device)
    j = slot - (n - (starts[1:] - starts[:-1])[:, None])  # the drafted token of each slot
    live = torch.where((j < 0)[:, None], True, sees.gather(2, j.clamp(0, most - 1)[:, None].expand(B, most, cap)))
    live &= (slot < n)[:, None]
    if mask is not None:
        live &= mask[:, None]
    score = pq.view(B, most, Hkv, -1, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D) @ k
    score.mul_(1.0 / math.sqrt(D)).view(B, Hkv, -1, most, cap).masked_fill_(~live[:, None, None], -math.inf)
    out = _softmax(score) @ v.masked_fill(~(slot < n)[:, None, :, None], 0.0)
    return [out.view(B, Hq, most, D).transpose(1, 2)[b, i].half()]


def _reserve_plain(s, counts, tokens):
    table, lengths, free, count = s["table"], s["lengths"], s["free"], s["free_count"]
    P, S = s["pool_k"].shape[:2]
    B, per = table.shape
    old = lengths.clone()
    want = torch.where(old + counts > per * S, old, (old + counts).clamp(min=0))  # past its table: refused
    had, has = (old + S - 1) // S, (want + S - 1) // S
    place = torch.arange(per, device=table.device)
    back = (place >= has[:, None]) & (place < had[:, None])
    pages = table[back]  # by sequence, then by place
    have = count + len(pages)
    free[(count + torch.arange(len(pages), device=table.device)).long()] = pages
    table.masked_fill_(back, -1)
    need = (has - had).clamp(min=0)
    upto = torch.cumsum(need, 0, dtype=torch.int32)
    fits = (need == 0) | (upto <= have)  # in order: one that does not fit leaves nothing to those after it
    new = torch.where(fits, want, old)
    take = (place >= had[:, None]) & (place < has[:, None]) & fits[:, None]
    j = (upto - need)[:, None] + place - had[:, None]
    table[take] = free[(have - 1 - j)[take].long()]
    count.copy_(have - torch.where(fits, need, torch.zeros_like(need)).sum())
    lengths.copy_(new)
    granted = new - old
    starts = torch.cat([torch.zeros_like(counts[:1]), torch.cumsum(counts.clamp(min=0), 0, dtype=torch.int32)])
    i = torch.arange(tokens, device=table.device, dtype=torch.int32)
    b = torch.searchsorted(starts[1:].contiguous(), i, right=True).clamp(max=B - 1)
    at = (old[b] + i - starts[b]).clamp(max=per * S - 1)
    slots = table[b, (at // S).long()].long() * S + at % S
    return [starts, torch.where((granted[b] > 0) & (i < starts[-1]), slots, torch.full_like(slots, -1)), granted]


def _append_plain(s):
    S = s["pool_k"].shape[1]
    page, slot = s["slots"] // S, s["slots"] % S
    s["pool_k"][page, slot], s["pool_v"][page, slot] = s["k"], s["v"]
    if s["sums"] is None:
        return [s["pool_k"], s["pool_v"]]
    s["sums"][page, :, slot] = 0.0
    s["positions"][page, :, slot] = s["at"][:, None]
    return [s["pool_k"], s["pool_v"], s["sums"], s["positions"]]


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    op = case["op"]
    if op == "append":  # copies, not computed
        return None
    s = prepare(case, seed)
    return {"prompt": _prompt_exact, "tree": _tree_exact, "reserve": _reserve_exact}[op](case, s)


def _prompt_exact(case, s):
    G, D = case["Hq"] // case["Hkv"], case["D"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    at = 0
    for n in _lengths(case):
        for h in range(case["Hq"] if n else 0):
            q, k, v = (x[at:at + n, y].double().contiguous() for x, y in ((s["q"], h), (s["k"], h // G), (s["v"], h // G)))
            x = q @ k.t().contiguous() / D ** 0.5
            if case["causal"]:
                x = x.masked_fill_(torch.ones((n, n), dtype=torch.bool, device=DEV).triu_(1), -math.inf)
            out[at:at + n, h] = torch.softmax(x, -1) @ v
        at += n
    return [out.cpu().numpy()]


def _tree_exact(case, s):
    G, D, S = case["Hq"] // case["Hkv"], case["D"], case["S"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    parents = s["parents"].tolist()
    at = 0
    for b, (n, t) in enumerate(zip(_lengths(case), _drafted(case))):
        slot = torch.arange(n, device=DEV)
        page = s["table"][b].long()[slot // S]
        sees = torch.ones((t, n), dtype=torch.bool)
        for i in range(t):
            sees[i, n - t:] = False
            j = i
            while j >= 0:
                sees[i, n - t + j] = True
                j = parents[at + j]
        sees = sees.to(DEV)
        if s["mask"] is not None:
            sees &= s["mask"][b, :n]
        none = ~sees.any(1, keepdim=True)
        for h in range(case["Hkv"] if t else 0):
            k, v = s["pool_k"][page, slot % S, h].double(), s["pool_v"][page, slot % S, h].double()
            for y in range(h * G, (h + 1) * G):
                x = s["q"][at:at + t, y].double() @ k.t().contiguous() / D ** 0.5
                p = torch.softmax(x.masked_fill(~sees & ~none, -math.inf), -1)
                out[at:at + t, y] = p.masked_fill(none, 0.0) @ v
        at += t
    return [out.cpu().numpy()]


def _reserve_exact(case, s):
    S = case["S"]
    table, lengths, free = s["table"].cpu().numpy(), s["lengths"].cpu().numpy(), s["free"].cpu().numpy()
    stack = free[:int(s["free_count"])].tolist()
    counts, result = s["counts"].cpu().numpy(), []
    for tokens in s["tokens"]:
        granted, slots, starts, room = np.zeros_like(counts), np.full(tokens, -1, np.int64), [0], True
        for b, c in enumerate(counts):  # pages come back before any are given out
            if c < 0:
                new = max(0, lengths[b] + c)
                for i in range(-(-new // S), -(-lengths[b] // S)):
                    stack.append(table[b, i])
                    free[len(stack) - 1] = table[b, i]
                    table[b, i] = -1
                granted[b], lengths[b] = new - lengths[b], new
        for b, c in enumerate(counts):
            starts.append(starts[-1] + max(0, c))
            new = lengths[b] + c
            if c <= 0 or new > table.shape[1] * S:
                continue
            first, last = -(-lengths[b] // S), -(-new // S)
            if last > first:
                room = room and last - first <= len(stack)
                if not room:
                    continue
            for i in range(first, last):
                table[b, i] = stack.pop()
            t = np.arange(lengths[b], new)
            slots[starts[-2]:starts[-1]] = table[b, t // S].astype(np.int64) * S + t % S
            granted[b], lengths[b] = c, new
        result += [np.array(starts, np.int32), slots, granted]
        counts = -granted
    return result + [table, lengths, free, np.array([len(stack)], np.int32)]
