"""Workloads of eviction by accumulated attention weight: the causal attention of prompts, packed behind each other
or a batch, the weights that it puts on every key, the weights of decode steps on a cache's rows, and the eviction
by their sums.

``listed()`` names the workloads, ``draw`` makes more of the same ranges, ``prepare`` makes the inputs of one on the
GPU and ``run`` makes one pass: with ``own`` set through the package's entry points, otherwise in plain torch
operations in 32 bits. ``exact`` computes the same results from the definitions in 64 bits, and ``work`` counts the
bytes and operations that no pass can do without.

The sizes are those of this repository's workloads where it has them: heads of 128 elements, 8 KV heads with several
query heads each; blocks of up to 8192 tokens; budgets of 512 to 4096 rows; decode steps of 32 sequences.
"""
import math
import random

import torch

own = False

D = 128                     # head dimension of the whole package
DEV = "cuda"


# --------------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------------
def listed():
    return [
        # a few chat turns at once, one of them a single token: the latency of a small call
        dict(name="prompt-turns", op="prompt", seqs=4, longest=45, packed=True, hq=12, hkv=4, layout="token"),
        # a server's prompts of different lengths, packed behind each other
        dict(name="prompt-packed", op="prompt", seqs=24, longest=1021, packed=True, hq=32, hkv=8, layout="token"),
        # a batch of prompts of one length, heads first
        dict(name="prompt-batch", op="prompt", seqs=4, longest=2048, packed=False, hq=40, hkv=8, layout="head"),
        # one long document
        dict(name="prompt-document", op="prompt", seqs=1, longest=8192, packed=True, hq=28, hkv=4, layout="token"),
        # the same turns' weights
        dict(name="weights-turns", op="weights", seqs=4, longest=45, packed=True, hq=12, hkv=4, layout="token", last=0),
        # packed prompts, every query counted
        dict(name="weights-packed", op="weights", seqs=24, longest=1021, packed=True, hq=32, hkv=8, layout="token", last=0),
        # a batch of long blocks of which the last queries alone decide what stays
        dict(name="weights-window", op="weights", seqs=8, longest=8192, packed=False, hq=32, hkv=8, layout="head", last=64),
        # one long document, every query counted
        dict(name="weights-document", op="weights", seqs=1, longest=8192, packed=True, hq=28, hkv=4, layout="token", last=0),
        # a decode step of 32 sequences, each with a cache of its own
        dict(name="weigh-decode", op="weigh", caches=32, fan=1, m=1, rows=512, hq=32, hkv=8, ragged=False),
        # drafts of 16 sequences behind one long prompt that they share, a different number for each
        dict(name="weigh-shared", op="weigh", caches=1, fan=16, m=5, rows=16384, hq=32, hkv=8, ragged=True),
        # the same decode step's eviction: one row joins every cache, one leaves
        dict(name="evict-step", op="evict", caches=32, hkv=8, m=1, budget=512, sink=4, recent=128, fresh=False),
        # long prompts into an empty cache, by the weights that their rows got
        dict(name="evict-prompt", op="evict", caches=4, hkv=8, m=8192, budget=4096, sink=4, recent=64, fresh=True),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "weights", "weights", "weigh", "evict"])
    most = [work(c) for c in listed() if c["op"] == op]
    while True:
        hq, hkv = rng.choice([(12, 4), (32, 8), (8, 8), (28, 4), (40, 8), (16, 2), (3, 1)])
        if op in ("prompt", "weights"):
            c = dict(op=op, seqs=_log(rng, 1, 64), longest=_log(rng, 1, 8192), packed=rng.random() < 0.7, hq=hq, hkv=hkv,
                     layout=rng.choice(["token", "head"]))
            if c["seqs"] * hq * c["longest"] ** 2 > 2e9:     # the plain form's logits
                continue
            if op == "weights":
                c["last"] = rng.choice([0, 0, _log(rng, 1, 512)])
        elif op == "weigh":
            c = dict(op=op, caches=_log(rng, 1, 64), fan=rng.choice([1, 1, _log(rng, 2, 64)]), m=rng.choice([1, 1, _log(rng, 2, 16)]),
                     rows=_log(rng, 1, 16384), hq=hq, hkv=hkv, ragged=rng.random() < 0.5)
            if c["caches"] * c["fan"] * c["m"] * hq * c["rows"] > 5e8:
                continue
        else:
            budget = _log(rng, 16, 4096)
            c = dict(op=op, caches=_log(rng, 1, 64), hkv=hkv, m=rng.choice([1, _log(rng, 1, 64), _log(rng, 1, 8192)]), budget=budget,
                     sink=rng.choice([0, 4]), recent=rng.choice([0, _log(rng, 1, budget // 2)]), fresh=rng.random() < 0.3)
        w = work(c)
        if w["bytes"] <= max(x["bytes"] for x in most) and w["flops"] <= max(x["flops"] for x in most):
            return c


def _lengths(c):
    """Tokens of every sequence: all the same in a batch, otherwise between 1 and the longest, which one has."""
    if not c["packed"]:
        return [c["longest"]] * c["seqs"]
    r = random.Random("%d.%d" % (c["seqs"], c["longest"]))
    got = [r.randint(1, c["longest"]) for _ in range(c["seqs"])]
    got[r.randrange(c["seqs"])] = c["longest"]
    if c["seqs"] > 2:
        got[0] = 1
    return got


def _news(c):
    """New tokens of every sequence of a decode step."""
    n = c["caches"] * c["fan"]
    if not c["ragged"]:
        return [c["m"]] * n
    r = random.Random("%d.%d.%d" % (n, c["m"], c["rows"]))
    got = [r.randint(0, c["m"]) for _ in range(n)]
    got[r.randrange(n)] = c["m"]
    return got


def work(c):
    if c["op"] in ("prompt", "weights"):
        lens = _lengths(c)
        tokens = sum(lens)
        last = c.get("last") or max(lens)
        first = [max(0, l - last) for l in lens]
        pairs = c["hq"] * sum((l - f) * (l + f + 1) // 2 for l, f in zip(lens, first))
        asked = c["hq"] * sum(l - f for l, f in zip(lens, first))
        if c["op"] == "prompt":
            return {"bytes": 2 * D * (2 * asked + 2 * c["hkv"] * tokens) + 4 * asked, "flops": 4 * D * pairs}
        return {"bytes": 2 * D * (asked + c["hkv"] * tokens) + 4 * asked + 4 * c["hkv"] * tokens, "flops": 2 * D * pairs}
    if c["op"] == "weigh":
        asked, rows = c["hq"] * sum(_news(c)), c["caches"] * c["hkv"] * c["rows"]
        return {"bytes": 2 * D * (asked + rows) + 4 * asked + 8 * rows, "flops": 2 * D * asked * c["rows"]}
    units, n = c["caches"] * c["hkv"], c["m"] + (0 if c["fresh"] else c["budget"])
    stay = min(n, c["budget"])
    came = min(c["m"], stay) if c["fresh"] else min(c["m"], max(c["recent"], 1))     # rows of the block that stay at least
    return {"bytes": units * (4 * n + came * (4 * D * 2 + 8)), "flops": units * n}


# --------------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------------
def _rows(g, batch, heads, m, layout, std=1.0):
    """bf16 rows [batch, heads, m, D]: dense, or a view of a projection's [batch, m, heads, D]."""
    shape = (batch, m, heads, D) if layout == "token" else (batch, heads, m, D)
    x = torch.randn(shape, device=DEV, generator=g).mul_(std).to(torch.bfloat16)
    return x.transpose(1, 2) if layout == "token" else x


def _spread(g, x):
    """Keys whose lengths differ, so that some are heavier than others."""
    return x.mul_(torch.randn(x.shape[:-1], device=DEV, generator=g).mul_(0.3).exp_()[..., None])


def prepare(c, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": c}
    if own:
        from kv_cache_token_bf16_gb300 import binding, prompt
    if c["op"] in ("prompt", "weights"):
        lens = _lengths(c)
        batch, m = (1, sum(lens)) if c["packed"] else (c["seqs"], c["longest"])
        s["q"] = _rows(g, batch, c["hq"], m, c["layout"], 1.5)
        s["k"] = _spread(g, _rows(g, batch, c["hkv"], m, c["layout"]))
        ends = torch.tensor(lens).cumsum(0)
        s["starts"] = torch.cat([torch.zeros(1, dtype=torch.int64), ends]).to(torch.int32).to(DEV) if c["packed"] else None
        if c["op"] == "prompt":
            s["v"] = _rows(g, batch, c["hkv"], m, c["layout"])
            s["out"] = torch.zeros(batch, m, c["hq"], D, dtype=torch.bfloat16, device=DEV).transpose(1, 2)
            s["lse"] = torch.zeros(batch, c["hq"], m, device=DEV)
        else:
            # as an attention over these keys leaves them, but for a little: the weights of a query need not add up to 1
            s["lse"] = torch.randn(batch, c["hq"], m, device=DEV, generator=g).mul_(0.2).add_(2.0)
            s["lse"] += torch.log1p(torch.cat([torch.arange(l) for l in lens]).to(DEV).float().view(batch, 1, m) if c["packed"]
                                    else torch.arange(m, device=DEV).float())
            s["weights"] = torch.zeros(batch, c["hkv"], m, device=DEV)
        if own:
            s["packing"] = prompt.Packing(s["starts"]) if c["packed"] else None
        return s
    b, h = c["caches"], c["hkv"]
    n = c["rows"] if c["op"] == "weigh" else 0 if c["fresh"] else c["budget"]
    s["k"], s["v"] = _spread(g, _rows(g, b, h, n, "head")), _rows(g, b, h, n, "head")
    s["pos"] = (torch.arange(n, device=DEV) * 3).to(torch.int32).expand(b, h, n).contiguous()
    s["score"] = torch.randn(b, h, n, device=DEV, generator=g).exp_()
    if own:
        budget = c.get("budget", c.get("rows"))
        s["cache"] = binding.EvictCache("attention", b, h, budget=budget, n_sink=c.get("sink", 0), recent=c.get("recent", 0),
                                        max_block=c["m"])
        s["cache"].set_state(s["k"], s["v"], s["pos"], s["score"], offset=3 * n)
    if c["op"] == "weigh":
        s["q"] = _rows(g, b * c["fan"], c["hq"], c["m"], "token", 1.5)
        s["lse"] = torch.randn(b * c["fan"], c["hq"], c["m"], device=DEV, generator=g).mul_(0.2).add_(2.0 + math.log(n))
        s["n_new"] = torch.tensor(_news(c), dtype=torch.int32, device=DEV) if c["ragged"] else None
    else:
        s["new_k"], s["new_v"] = _rows(g, b, h, c["m"], "head"), _rows(g, b, h, c["m"], "head")
        s["new_pos"] = (3 * n + torch.arange(c["m"], device=DEV)).to(torch.int32).expand(b, c["m"]).contiguous()
        s["new_score"] = torch.randn(b, h, c["m"], device=DEV, generator=g).exp_()
    return s


# --------------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------------
def run(s):
    c = s["case"]
    if own:
        from kv_cache_token_bf16_gb300 import prompt
        if c["op"] == "prompt":
            prompt.attention(s["q"], s["k"], s["v"], s["packing"], out=s["out"], lse=s["lse"])
            return s["out"], s["lse"]
        if c["op"] == "weights":
            return prompt.weights(s["q"], s["k"], s["lse"], s["packing"], last=c["last"], out=s["weights"])
        cache = s["cache"]
        if c["op"] == "weigh":
            cache.weigh(s["q"], s["lse"], n_new=s["n_new"])
            return cache.view()[3]
        if c["fresh"]:
            cache.reset()
        return cache.update_and_fetch(s["new_k"], s["new_v"], pos=s["new_pos"], score=s["new_score"])
    if c["op"] == "prompt":
        return _plain_prompt(s)
    if c["op"] == "weights":
        return _plain_weights(s)
    return _plain_weigh(s) if c["op"] == "weigh" else _plain_evict(s)


def _padded(s, x, w):
    """The last w tokens of every sequence [seqs, heads, w, ...] of x [batch, heads, m, ...], their indices in the sequence
    (negative: none) and, where the sequences are packed, in m."""
    c = s["case"]
    if not c["packed"]:
        m = x.shape[2]
        return x[:, :, m - w:], torch.arange(m - w, m, device=DEV).expand(c["seqs"], w), None
    starts = s["starts"].long()
    t = (starts[1:] - starts[:-1])[:, None] - w + torch.arange(w, device=DEV)
    at = starts[:-1, None] + t
    return x[0][:, at.clamp(min=0)].transpose(0, 1), t, at


def _plain_logits(s, w):
    """Scaled products of the last w queries of every sequence [seqs, hkv, group, w, longest], -inf where a query does not
    see a key. (Both are aligned to the sequences' ends.)"""
    c = s["case"]
    q, t, at = _padded(s, s["q"].float(), w)
    k, j, _ = _padded(s, s["k"].float(), c["longest"])
    n, hkv, l = k.shape[:3]
    z = (q.reshape(n, hkv, -1, D) @ k.transpose(2, 3)).mul_(1.0 / math.sqrt(D)).view(n, hkv, c["hq"] // hkv, w, l)
    hide = (j[:, None, :] > t[:, :, None]) | (j < 0)[:, None, :]
    return z.masked_fill_(hide[:, None, None], float("-inf")), t, at


def _put(x, y, t, at):
    """The rows y [seqs, heads, w, ...] into x [batch, heads, m, ...]."""
    if at is None:
        x.copy_(y)
    else:
        x[0].transpose(0, 1)[at[t >= 0]] = y.transpose(1, 2)[t >= 0]


def _plain_prompt(s):
    c = s["case"]
    z, t, at = _plain_logits(s, c["longest"])
    v, _, _ = _padded(s, s["v"].float(), c["longest"])
    n, hkv, g, l, _ = z.shape
    top = z.amax(-1, keepdim=True).clamp_(min=-1e30)
    p = z.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (top + total.log()).reshape(n, c["hq"], l)
    o = (p.view(n, hkv, g * l, l) @ v).view(n, hkv, g, l, D).div_(total).reshape(n, c["hq"], l, D).to(torch.bfloat16)
    _put(s["out"], o, t, at)
    _put(s["lse"], lse, t, at)
    return s["out"], s["lse"]


def _plain_weights(s):
    c = s["case"]
    w = min(c["last"] or c["longest"], c["longest"])
    z, t, _ = _plain_logits(s, w)
    lse, _, _ = _padded(s, s["lse"], w)
    n, hkv, g, _, l = z.shape
    # queries of sequences that have fewer than w see nothing: their rows are -inf
    got = z.sub_(lse.reshape(n, hkv, g, w, 1)).exp_().sum((2, 3))
    _, j, at = _padded(s, s["lse"], l)
    _put(s["weights"], got, j, at)
    return s["weights"]


def _plain_weigh(s):
    c = s["case"]
    b, h, n, f, m = c["caches"], c["hkv"], c["rows"], c["fan"], c["m"]
    q = s["q"].float().reshape(b, f, h, -1, m, D).permute(0, 2, 1, 3, 4, 5).reshape(b, h, -1, D)
    lse = s["lse"].reshape(b, f, h, -1, m)
    if s["n_new"] is not None:
        pad = torch.arange(m, device=DEV) >= s["n_new"].long().view(b, f, 1)
        lse = lse.masked_fill(pad[:, :, None, None], float("inf"))
    lse = lse.transpose(1, 2).reshape(b, h, -1, 1)
    s["score"] += ((q @ s["k"].float().transpose(2, 3)).mul_(1.0 / math.sqrt(D)) - lse).exp_().sum(2)
    return s["score"]


def _plain_evict(s):
    c = s["case"]
    if c["fresh"]:
        k, v, score = s["new_k"], s["new_v"], s["new_score"]
        pos = s["new_pos"][:, None].expand(-1, c["hkv"], -1)
    else:
        k, v, score = (torch.cat([s[x], s["new_" + x]], dim=2) for x in ("k", "v", "score"))
        pos = torch.cat([s["pos"], s["new_pos"][:, None].expand(-1, c["hkv"], -1)], dim=2)
    n = k.shape[2]
    if n <= c["budget"]:
        k, v, pos, score = (x.clone() for x in (k, v, pos, score))       # the cache's own rows
    else:
        at = torch.arange(n, device=DEV)
        rank = score.masked_fill((at < c["sink"]) | (at >= n - c["recent"]), float("inf"))
        keep = rank.sort(dim=-1, descending=True, stable=True).indices[..., :c["budget"]].sort(dim=-1).values
        pos, score = pos.gather(2, keep), score.gather(2, keep)
        wide = keep[..., None].expand(-1, -1, -1, D)
        k, v = k.gather(2, wide), v.gather(2, wide)
    s["k"], s["v"], s["pos"], s["score"] = k, v, pos, score
    return k, v, pos, score


# --------------------------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------------------------
def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "evict":
        return _exact_evict(c, s)
    if work(c)["flops"] > 2e12:
        return None
    return _exact_weigh(c, s) if c["op"] == "weigh" else _exact_prompt(c, s)


def _exact_prompt(c, s):
    """Sequence by sequence and head by head."""
    g = c["hq"] // c["hkv"]
    lens = _lengths(c)
    whole = c["op"] == "prompt"
    lse = s["lse"].double().clone()
    out = s["out"].double().clone() if whole else s["weights"].double().clone()
    begin = 0
    for i, l in enumerate(lens):
        b, a = (0, begin) if c["packed"] else (i, 0)
        begin += l
        unseen = torch.ones(l, l, dtype=torch.bool, device=DEV).triu_(1)
        for h in range(c["hq"]):
            z = s["q"][b, h, a:a + l].double() @ s["k"][b, h // g, a:a + l].double().T / math.sqrt(D)
            z[unseen] = -math.inf
            if whole:
                lse[b, h, a:a + l] = torch.logsumexp(z, dim=-1)
                out[b, h, a:a + l] = torch.softmax(z, dim=-1) @ s["v"][b, h // g, a:a + l].double()
            else:
                w = torch.exp(z - s["lse"][b, h, a:a + l].double()[:, None])
                out[b, h // g, a:a + l] += w[max(0, l - c["last"]) if c["last"] else 0:].sum(0)
    return (out, lse) if whole else out


def _exact_weigh(c, s):
    """Sequence by sequence and head by head."""
    g = c["hq"] // c["hkv"]
    score = s["score"].double().clone()
    for i, n in enumerate(_news(c)):
        b = i // c["fan"]
        for h in range(c["hq"]):
            z = s["q"][i, h, :n].double() @ s["k"][b, h // g].double().T / math.sqrt(D)
            score[b, h // g] += torch.exp(z - s["lse"][i, h, :n].double()[:, None]).sum(0)
    return score


def _exact_evict(c, s):
    """Row by row: the protected ones, then the heaviest, the first of equals."""
    new = [s["new_" + x].cpu() for x in ("k", "v", "score")] + [s["new_pos"].cpu()[:, None].expand(-1, c["hkv"], -1)]
    old = [s[x].cpu() for x in ("k", "v", "score", "pos")]
    k, v, score, pos = new if c["fresh"] else [torch.cat(x, dim=2) for x in zip(old, new)]
    n = k.shape[2]
    stay = min(n, c["budget"])
    keep = torch.empty(c["caches"], c["hkv"], stay, dtype=torch.int64)
    for b in range(c["caches"]):
        for h in range(c["hkv"]):
            w = score[b, h].double().tolist()
            safe = set(range(min(c["sink"], n))) | set(range(max(0, n - c["recent"]), n)) if n > stay else set(range(n))
            rest = sorted((i for i in range(n) if i not in safe), key=lambda i: (-w[i], i))
            keep[b, h] = torch.tensor(sorted(safe | set(rest[:stay - len(safe)])))
    wide = keep[..., None].expand(-1, -1, -1, D)
    got = k.gather(2, wide).double(), v.gather(2, wide).double(), pos.gather(2, keep), score.gather(2, keep).double()
    return tuple(x.to(DEV) for x in got)
