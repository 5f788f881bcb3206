"""Workloads of the operators around the kept cache: position rotation, appending to pages and
attention of a batch over a shared prefix and its own pages.

``listed()`` names the workloads, ``draw`` makes more of the same ranges, ``prepare`` makes the
inputs of one on the GPU and ``run`` makes one pass: with ``own`` set through the package's entry
points, otherwise in plain torch operations in 32 bits. ``exact`` computes the same results from the
definitions in 64 bits, and ``work`` counts the bytes and operations that no pass can do without.

The sizes are those of this repository's workloads where it has them: 8 KV heads of 128 elements with
several query heads each; batches of 4, 8 and 32 sequences; kept prefixes (budgets) of 1024 to 4096
rows and caches of 16384; blocks of 512 to 8192 tokens.
"""
import math
import random

import torch

own = False

D = 128                     # head dimension of the whole package
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# --------------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------------
def listed():
    return [
        # one decode step of 32 sequences: the queries and keys of the new tokens
        dict(name="rotate-decode", op="rotate", batch=32, m=1, hq=32, hkv=8, dtype="bf16", rotary=128, pairs="half",
             axes=1, order="blocks", base=500000.0, far=4096, transpose=False, layout="token"),
        # a long prompt of text and frames: time, height and width positions, projections laid out by token
        dict(name="rotate-frames", op="rotate", batch=1, m=8192, hq=28, hkv=4, dtype="bf16", rotary=128, pairs="half",
             axes=3, order="blocks", base=1000000.0, far=16384, transpose=False, layout="token"),
        # gradients of a partly rotated head in fp32, adjacent pairs, odd length, far positions
        dict(name="rotate-gradient", op="rotate", batch=4, m=1023, hq=32, hkv=8, dtype="fp32", rotary=64, pairs="adjacent",
             axes=3, order="turns", base=10000.0, far=131072, transpose=True, layout="head"),
        # one decode step of 32 sequences into small pages
        dict(name="append-decode", op="append", batch=32, m=1, hq=32, hkv=8, dtype="bf16", rotary=128, pairs="half",
             axes=1, order="blocks", base=500000.0, rows=2048, page=16, ragged=False, pos="index", layout="token"),
        # prompts of different lengths, padded to the longest, one of them empty
        dict(name="append-prompts", op="append", batch=8, m=2048, hq=32, hkv=8, dtype="bf16", rotary=128, pairs="half",
             axes=3, order="blocks", base=1000000.0, rows=4096, page=64, ragged=True, pos="given", layout="token"),
        # an fp32 block of odd length, partly rotated
        dict(name="append-fp32", op="append", batch=3, m=1021, hq=8, hkv=8, dtype="fp32", rotary=96, pairs="adjacent",
             axes=1, order="blocks", base=10000.0, rows=1537, page=128, ragged=True, pos="given", layout="head"),
        # a few sequences that have just begun behind a shared prompt: the latency of a small step
        dict(name="attend-few", op="attend", batch=4, m=1, hq=12, hkv=4, prefix=1024, groups=1, rows=64, page=16,
             ragged=False),
        # a decode step of 32 sequences behind one shared prompt
        dict(name="attend-decode", op="attend", batch=32, m=1, hq=32, hkv=8, prefix=4096, groups=1, rows=512, page=16,
             ragged=False),
        # many sequences behind a long shared prompt
        dict(name="attend-many", op="attend", batch=128, m=1, hq=32, hkv=8, prefix=16384, groups=1, rows=1024, page=64,
             ragged=False),
        # draft tokens to verify, a different number for each sequence
        dict(name="attend-drafts", op="attend", batch=32, m=5, hq=32, hkv=8, prefix=8192, groups=1, rows=777, page=32,
             ragged=True),
        # eight prompts, evicted to a budget of 2048 rows, four answers of each
        dict(name="attend-answers", op="attend", batch=32, m=1, hq=40, hkv=8, prefix=2048, groups=8, rows=512, page=64,
             ragged=False),
        # the sequences' own questions, prefilled behind the shared prompt
        dict(name="attend-questions", op="attend", batch=8, m=509, hq=32, hkv=8, prefix=4096, groups=1, rows=700, page=64,
             ragged=True),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _limits(op):
    cs = [work(c) for c in listed() if c["op"] == op]
    return max(w["bytes"] for w in cs), max(w["flops"] for w in cs)


def draw(rng):
    op = rng.choice(["rotate", "append", "attend", "attend"])
    max_bytes, max_flops = _limits(op)
    while True:
        hq, hkv = rng.choice([(12, 4), (32, 8), (8, 8), (28, 4), (40, 8), (16, 2), (3, 1)])
        if op == "attend":
            groups = rng.choice([1, 1, 1, 2, 8])
            c = dict(op=op, batch=groups * _log(rng, 1, 128 // groups), m=rng.choice([1, 1, 1, 2, 5, _log(rng, 3, 512)]),
                     hq=hq, hkv=hkv, prefix=rng.choice([0, 1, 2, 3, 4, 5]) and _log(rng, 1, 16384), groups=groups,
                     rows=0, page=rng.choice([16, 32, 64, 128]), ragged=rng.random() < 0.5)
            c["rows"] = c["m"] + _log(rng, 1, 1024) - 1
        else:
            axes = rng.choice([1, 1, 2, 3])
            c = dict(op=op, batch=_log(rng, 1, 64), m=rng.choice([1, 1, _log(rng, 2, 8192), _log(rng, 2, 8192)]), hq=hq,
                     hkv=hkv, dtype=rng.choice(["bf16", "bf16", "fp32"]), rotary=rng.choice([128, 128, 64, 96, 32, 20]),
                     pairs=rng.choice(["half", "adjacent"]), axes=axes, order=rng.choice(["blocks", "turns"]),
                     base=rng.choice([10000.0, 500000.0, 1000000.0]), layout=rng.choice(["token", "head"]))
            if op == "rotate":
                c.update(far=_log(rng, 1024, 1 << 20), transpose=rng.random() < 0.3)
            else:
                c.update(rows=c["m"] + _log(rng, 1, 2048) - 1, page=rng.choice([16, 32, 64, 128]), ragged=rng.random() < 0.5,
                         pos=rng.choice(["index", "given"]))
        w = work(c)
        if w["bytes"] <= max_bytes and w["flops"] <= max_flops:
            return c


def _counts(c):
    """(n_new, lens) of a case's sequences: new rows and rows with them, Python lists."""
    r = random.Random("%d.%d.%d.%d" % (c["batch"], c["m"], c["rows"], c["page"]))
    n_new = [r.randint(0, c["m"]) if c["ragged"] else c["m"] for _ in range(c["batch"])]
    if c["ragged"]:
        n_new[r.randrange(c["batch"])] = c["m"]          # the one that the others are padded to
    lens = [r.randint(n, c["rows"]) for n in n_new]
    return n_new, lens


def work(c):
    e = 4 if c.get("dtype") == "fp32" else 2
    if c["op"] == "rotate":
        rows = c["batch"] * c["m"] * (c["hq"] + c["hkv"])
        return {"bytes": 2 * rows * D * e + 4 * c["axes"] * c["batch"] * c["m"], "flops": 3 * rows * c["rotary"]}
    n_new, lens = _counts(c)
    if c["op"] == "append":
        tokens = sum(n_new)
        pos = 4 * c["axes"] * tokens if c["pos"] == "given" else 0
        return {"bytes": 2 * tokens * (c["hq"] + 2 * c["hkv"]) * D * e + pos + 8 * c["batch"],
                "flops": 3 * tokens * (c["hq"] + c["hkv"]) * c["rotary"]}
    queries = sum(n_new) * c["hq"]
    pairs = queries * c["prefix"]
    seen = 0
    for n, l in zip(n_new, lens):
        pairs += c["hq"] * sum(l - n + t + 1 for t in range(n))
        seen += l if n else 0
    kv = 2 * c["hkv"] * D * 2 * (c["groups"] * c["prefix"] + seen)
    return {"bytes": 2 * queries * D * 2 + kv + 8 * c["batch"], "flops": 4 * D * pairs}


# --------------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _rows(g, batch, heads, m, dtype, layout, std=1.0):
    """Rows [batch, heads, m, D]: dense, or a view of a projection's [batch, m, heads, D]."""
    if layout == "token":
        x = torch.randn(batch, m, heads, D, device=DEV, generator=g).mul_(std).to(dtype)
        return x.transpose(1, 2)
    return torch.randn(batch, heads, m, D, device=DEV, generator=g).mul_(std).to(dtype)


def _inv_freq(c):
    """Radians a position of every pair, as a model holds them: fp32 values."""
    i = torch.arange(0, c["rotary"], 2, dtype=torch.float64)
    return (1.0 / c["base"] ** (i / c["rotary"])).float()


def _axis(c):
    """Position axis of every pair: the axes' sections one behind the other, or taking turns."""
    n = c["rotary"] // 2
    if c["order"] == "turns":
        return [i % c["axes"] for i in range(n)]
    return [min(i * c["axes"] // n, c["axes"] - 1) for i in range(n)]


def _positions(g, c, far):
    """Positions [axes, batch, m]: time runs on, the other axes repeat inside a frame."""
    b, m = c["batch"], c["m"]
    start = torch.randint(0, max(1, far - m), (b, 1), device=DEV, generator=g)
    t = start + torch.arange(m, device=DEV)[None, :]
    pos = [t]
    for a in range(1, c["axes"]):
        pos.append(start + (torch.arange(m, device=DEV)[None, :] // (24 ** (a - 1))) % 24)
    return torch.stack(pos).to(torch.int32).contiguous()


def _pool(g, c, dtype, lens):
    """K and V pages, the table of every sequence's pages (in no order) and its page count."""
    p = c["page"]
    width = -(-c["rows"] // p)
    n_pages = c["batch"] * width + 3
    shape = (n_pages, c["hkv"], p, D)
    scale = torch.randn(n_pages, c["hkv"], p, 1, device=DEV, generator=g).mul_(0.3).exp_()
    k = torch.randn(shape, device=DEV, generator=g).mul_(scale).to(dtype)
    v = torch.randn(shape, device=DEV, generator=g).to(dtype)
    order = torch.randperm(n_pages, device=DEV, generator=g)[:c["batch"] * width]
    return k, v, order.view(c["batch"], width).to(torch.int32).contiguous()


def prepare(c, seed):
    g = _gen(seed)
    s = {"case": c}
    if own:
        from kv_cache_token_bf16_gb300 import paged
    if c["op"] in ("rotate", "append"):
        dtype = TYPES[c["dtype"]]
        s["inv_freq"], s["axis"] = _inv_freq(c).to(DEV), torch.tensor(_axis(c), device=DEV)
        if own:
            s["rotary"] = paged.Rotary(c["rotary"], inv_freq=_inv_freq(c), axis=_axis(c), n_axes=c["axes"],
                                       pairs=c["pairs"])
        s["q"] = _rows(g, c["batch"], c["hq"], c["m"], dtype, c["layout"])
        s["k"] = _rows(g, c["batch"], c["hkv"], c["m"], dtype, c["layout"])
    if c["op"] == "rotate":
        s["pos"] = _positions(g, c, c["far"])
        return s
    n_new, lens = _counts(c)
    s["n_new"] = torch.tensor(n_new, dtype=torch.int32, device=DEV)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    if c["op"] == "append":
        s["v"] = _rows(g, c["batch"], c["hkv"], c["m"], dtype, c["layout"])
        s["pos"] = _positions(g, c, 65536) if c["pos"] == "given" else None
        s["q_out"] = torch.zeros(c["batch"], c["hq"], c["m"], D, dtype=dtype, device=DEV)
    else:
        dtype = torch.bfloat16
        s["q"] = _rows(g, c["batch"], c["hq"], c["m"], dtype, "token", 1.5)
        scale = torch.randn(c["groups"], c["hkv"], c["prefix"], 1, device=DEV, generator=g).mul_(0.3).exp_()
        s["pk"] = torch.randn(c["groups"], c["hkv"], c["prefix"], D, device=DEV, generator=g).mul_(scale).to(dtype)
        s["pv"] = torch.randn(c["groups"], c["hkv"], c["prefix"], D, device=DEV, generator=g).to(dtype)
        s["out"] = torch.zeros(c["batch"], c["m"], c["hq"], D, dtype=dtype, device=DEV).transpose(1, 2)
        s["lse"] = torch.zeros(c["batch"], c["hq"], c["m"], device=DEV)
    s["k_pages"], s["v_pages"], s["table"] = _pool(g, c, dtype, lens)
    if own:
        s["cache"] = paged.PagedCache(k_pages=s["k_pages"], v_pages=s["v_pages"], table=s["table"], lens=s["lens"])
    return s


# --------------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------------
def run(s):
    c = s["case"]
    n_new = s["n_new"] if c["op"] != "rotate" and c["ragged"] else None
    if own:
        from kv_cache_token_bf16_gb300 import paged
        if c["op"] == "rotate":
            return paged.rotate(s["rotary"], (s["q"], s["k"]), pos=s["pos"], transpose=c["transpose"])
        if c["op"] == "append":
            s["cache"].append(s["k"], s["v"], rotary=s["rotary"], pos=s["pos"], n_new=n_new, q=s["q"], q_out=s["q_out"])
            return s["k_pages"], s["v_pages"], s["q_out"]
        s["cache"].attend(s["q"], prefix=(s["pk"], s["pv"]), n_new=n_new, out=s["out"], lse=s["lse"])
        return s["out"], s["lse"]
    if c["op"] == "rotate":
        return _plain_rotate(s, s["q"], s["pos"]), _plain_rotate(s, s["k"], s["pos"])
    if c["op"] == "append":
        return _plain_append(s)
    return _plain_attend(s)


def _plain_rotate(s, x, pos):
    c = s["case"]
    r = c["rotary"]
    angle = pos.double()[s["axis"]].permute(1, 2, 0) * s["inv_freq"].double()          # [batch, m, pairs]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if c.get("transpose"):
        sin = -sin
    xf = x.float()
    if c["pairs"] == "half":
        a, b = xf[..., :r // 2], xf[..., r // 2:r]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos, xf[..., r:]], dim=-1)
    else:
        a, b = xf[..., 0:r:2], xf[..., 1:r:2]
        y = torch.cat([torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2), xf[..., r:]], dim=-1)
    return y.to(x.dtype)


def _plain_append(s):
    c = s["case"]
    p, m = c["page"], c["m"]
    t = torch.arange(m, device=DEV)
    new = s["n_new"].long()[:, None]
    j = s["lens"].long()[:, None] - new + t                                            # index in the sequence
    pos = s["pos"] if s["pos"] is not None else j.expand(c["axes"], -1, -1)
    valid = t < new
    k, q = _plain_rotate(s, s["k"], pos), _plain_rotate(s, s["q"], pos)
    page = torch.gather(s["table"].long(), 1, (j // p).clamp(0, s["table"].shape[1] - 1))
    bi, ti = valid.nonzero(as_tuple=True)
    pg, row = page[bi, ti], (j % p)[bi, ti]
    s["k_pages"][pg, :, row] = k[bi, :, ti]
    s["v_pages"][pg, :, row] = s["v"][bi, :, ti]
    s["q_out"][bi, :, ti] = q[bi, :, ti]
    return s["k_pages"], s["v_pages"], s["q_out"]


def _own_rows(s, pages, dtype):
    """The sequences' own rows, gathered: [batch, hkv, width * page, D]."""
    x = pages[s["table"].long()].to(dtype)                                             # [batch, width, hkv, page, D]
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _plain_attend(s):
    c = s["case"]
    b, m, hq, hkv, gr = c["batch"], c["m"], c["hq"], c["hkv"], c["groups"]
    g = hq // hkv
    scale = 1.0 / math.sqrt(D)
    q = s["q"].float().contiguous()
    # scores against the prefix, all sequences of a group in one product for each KV head
    qg = q.reshape(gr, b // gr, hkv, g, m, D).permute(0, 2, 1, 3, 4, 5).reshape(gr, hkv, -1, D)
    z0 = (qg @ s["pk"].float().transpose(2, 3)) * scale                                # [gr, hkv, rows, prefix]
    ko, vo = _own_rows(s, s["k_pages"], torch.float32), _own_rows(s, s["v_pages"], torch.float32)
    qo = q.reshape(b, hkv, g * m, D)
    z1 = (qo @ ko.transpose(2, 3)) * scale                                             # [b, hkv, g * m, own]
    t = torch.arange(m, device=DEV)
    last = s["lens"].long()[:, None] - s["n_new"].long()[:, None] + t                  # [b, m]
    hide = torch.arange(ko.shape[2], device=DEV) > last[..., None]                     # [b, m, own]
    z1 = z1.reshape(b, hkv, g, m, -1).masked_fill(hide[:, None, None], float("-inf")).reshape(b, hkv, g * m, -1)
    mx0 = z0.amax(-1) if c["prefix"] else z0.new_full(z0.shape[:-1], float("-inf"))
    mx0 = mx0.reshape(gr, hkv, b // gr, g * m).transpose(1, 2).reshape(b, hkv, g * m)
    mx = torch.maximum(mx0, z1.amax(-1))
    mx = torch.where(mx == float("-inf"), torch.zeros_like(mx), mx)
    mxg = mx.reshape(gr, b // gr, hkv, g * m).transpose(1, 2).reshape(gr, hkv, -1, 1)
    p0, p1 = torch.exp(z0 - mxg), torch.exp(z1 - mx[..., None])
    o0, l0 = p0 @ s["pv"].float(), p0.sum(-1)
    o0 = o0.reshape(gr, hkv, b // gr, g * m, D).transpose(1, 2).reshape(b, hkv, g * m, D)
    l0 = l0.reshape(gr, hkv, b // gr, g * m).transpose(1, 2).reshape(b, hkv, g * m)
    seen = ~hide.all(1)                                                                # rows that some query sees
    o1 = p1 @ vo.masked_fill(~seen[:, None, :, None], 0.0)
    l = l0 + p1.sum(-1)
    o = (o0 + o1) / torch.where(l > 0, l, torch.ones_like(l))[..., None]
    lse = mx + torch.log(l)
    valid = (t < s["n_new"].long()[:, None])[:, None]                                  # [b, 1, m]
    s["out"].copy_(torch.where(valid[..., None], o.reshape(b, hq, m, D).to(s["out"].dtype), s["out"]))
    s["lse"].copy_(torch.where(valid, lse.reshape(b, hq, m), s["lse"]))
    return s["out"], s["lse"]


# --------------------------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------------------------
def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "rotate":
        return tuple(_exact_rotate(c, x, s["pos"]) for x in (s["q"], s["k"]))
    if c["op"] == "append":
        return _exact_append(c, s)
    if work(c)["flops"] > 4e12:
        return None
    return _exact_attend(c, s)


def _exact_rotate(c, x, pos):
    """Multiply each pair, as a complex number, by exp(i * angle)."""
    r = c["rotary"]
    freq = _inv_freq(c).tolist()
    phase = torch.stack([pos[a].double() * w for a, w in zip(_axis(c), freq)], dim=-1)     # [batch, m, pairs]
    turn = torch.polar(torch.ones_like(phase), -phase if c.get("transpose") else phase).unsqueeze(1)
    first = list(range(r // 2)) if c["pairs"] == "half" else list(range(0, r, 2))
    second = [i + (r // 2 if c["pairs"] == "half" else 1) for i in first]
    y = x.double().clone()
    z = torch.complex(y[..., first], y[..., second]) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_append(c, s):
    n_new, lens = _counts(c)
    kp, vp, qo = s["k_pages"].double(), s["v_pages"].double(), s["q_out"].double()
    table = s["table"].tolist()
    for b in range(c["batch"]):
        n = n_new[b]
        if not n:
            continue
        idx = list(range(lens[b] - n, lens[b]))
        at = torch.tensor(idx, device=DEV)
        pos = s["pos"][:, b:b + 1, :n] if s["pos"] is not None else at.view(1, 1, n).expand(c["axes"], 1, n)
        pages = torch.tensor([table[b][i // c["page"]] for i in idx], device=DEV)
        rows = at % c["page"]
        kp[pages, :, rows] = _exact_rotate(c, s["k"][b:b + 1, :, :n], pos)[0].transpose(0, 1)
        vp[pages, :, rows] = s["v"][b, :, :n].double().transpose(0, 1)
        qo[b, :, :n] = _exact_rotate(c, s["q"][b:b + 1, :, :n], pos)[0]
    return kp, vp, qo


def _exact_attend(c, s):
    """Sequence by sequence: the visible rows in one list, one softmax over them."""
    n_new, lens = _counts(c)
    g = c["hq"] // c["hkv"]
    out, lse = s["out"].double().clone(), s["lse"].double().clone()
    for b in range(c["batch"]):
        n, l = n_new[b], lens[b]
        if not n:
            continue
        grp = b // (c["batch"] // c["groups"])
        pages = s["table"][b].long()
        rows = [x[pages].transpose(0, 1).flatten(1, 2)[:, :l].double() for x in (s["k_pages"], s["v_pages"])]
        k = torch.cat([s["pk"][grp].double(), rows[0]], dim=1)                         # [hkv, prefix + l, D]
        v = torch.cat([s["pv"][grp].double(), rows[1]], dim=1)
        total = c["prefix"] + l
        reach = c["prefix"] + l - n + 1 + torch.arange(n, device=DEV)                  # visible rows of query t
        unseen = torch.arange(total, device=DEV)[None, :] >= reach[:, None]
        for h in range(c["hq"]):
            z = s["q"][b, h, :n].double() @ k[h // g].T / math.sqrt(D)
            z[unseen] = -math.inf
            lse[b, h, :n] = torch.logsumexp(z, dim=-1)
            out[b, h, :n] = torch.softmax(z, dim=-1) @ v[h // g]
    return out, lse
