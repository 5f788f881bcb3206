"""Attention over a shared prefix and own pages, against the definition in 64 bits."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from kv_cache_token_bf16_gb300 import binding, paged  # noqa: E402
from tests.paged_util import D, attend64, attend_bounds, gather, inv_freq, rotate64  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def randn(seed, *shape, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (std * torch.randn(*shape, generator=g)).to(torch.bfloat16).cuda()


def make(seed, B, hq, h, m, n_prefix, groups, page, lens, new=None, layout="token"):
    s = {"q": randn(seed, B, m, hq, D, std=1.5).transpose(1, 2)}
    if layout == "head":
        s["q"] = s["q"].contiguous()
    s["prefix"] = (randn(seed + 1, groups, h, n_prefix, D), randn(seed + 2, groups, h, n_prefix, D)) if n_prefix else None
    s["new"] = torch.tensor(new, dtype=torch.int32).cuda() if new is not None else None
    if lens is not None:
        width = max(1, -(-max(lens) // page))
        n_pages = B * width + 2
        g = torch.Generator().manual_seed(seed + 3)
        s["table"] = torch.randperm(n_pages, generator=g)[:B * width].view(B, width).to(torch.int32).cuda()
        s["kp"], s["vp"] = randn(seed + 4, n_pages, h, page, D), randn(seed + 5, n_pages, h, page, D)
        s["own"] = list(zip(gather(s["kp"], s["table"], lens), gather(s["vp"], s["table"], lens)))
        # rows that nobody may read hold NaN and infinities
        junk = torch.tensor([math.nan, math.inf, -math.inf, 3e38], dtype=torch.bfloat16).repeat(D // 4).cuda()
        live = torch.zeros(n_pages, page, dtype=torch.bool)
        for b, n in enumerate(lens):
            for j in range(n):
                live[int(s["table"][b, j // page]), j % page] = True
        dead = ~live[:, None, :].expand(-1, h, -1).cuda()
        s["kp"][dead], s["vp"][dead] = junk, junk
        s["cache"] = paged.PagedCache(k_pages=s["kp"], v_pages=s["vp"], table=s["table"],
                                      lens=torch.tensor(lens, dtype=torch.int32).cuda())
    return s


def attend(s, scale=None, **kw):
    B, hq, m, _ = s["q"].shape
    lse = torch.full((B, hq, m), 7.0, device="cuda")
    if s.get("cache"):
        out = s["cache"].attend(s["q"], prefix=s["prefix"], n_new=s["new"], scale=scale, lse=lse, **kw)
        s["cache"].sync()
    else:
        out = paged.shared_attention(s["q"], prefix=s["prefix"], n_new=s["new"], scale=scale, lse=lse, **kw)
    return out, lse


def check(s, out, lse, scale=None, weights=2.0 ** -8):
    """Weights may be rounded to bf16 (half a step, 2^-8) before they meet the values."""
    new = s["new"].tolist() if s["new"] is not None else None
    own = s.get("own")
    ro, rl, wt = attend64(s["q"], s["prefix"], own, new, scale)
    kmax = max([float(k.double().norm(dim=-1).max()) for k in ([s["prefix"][0]] if s["prefix"] else []) +
                ([k for k, _ in own if k.numel()] if own else [])] or [0.0])
    bo, bl = attend_bounds(s["q"], kmax, ro, rl, wt, scale, weights)
    go, gl = out.double().cpu(), lse.double().cpu()
    pad = ro.isnan()
    assert bool((go[pad] == 0).all()) and bool((gl[rl.isnan()] == 7.0).all())
    eo = (go - ro).abs()
    assert bool((eo[~pad] <= bo[~pad]).all()), float((eo / bo)[~pad].max())
    fin = rl.isfinite()
    assert bool((gl[rl == -math.inf] == -math.inf).all())
    assert bool(((gl - rl).abs()[fin] <= bl[fin]).all()), float(((gl - rl).abs() / bl)[fin].max())


CASES = [
    # B, hq, h, m, n_prefix, groups, page, lens, new
    (1, 1, 1, 1, 1, 1, 16, None, None),
    (1, 1, 1, 1, 0, 1, 16, [1], None),
    (1, 8, 1, 1, 300, 1, 16, [16], None),
    (3, 12, 4, 1, 129, 1, 16, [15, 17, 128], None),
    (4, 6, 2, 1, 128, 2, 32, [0, 1, 33, 129], None),
    (4, 4, 4, 1, 0, 1, 64, [0, 5, 64, 400], None),
    (5, 8, 2, 3, 77, 1, 16, [3, 20, 130, 0, 16], [3, 2, 1, 0, 3]),
    (2, 14, 2, 7, 260, 2, 128, [7, 300], None),
    (2, 4, 1, 33, 40, 1, 256, [33, 290], [33, 12]),
    (6, 16, 2, 1, 1000, 3, 16, None, None),
    (40, 8, 2, 1, 200, 1, 16, [b % 50 for b in range(40)], None),
    (3, 4, 2, 2, 0, 1, 16, [1, 0, 40], [2, 2, 2]),     # a query before the first row sees nothing
    (2, 64, 1, 2, 513, 1, 64, [3, 700], None),
    (3, 4, 2, 130, 100, 1, 64, [130, 400, 131], [130, 129, 3]),
    # more units than CTAs: the wide kernel's parts of units, with a group that has no work in some
    (12, 8, 8, 300, 200, 1, 16, [300, 20, 700, 3, 0, 310, 256, 299, 33, 64, 1, 500],
     [300, 0, 290, 3, 0, 44, 256, 2, 33, 0, 1, 257]),
    (64, 160, 8, 1, 100, 32, 16, None, None),
    (64, 160, 8, 1, 300, 32, 16, [b % 40 for b in range(64)], [b % 2 for b in range(64)]),
    (2, 8, 2, 300, 0, 1, 128, [300, 1200], None),
    (3, 4, 1, 64, 0, 1, 32, [0, 64, 30], [64, 64, 64]),
    (2, 36, 1, 2, 700, 2, 16, [2, 450], None),
    (32, 32, 8, 5, 2000, 1, 32, [5 + (b * 97) % 770 for b in range(32)], [(b * 7) % 6 for b in range(32)]),
    (24, 40, 8, 1, 650, 8, 16, [(b * 131) % 500 for b in range(24)], [(b * 5) % 2 for b in range(24)]),
    (5, 2, 1, 300, 1, 1, 16, None, [300, 0, 1, 129, 128]),
    # long prefixes: few rows in the wide kernel, sequences of more than 128 rows in tiles that they share
    (2, 8, 4, 1, 4200, 1, 16, [1, 40], None),
    (3, 8, 2, 40, 2100, 1, 16, [40, 170, 300], None),
    (3, 8, 2, 40, 2100, 1, 16, [40, 170, 300], [40, 33, 0]),
    (4, 12, 2, 50, 2300, 2, 64, [50, 51, 260, 0], [50, 1, 50, 0]),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c[:7]))
@pytest.mark.parametrize("layout", ["token", "head"])
def test_attention_matches_the_definition(case, layout):
    s = make(100, *case, layout=layout)
    out, lse = attend(s, out=torch.zeros(s["q"].shape, dtype=torch.bfloat16, device="cuda"))
    check(s, out, lse)


@pytest.mark.parametrize("scale", [0.3, -0.05, 1e-3])
@pytest.mark.parametrize("hq", [8, 40, 200], ids=["few", "wide", "joint"])
def test_other_scales(scale, hq):
    s = make(120, 3, hq, 2, 2, 150, 1, 16, [2, 40, 133])
    check(s, *attend(s, scale=scale), scale=scale)


@pytest.mark.parametrize("hq", [8, 100, 260], ids=["few", "wide", "joint"])
def test_large_logits_keep_their_order(hq):
    # logits up to hundreds: a running maximum that moves by far, weights that vanish
    s = make(121, 4, hq, 2, 1, 700, 1, 16, [1, 100, 300, 17])
    s["q"].mul_(30)
    check(s, *attend(s))


@pytest.mark.parametrize("hq", [8, 100, 260], ids=["few", "wide", "joint"])
def test_rising_logits(hq):
    # keys that grow along the prefix: the maximum rises at every step, by far more than fp32's range
    s = make(122, 4, hq, 2, 1, 1000, 1, 16, [1, 100, 300, 17])
    k = s["prefix"][0]
    q = s["q"]
    q.copy_(q.abs())
    k.copy_((k.abs() * torch.linspace(0.01, 60, 1000, device="cuda")[:, None]).to(torch.bfloat16))
    check(s, *attend(s))


@pytest.mark.parametrize("hq,m", [(8, 1), (40, 1), (100, 2), (260, 1), (400, 2)])
def test_spikes_anywhere(hq, m):
    # a maximum that jumps at some columns, for some rows: in any part of a step, first or last
    s = make(124, 4, hq, 2, m, 1500, 1, 16, [m, 100, 300, 17])
    k = s["prefix"][0]
    g = torch.Generator().manual_seed(125)
    for j in [31, 32, 63, 64, 127, 128, 191, 192, 1472, 1499] + torch.randint(0, 1500, (24,), generator=g).tolist():
        k[:, :, j] *= 20
    check(s, *attend(s))


@pytest.mark.parametrize("hq", [8, 100, 260], ids=["few", "wide", "joint"])
def test_results_are_the_same_every_time(hq):
    s = make(123, 7, hq, 2, 3, 3000, 1, 16, [3 + 100 * b for b in range(7)])
    a, la = attend(s)
    for _ in range(5):
        b, lb = attend(s)
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_kept_rows_of_a_cache():
    B, H, budget = 2, 2, 96
    cache = binding.EvictCache("knorm", B, H, budget=budget, max_block=256)
    k, v = randn(130, B, H, 256, D), randn(131, B, H, 256, D)
    kk, vv, _, _ = cache.update_and_fetch(k, v)
    for fan, hq in ((1, 2), (3, 8)):
        q = randn(132, B * fan, hq, 2, D)
        lse = torch.full((B * fan, hq, 2), 7.0, device="cuda")
        out = cache.attend(q, lse=lse)
        check({"q": q, "prefix": (kk.contiguous(), vv.contiguous()), "new": None}, out, lse)
    cache.sync()
    cache.close()


@pytest.mark.parametrize("hq,n_prefix", [(4, 60), (40, 60), (400, 60), (50, 2100)], ids=["few", "wide", "joint", "shared"])
def test_masked_rows_may_hold_anything(hq, n_prefix):
    # new rows with infinities and NaN: queries before them are untouched, queries from them on see them
    m, lens = 6, [6, 50]
    s = make(140, 2, hq, 2, m, n_prefix, 1, 16, lens)
    clean, _ = attend(s)
    page = 16
    for b, j, val in ((0, 4, math.nan), (1, 47, math.inf), (1, 49, math.nan)):
        pg, row = int(s["table"][b, j // page]), j % page
        s["vp"][pg, :, row] = val
        if val != val:
            s["kp"][pg, :, row] = val
    got, lse = attend(s)
    # sequence 0: row 4 is query 4's own; sequence 1: rows 47 and 49 are queries 3's and 5's
    assert torch.equal(got[0, :, :4], clean[0, :, :4])
    assert bool(got[0, :, 4:].isnan().all()) and bool(lse[0, :, 4:].isnan().all())
    ref = attend64(s["q"][1:, :, :3], s["prefix"], [(s["own"][1][0][:, :47], s["own"][1][1][:, :47])])
    e = (got[1:, :, :3].double().cpu() - ref[0]).abs()
    assert bool((e <= attend_bounds(s["q"][1:, :, :3], 20.0, *ref, weights=2.0 ** -8)[0]).all())
    assert bool((got[1, :, 3:5] == math.inf).all())
    assert bool(got[1, :, 5].isnan().all())


@pytest.mark.parametrize("hq", [2, 50, 200], ids=["few", "wide", "joint"])
def test_visible_infinite_logits(hq):
    s = make(141, 1, hq, 1, 1, 40, 1, 16, [20])
    s["prefix"][0][0, 0, 3] = math.inf          # some logit is an infinity or NaN: so is the result
    out, lse = attend(s)
    assert bool(out.isnan().all()) and bool((lse.isnan() | (lse == math.inf)).all())


def test_empty_everything():
    q = randn(142, 2, 4, 3, D)
    c = paged.PagedCache(n_pages=2, page_size=16, n_kv_heads=2, batch=2, max_rows=16)
    lse = torch.zeros(2, 4, 3, device="cuda")
    out = c.attend(q, out=torch.full_like(q, 5.0), lse=lse)
    c.sync()
    assert not bool(out.any()) and bool((lse == -math.inf).all())
    k = torch.zeros(1, 2, 0, D, dtype=torch.bfloat16, device="cuda")
    out = paged.shared_attention(q, prefix=(k, k), out=torch.full_like(q, 5.0), lse=lse)
    assert not bool(out.any())
    assert paged.shared_attention(q[:, :, :0], prefix=(k, k)).shape == (2, 4, 0, D)


@pytest.mark.parametrize("hq", [4, 40, 400], ids=["few", "wide", "joint"])
def test_only_padding(hq):
    s = make(144, 3, hq, 2, 4, 200, 1, 16, [0, 3, 70], [0, 0, 0])
    out, lse = attend(s, out=torch.full_like(s["q"], 5.0))
    assert bool((out == 5).all()) and bool((lse == 7).all())


def test_the_largest_batch():
    n = 4096
    s = make(145, n, 4, 2, 2, 130, 4, 16, [b * 7 % 41 for b in range(n)], [min(2, b * 7 % 41) for b in range(n)])
    out, lse = attend(s, out=torch.zeros_like(s["q"]))
    # the definition for some of them, each group's first and last among them
    at = [0, 1, 1023, 1024, 2047, 2048, 3000, 3071, 4095]
    few = dict(q=s["q"][at], new=s["new"][at], own=[s["own"][b] for b in at], prefix=None)
    for i, b in enumerate(at):
        one = dict(q=few["q"][i:i + 1], new=few["new"][i:i + 1], own=[few["own"][i]],
                   prefix=tuple(x[b // 1024][None] for x in s["prefix"]))
        check(one, out[b:b + 1], lse[b:b + 1])
    with pytest.raises(binding.EvictError, match="4096") as e:
        paged.shared_attention(torch.zeros(n + 1, 4, 1, D, dtype=torch.bfloat16, device="cuda"),
                               prefix=tuple(x[:1] for x in s["prefix"]))
    assert e.value.code == binding.EVICT_ELIMIT


def test_bad_tables_and_lengths_are_reported():
    s = make(143, 2, 4, 2, 1, 30, 1, 16, [20, 40])
    for table, lens, new in (((0, 1, 99), None, None), ((0, -5, 1), None, None), (None, [20, 100], None),
                             (None, [-3, 40], None), (None, None, [1, 4]), (None, None, [-1, 1])):
        t, l = s["table"].clone(), s["cache"].lens.clone()
        if table:
            t[1] = torch.tensor(table, dtype=torch.int32)
        if lens:
            l.copy_(torch.tensor(lens))
        c = paged.PagedCache(k_pages=s["kp"], v_pages=s["vp"], table=t, lens=l)
        c.attend(s["q"], prefix=s["prefix"], n_new=torch.tensor(new, dtype=torch.int32).cuda() if new else None)
        with pytest.raises(binding.EvictError, match="index") as e:
            c.sync()
        assert e.value.code == binding.EVICT_EDEVICE
    c = paged.PagedCache(k_pages=s["kp"], v_pages=s["vp"], table=s["table"], lens=s["cache"].lens)
    c.attend(s["q"], prefix=s["prefix"])
    c.sync()


def test_strided_prefix_pages_and_outputs():
    B, hq, h, m, n = 4, 8, 2, 2, 90
    s = make(144, B, hq, h, m, n, 2, 32, [2, 30, 64, 99])
    ref, rl = attend(s)
    big = torch.zeros(2, 2, h, n + 30, D, dtype=torch.bfloat16, device="cuda")      # K and V inside one tensor
    big[:, 0, :, :n], big[:, 1, :, :n] = s["prefix"]
    big[:, :, :, n:] = math.nan
    both = torch.stack([s["kp"], s["vp"]], 1)                                       # pages of K and V side by side
    wide = torch.zeros(B, s["table"].shape[1] + 3, dtype=torch.int32, device="cuda")
    wide[:, :s["table"].shape[1]] = s["table"]
    c = paged.PagedCache(k_pages=both[:, 0], v_pages=both[:, 1], table=wide[:, :s["table"].shape[1]], lens=s["cache"].lens)
    room = torch.full((B, m, hq + 3, D), 9.0, dtype=torch.bfloat16, device="cuda")
    out = room.transpose(1, 2)[:, :hq]
    lse = torch.zeros_like(rl)
    c.attend(s["q"], prefix=(big[:, 0, :, :n], big[:, 1, :, :n]), out=out, lse=lse)
    c.sync()
    assert torch.equal(out, ref) and torch.equal(lse, rl)
    assert bool((room[:, :, hq:] == 9.0).all())


def test_pages_beyond_32_bit_offsets():
    H, page = 8, 256
    n_pages = (1 << 31) // (H * page * D) + 3
    kp = torch.zeros(n_pages, H, page, D, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    k, v, q = randn(145, 2, H, 300, D), randn(146, 2, H, 300, D), randn(147, 2, H, 1, D)
    table = torch.tensor([[n_pages - 1, 0], [1, n_pages - 2]], dtype=torch.int32).cuda()
    for pool, x in ((kp, k), (vp, v)):
        for b in range(2):
            pool[int(table[b, 0])] = x[b, :, :256]
            pool[int(table[b, 1]), :, :44] = x[b, :, 256:]
    c = paged.PagedCache(k_pages=kp, v_pages=vp, table=table, lens=torch.tensor([300, 299], dtype=torch.int32).cuda())
    lse = torch.full((2, H, 1), 7.0, device="cuda")
    out = c.attend(q, lse=lse)
    c.sync()
    check({"q": q, "prefix": None, "new": None, "own": [(k[0], v[0]), (k[1, :, :299], v[1, :, :299])]}, out, lse)


@pytest.mark.parametrize("m", [1, 4, 40])
def test_two_streams_and_two_graphs_at_once(m):
    a = make(150, 8, 8, 2, m, 900, 1, 16, [m + 7 * b for b in range(8)])
    b = make(151, 8, 8, 2, m, 500, 2, 16, [m + 11 * b for b in range(8)])
    want = [attend(s)[0].clone() for s in (a, b)]
    outs = [torch.zeros_like(w) for w in want]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, o, st in zip((a, b), outs, streams):
            with torch.cuda.stream(st):
                s["cache"].attend(s["q"], prefix=s["prefix"], out=o)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    graphs = []
    for s, o, st in zip((a, b), outs, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            s["cache"].attend(s["q"], prefix=s["prefix"], out=o)
        graphs.append(g)
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_two_host_threads():
    import threading
    cases = [make(152 + i, 8, 8, 2, m, 600, 1, 16, [m + 9 * b for b in range(8)]) for i, m in enumerate((1, 40))]
    want = [attend(s)[0].clone() for s in cases]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            for _ in range(50):
                out = cases[i]["cache"].attend(cases[i]["q"], prefix=cases[i]["prefix"])
            st.synchronize()
            if not torch.equal(out, want[i]):
                bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_a_captured_step_follows_the_lengths():
    # one decode step captured once: append, then attend; lens, table and inputs change between replays
    B, hq, h, page, n0 = 3, 8, 2, 16, 60
    base = 1000
    rot = paged.Rotary(base=10000.0)
    freq, axis = inv_freq(128), [0] * 64
    prefix = (randn(160, 1, h, n0, D), randn(161, 1, h, n0, D))
    c = paged.PagedCache(n_pages=32, page_size=page, n_kv_heads=h, batch=B, max_rows=64)
    k, v, q = (torch.zeros(B, x, 1, D, dtype=torch.bfloat16, device="cuda") for x in (h, h, hq))
    qr, out = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((B, hq, 1), 7.0, device="cuda")
    st = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        c.append(k, v, rotary=rot, pos_base=base, q=q, q_out=qr)
        c.attend(qr, prefix=prefix, out=out, lse=lse)
    seen = [([], []) for _ in range(B)]
    for step in range(20):
        ks, vs, qs = randn(170 + step, B, h, 1, D), randn(270 + step, B, h, 1, D), randn(370 + step, B, hq, 1, D)
        for t, x in ((k, ks), (v, vs), (q, qs)):
            t.copy_(x)
        c.grow(1)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        c.sync()
        # the appended keys' own rounding is not at test here: compare with the stored rows
        lens = c.rows()
        own = list(zip(gather(c.k_pages, c.table, lens), gather(c.v_pages, c.table, lens)))
        pos = torch.full((1, B, 1), base + step)
        rk = rotate64(ks, pos, freq, axis)
        for b in range(B):
            assert bool(((own[b][0][:, -1].double().cpu() - rk[b, :, 0]).abs() <= 2.0 ** -8 * rk[b, :, 0].abs() + 1e-5).all())
            assert torch.equal(own[b][1][:, -1], vs[b, :, 0])
        check({"q": qr, "prefix": prefix, "new": None, "own": own}, out, lse)
    del seen


def test_a_served_batch_behind_an_evicted_prompt():
    """A prompt is rotated and absorbed by an evicting cache; three requests behind it bring their
    questions (of different lengths, padded) and then decode, one of them ending early."""
    h, hq, S, budget, B = 2, 6, 400, 128, 3
    rot = paged.Rotary(base=500000.0)
    prompt = binding.EvictCache("knorm", 1, h, budget=budget, max_block=S)
    k0, v0 = randn(180, 1, h, S, D), randn(181, 1, h, S, D)
    kept = prompt.update_and_fetch(paged.rotate(rot, k0, pos_base=0), v0)
    offset = prompt.stats()["offset"]
    assert offset == S and kept[0].shape[2] == budget
    prefix = (kept[0], kept[1])
    own = paged.PagedCache(n_pages=40, page_size=16, n_kv_heads=h, batch=B, max_rows=100)
    all_k = [torch.zeros(h, 0, D, dtype=torch.bfloat16, device="cuda") for _ in range(B)]
    all_v = [x.clone() for x in all_k]

    def step(seed, m, new):
        k, v, q = randn(seed, B, h, m, D), randn(seed + 1, B, h, m, D), randn(seed + 2, B, hq, m, D)
        n = torch.tensor(new, dtype=torch.int32).cuda()
        at = own.rows()
        own.grow(new)
        qr = own.append(k, v, rotary=rot, pos_base=offset, n_new=n, q=q)
        lse = torch.full((B, hq, m), 7.0, device="cuda")
        out = own.attend(qr, prefix=prefix, n_new=n, lse=lse)
        own.sync()
        for b in range(B):
            pos = (offset + at[b] + torch.arange(m))[None].to(torch.int32).cuda()
            kr = paged.rotate(rot, k[b:b + 1].contiguous(), pos=pos)
            all_k[b] = torch.cat([all_k[b], kr[0, :, :new[b]]], 1)
            all_v[b] = torch.cat([all_v[b], v[b, :, :new[b]]], 1)
        check({"q": qr, "prefix": prefix, "new": n, "own": list(zip(all_k, all_v))}, out, lse)

    step(200, 37, [37, 1, 20])
    for i in range(4):
        step(300 + 10 * i, 1, [1, 1, 0 if i > 1 else 1])
    own.release(2)
    all_k[2], all_v[2] = all_k[2][:, :0], all_v[2][:, :0]
    step(400, 5, [2, 1, 5])
    prompt.close()


def test_bad_attention_tensors_are_refused():
    s = make(190, 2, 4, 2, 1, 30, 1, 16, [20, 40])
    q, (pk, pv) = s["q"], s["prefix"]
    for args, kw in (((q.float(),), dict(prefix=(pk, pv))), ((q,), dict(prefix=(pk.float(), pv))),
                     ((q,), dict(prefix=(pk, pv[:, :, :5]))), ((q,), dict(prefix=(pk[..., :64], pv[..., :64]))),
                     ((q,), {}), ((q[:1],), dict(pages=s["cache"])), ((q,), dict(prefix=(pk, pv), scale=0)),
                     ((q,), dict(prefix=(pk, pv), out=q[:1])), ((q,), dict(prefix=(pk, pv), lse=q)),
                     ((q,), dict(prefix=(pk, pv), n_new=torch.zeros(2, device="cuda"))),
                     ((q,), dict(prefix=(pk[:, :1], pv[:, :1]), pages=s["cache"])),
                     ((q,), dict(prefix=(pk[:, :, ::2], pv[:, :, ::2]))), ((q[0],), dict(prefix=(pk, pv)))):
        with pytest.raises(ValueError):
            paged.shared_attention(*args, **kw)
    with pytest.raises(binding.EvictError):
        paged.shared_attention(randn(191, 2, 3, 1, D), prefix=(pk, pv))
    with pytest.raises(binding.EvictError):
        paged.shared_attention(randn(192, 3, 4, 1, D), prefix=(pk.expand(2, -1, -1, -1), pv.expand(2, -1, -1, -1)))


def test_expanded_prefix_equals_the_shared_one():
    s = make(193, 3, 4, 2, 1, 200, 1, 16, [4, 30, 9])
    want, _ = attend(s)
    pk, pv = s["prefix"]
    s["prefix"] = (pk.repeat(3, 1, 1, 1), pv.repeat(3, 1, 1, 1))
    got, lse = attend(s)
    check(s, got, lse)
    # the same rows, cut into other partial results: equal to the outputs' rounding
    assert float((got.double() - want.double()).abs().max()) <= 2.0 ** -7 * float(want.abs().max())
