"""Calls around pages and attention that a user may make and that the ordinary cases leave out."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from kv_cache_token_bf16_gb300 import binding, paged  # noqa: E402
from tests.paged_util import D, gather  # noqa: E402
from tests.test_gpu_attend import _built, attend, check, make, randn  # noqa: E402,F401


def test_a_table_shared_by_all_sequences_has_to_be_repeated():
    kp, vp = randn(40, 6, 2, 16, D), randn(41, 6, 2, 16, D)
    row, lens = torch.tensor([[3, 1]], dtype=torch.int32).cuda(), torch.tensor([20, 31, 5], dtype=torch.int32).cuda()
    for bad in (dict(table=row.expand(3, 2)),
                dict(table=row.repeat(3, 1), k_pages=kp[:1].expand_as(kp), v_pages=vp[:1].expand_as(vp))):
        with pytest.raises(ValueError, match="table|pages"):
            paged.PagedCache(**dict(dict(k_pages=kp, v_pages=vp, lens=lens), **bad))
    # repeated, the sequences read the same pages; a single sequence's row may come with any stride
    s = {"q": randn(42, 3, 4, 1, D), "prefix": None, "new": None}
    table = row.repeat(3, 1)
    s["own"] = list(zip(gather(kp, table, lens.tolist()), gather(vp, table, lens.tolist())))
    s["cache"] = paged.PagedCache(k_pages=kp, v_pages=vp, table=table, lens=lens)
    check(s, *attend(s))
    for b in range(3):
        one = dict(s, q=s["q"][b:b + 1], own=s["own"][b:b + 1])
        one["cache"] = paged.PagedCache(k_pages=kp, v_pages=vp, table=row.as_strided((1, 2), (0, 1)), lens=lens[b:b + 1])
        check(one, *attend(one))


WAIT = 40_000_000                   # clocks: some 20 ms


@pytest.mark.parametrize("default", [True, False], ids=["default", "own"])
def test_kept_rows_attended_to_on_another_stream(default):
    # the cache's stream is late: the attention waits for it; and then the other way round
    B, H, n = 2, 2, 64
    mine, other = torch.cuda.Stream(), torch.cuda.Stream()
    made = torch.cuda.current_stream() if default else mine
    k, v, q = randn(500, B, H, 4 * n, D), randn(501, B, H, 4 * n, D), randn(502, B, 8, 2, D)
    block = [(k[:, :, i * n:(i + 1) * n].contiguous(), v[:, :, i * n:(i + 1) * n].contiguous()) for i in range(4)]
    with torch.cuda.stream(made):
        cache = binding.EvictCache("knorm", B, H, budget=4 * n, max_block=n, n_sink=4, recent=8)
    assert binding.evict_get_stream(cache.handle) == made.cuda_stream
    torch.cuda.synchronize()
    for i in (0, 2):
        lse = [torch.full((B, 8, 2), 7.0, device="cuda") for _ in range(2)]
        torch.cuda.synchronize()
        with torch.cuda.stream(made):
            torch.cuda._sleep(WAIT)
            cache.update_and_fetch(*block[i])
        with torch.cuda.stream(other):
            first = cache.attend(q, lse=lse[0])              # behind the update
            torch.cuda._sleep(WAIT)
            second = cache.attend(q, lse=lse[1])             # before the next one
        with torch.cuda.stream(made):
            cache.update_and_fetch(*block[i + 1])
            # the rows read above are overwritten: the cache starts again
            cache.set_state(k[:, :, 4 * n - 8:].contiguous(), v[:, :, 4 * n - 8:].contiguous(),
                            torch.arange(8, dtype=torch.int32, device="cuda").expand(B, H, 8).contiguous())
            cache.set_state(k[:, :, :(i + 2) * n].contiguous(), v[:, :, :(i + 2) * n].contiguous(),
                            torch.arange((i + 2) * n, dtype=torch.int32, device="cuda").expand(B, H, (i + 2) * n).contiguous())
        torch.cuda.synchronize()
        s = {"q": q, "prefix": (k[:, :, :(i + 1) * n], v[:, :, :(i + 1) * n]), "new": None}
        check(s, first, lse[0])
        check(s, second, lse[1])
    cache.sync()
    cache.close()


def test_kept_rows_attended_to_in_a_captured_graph():
    # captured on another stream than the cache's: a replay reads what is kept then
    k, v, q = randn(510, 1, 2, 128, D), randn(511, 1, 2, 128, D), randn(512, 3, 4, 1, D)
    cache = binding.EvictCache("knorm", 1, 2, budget=128, max_block=128, n_sink=4, recent=8)
    cache.update_and_fetch(k, v)
    out = torch.zeros_like(q)
    lse = torch.full((3, 4, 1), 7.0, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.attend(q, out=out, lse=lse)
    for seed in (513, 514):
        k2 = randn(seed, 1, 2, 128, D)
        cache.set_state(k2, v, torch.arange(128, dtype=torch.int32, device="cuda").expand(1, 2, 128).contiguous())
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        check({"q": q, "prefix": (k2, v), "new": None}, out, lse)
    cache.close()


def test_update_and_attention_on_two_streams_of_one_graph():
    # the cache's stream joins the capture: its update comes before the attention in every replay
    origin, mine = torch.cuda.Stream(), torch.cuda.Stream()
    k, v, q = randn(515, 1, 2, 64, D), randn(516, 1, 2, 64, D), randn(517, 3, 4, 1, D)
    with torch.cuda.stream(mine):
        cache = binding.EvictCache("knorm", 1, 2, budget=64, max_block=64, n_sink=4, recent=8)
    out, lse = torch.zeros_like(q), torch.full((3, 4, 1), 7.0, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=origin):
        mine.wait_stream(origin)
        with torch.cuda.stream(mine):
            torch.cuda._sleep(WAIT // 4)
            cache.update_and_fetch(k, v)
        cache.attend(q, out=out, lse=lse)
        with pytest.raises(ValueError, match="under it"):
            with torch.cuda.stream(torch.cuda.Stream()):
                cache.attend(q, out=out)                # a third stream, outside the capture
    for seed in (518, 519):
        k.copy_(randn(seed, 1, 2, 64, D))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        check({"q": q, "prefix": (k, v), "new": None}, out, lse)
    cache.sync()
    del g
    cache.close()


@pytest.mark.parametrize("hq,m,n_prefix", [(4, 1, 60), (4, 3, 60), (40, 3, 60), (400, 3, 60), (50, 3, 2100)],
                         ids=["few-1", "few", "wide", "joint", "shared"])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_values_that_every_query_sees_may_be_infinite(hq, m, n_prefix, value):
    # in the prefix and in own rows, of the largest weight, small ones and one in between: the result is
    # that infinity, wherever the row lies in its box or tile, and finite columns are untouched
    lens = [m, 90, 40]
    s = make(520, 3, hq, 2, m, n_prefix, 1, 16, lens)
    k, v = s["prefix"]
    k[0, :, 5] = s["q"][0, 0, 0]                           # a large logit for some, a small one for others
    want, _ = attend(s)
    cols = {}
    for i, row in enumerate((0, 5, 17, n_prefix - 1)):
        v[0, :, row, 3 * i] = value
        cols[3 * i] = (0, 1, 2)
    for i, (b, row) in enumerate(((1, 0), (1, 33), (2, 3))):
        s["vp"][int(s["table"][b, row // 16]), :, row % 16, 50 + i] = value
        cols[50 + i] = (b,)
    got, _ = attend(s)
    hit = torch.zeros(3, D, dtype=torch.bool, device="cuda")
    for c, bs in cols.items():
        hit[list(bs), c] = True
    hit = hit[:, None, None].expand_as(got)
    assert bool((got[hit] == value).all() if value == value else got[hit].isnan().all())
    assert torch.equal(got[~hit], want[~hit])


def test_growing_waits_for_nothing():
    # fifty steps of growing and releasing, enqueued behind work that is still running: each takes
    # effect in its place
    B, page, width = 6, 16, 5
    c = paged.PagedCache(n_pages=B * width, page_size=page, n_kv_heads=1, batch=B, max_rows=page * width)
    stream = torch.cuda.Stream()

    def steps():
        want, got = [], []
        for i in range(50):
            for b in range(B):
                if c.rows()[b] > page * (width - 2):
                    c.release(b)
            c.grow([(i * 7 + b * 5) % 20 for b in range(B)])
            want.append((c.rows(), [list(p) for p in c._pages]))
            got.append((c.lens.clone(), c.table.clone()))
        return want, got

    with torch.cuda.stream(stream):
        torch.cuda._sleep(WAIT)
        steps()                                     # torch's pinned memory for so many copies at once
        stream.synchronize()
        torch.cuda._sleep(40 * WAIT)
        want, got = steps()
        assert not stream.query()                   # still asleep: nothing above has waited
    torch.cuda.synchronize()
    for (rows, pages), (lens, table) in zip(want, got):
        assert lens.tolist() == rows
        for b in range(B):
            assert table[b, :len(pages[b])].tolist() == pages[b]
            assert len(pages[b]) == -(-rows[b] // page)
        used = [p for q in pages for p in q]
        assert len(used) == len(set(used))


def test_growing_cannot_be_captured():
    c = paged.PagedCache(n_pages=4, page_size=16, n_kv_heads=1, batch=2, max_rows=32)
    c.grow([3, 17])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    x = torch.zeros(4, device="cuda")
    with torch.cuda.graph(g):
        x += 1
        for call in (lambda: c.grow(1), lambda: c.release(1)):
            with pytest.raises(ValueError, match="captured"):
                call()
    assert c.rows() == [3, 17]
    g.replay()
    c.grow(1)
    assert c.lens.tolist() == c.rows() == [4, 18]


def workspace(batch, m, hq, h, n_prefix=0, groups=1, rows=0):
    a = binding.EvictAttention(batch=batch, m=m, n_q_heads=hq, n_kv_heads=h, n_prefix=n_prefix, prefix_batch=groups)
    if rows:
        g = binding.EvictPages(page_size=16, table_width=-(-rows // 16))
        a.pages = ctypes.pointer(g)
    return binding.evict_shared_attention_workspace(a)


def test_workspace_is_no_more_than_partial_results_need():
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    row = (D + 2) * 4                               # a row of a partial result
    # long blocks: at most two parts of 256 rows for each SM, however many tokens there are
    for args in ((8, 8192, 32, 8, 0, 1, 8192), (128, 512, 32, 8, 1024, 2, 600), (1, 8192, 32, 8), (1, 300, 8, 8, 0, 1, 300)):
        assert workspace(*args) <= 2 * sms * 256 * row + (1 << 20), args
    # units of 36 rows: two groups' rows of each, not a whole tile
    assert workspace(4096, 9, 32, 8, 4096, 4096, 64) <= 2 * (4096 * 8 + sms) * 2 * 36 * row + (1 << 20)
    # one token of each of 4,096 sequences: four rows of each of their 8 heads
    assert workspace(4096, 1, 32, 8, 0, 1, 4096) <= (4096 * 8 + 12 * sms) * 4 * row + (1 << 20)


@pytest.mark.parametrize("hq,h,m,n_prefix,groups", [(36, 4, 4, 2300, 2), (36, 4, 4, 30, 8), (20, 4, 7, 2500, 4), (8, 8, 30, 2300, 1),
                                                    (8, 2, 32, 2600, 8), (8, 2, 33, 2600, 8), (6, 2, 1, 40, 1), (6, 2, 5, 0, 1)])
@pytest.mark.parametrize("ragged", [False, True])
def test_partial_results_of_any_number_of_rows(hq, h, m, n_prefix, groups, ragged):
    B = 8
    lens = [m + (b * 211) % 900 for b in range(B)]
    new = [m if b % 3 == 0 else (b * 5) % (m + 1) for b in range(B)] if ragged else None
    s = make(530, B, hq, h, m, n_prefix, groups, 32, lens, new)
    check(s, *attend(s, out=torch.zeros_like(s["q"])))


@pytest.mark.parametrize("transpose", [False, True])
def test_fp32_angles_keep_their_bits_all_around(transpose):
    """Rows (1, 0) give cosine and sine themselves. The angle's fraction of a turn is cut to 2^-32 (2 pi
    2^-32 < 0.03 U32 radians) and, less whole quarters, rounded to fp32: at most 2^-27 half turns (pi
    2^-27 < 0.4 U32). sincospif is within one step of its value, 2 U32 of it at most. The products
    with 1 and 0 are exact."""
    u = 2.0 ** -24
    n = 4096
    rot = paged.Rotary(2, inv_freq=[1.0])
    x = torch.zeros(1, 1, n, D, device="cuda")
    x[..., 0] = 1
    g = torch.Generator().manual_seed(540)
    for hi in (1 << 12, 1 << 30):
        pos = torch.randint(-hi, hi, (1, n), generator=g, dtype=torch.int64).to(torch.int32)
        got = paged.rotate(rot, x, pos=pos.cuda(), transpose=transpose)[0, 0].double().cpu()
        a = pos[0].double()
        c, s = a.cos(), (-a if transpose else a).sin()
        for v, ref, slope in ((got[:, 0], c, s), (got[:, 1], s, c)):
            err = (v - ref).abs()
            assert bool((err <= 0.43 * u * slope.abs() + 2 * u * ref.abs() + 1e-13).all()), float(err.max() / u)


@pytest.mark.parametrize("own", [True, False])
@pytest.mark.parametrize("hq,m", [(4, 1), (40, 1), (300, 2)], ids=["few", "wide", "joint"])
def test_prefixes_and_heads_expanded_over_an_axis(hq, m, own):
    # one prefix for every sequence, one head for every KV head, as torch's expand gives them
    B, h, n = 3, 2, 170
    s = make(560, B, hq, h, m, n, B, 16, [m + 3, m, m + 40] if own else None)
    k, v = s["prefix"]
    for over_b, over_h in ((True, False), (False, True), (True, True)):
        kk, vv = ((x[:1 if over_b else B, :1 if over_h else h]).expand(B, h, -1, -1) for x in (k, v))
        s["prefix"] = kk, vv
        if over_h and own:
            with pytest.raises(ValueError, match="repeat"):
                attend(s)
            continue
        got, lse = attend(s)
        s["prefix"] = kk.contiguous(), vv.contiguous()
        check(s, got, lse)
        if over_b and not over_h:                   # the very work of one prefix that is given as such
            s["prefix"] = k[:1], v[:1]
            want, wl = attend(s)
            assert torch.equal(got, want) and torch.equal(lse, wl)
