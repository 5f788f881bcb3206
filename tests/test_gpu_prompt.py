"""Attention of whole prompts and the weights of their keys, against plain 64-bit forms."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from kv_cache_token_bf16_gb300 import binding, paged, prompt  # noqa: E402
from tests.paged_util import D  # noqa: E402
from tests.prompt_util import SCALE, check_prompt, check_weights, spans_of, weights64  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built(lib):
    pass


def rows(seed, batch, heads, m, layout="token", std=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    if layout == "token":
        return torch.randn(batch, m, heads, D, device="cuda", generator=g).mul_(std).bfloat16().transpose(1, 2)
    if layout == "wide":                             # rows apart from each other, heads among other tensors'
        x = torch.randn(batch, m + 1, heads + 3, 2 * D, device="cuda", generator=g).mul_(std).bfloat16()
        return x[:, :m, 1:heads + 1, D:].transpose(1, 2)
    return torch.randn(batch, heads, m, D, device="cuda", generator=g).mul_(std).bfloat16()


def starts_of(lens, lead=0):
    got = [lead]
    for l in lens:
        got.append(got[-1] + l)
    return got


def run(q, k, v, starts=None, last=0, scale=None, layout="token"):
    """Both calls, checked."""
    B, hq, m, _ = q.shape
    pk = prompt.Packing(torch.tensor(starts, dtype=torch.int32).cuda()) if starts is not None else None
    out = torch.full((B, m, hq, D), 5.0, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    if layout == "head":
        out = out.contiguous()
    lse = torch.full((B, hq, m), 7.0, device="cuda")
    assert prompt.attention(q, k, v, pk, scale=scale, out=out, lse=lse) is out
    w = torch.full((B, k.shape[1], m), 3.0, device="cuda")
    assert prompt.weights(q, k, lse, pk, last=last, scale=scale, out=w) is w
    torch.cuda.synchronize()
    if pk is not None:
        pk.sync()
    spans = spans_of(starts, B, m)
    at = SCALE if scale is None else scale
    check_prompt(q, k, v, spans, out, lse, at, 5.0, 7.0)
    check_weights(w, *weights64(q, k, lse, spans, last, at), 3.0)
    return out, lse, w


@pytest.mark.parametrize("hq,hkv,lens,last", [
    (1, 1, [1], 0), (8, 2, [1, 1, 1], 1), (8, 8, [5], 3), (3, 1, [33, 64], 0), (12, 4, [1, 45, 20, 7], 0),
    (4, 4, [127, 128, 129], 0), (4, 4, [255, 256, 257], 5), (32, 8, [63, 64, 65, 31, 32, 33], 16),
    (28, 4, [17, 18, 19, 36, 37, 300], 0), (40, 8, [25, 50, 51, 401], 64), (24, 1, [200, 5], 7),
    (128, 1, [3, 130], 0), (100, 1, [140], 0), (65, 1, [70], 0),
    (8, 2, [300, 0, 1, 77, 513], 0), (8, 2, [0, 0, 40, 0], 32), (16, 2, [500, 524], 513),
    (8, 2, [1024], 0), (8, 2, [1025], 0), (8, 2, [900, 200], 1), (4, 4, [2049, 3], 0), (28, 4, [1500, 700], 64),
    (3, 1, [2048, 3, 1100], 0), (32, 8, [1] * 300, 0), (8, 8, [7] * 200, 4), (2, 2, [6000], 0), (2, 1, [4097, 4096], 4000)])
def test_packed_prompts(hq, hkv, lens, last):
    starts = starts_of(lens, 3)
    m = starts[-1] + 11
    q, k, v = rows(1, 1, hq, m, std=1.5), rows(2, 1, hkv, m), rows(3, 1, hkv, m)
    run(q, k, v, starts, last)


@pytest.mark.parametrize("layout", ["token", "head", "wide"])
@pytest.mark.parametrize("batch,m,hq,hkv,last,scale", [
    (1, 1, 4, 4, 0, None), (3, 100, 8, 2, 0, 0.11), (2, 257, 3, 1, 1, None), (2, 1100, 16, 2, 0, -0.07), (3, 1300, 10, 2, 100, None)])
def test_batches(layout, batch, m, hq, hkv, last, scale):
    q, k, v = rows(4, batch, hq, m, layout, 1.5), rows(5, batch, hkv, m, layout), rows(6, batch, hkv, m, layout)
    run(q, k, v, None, last, scale, layout)


def test_no_tokens():
    for m, starts in ((0, None), (0, [0]), (0, [0, 0]), (6, [2]), (6, [4, 4, 4])):
        q, k, v = rows(7, 1, 4, m), rows(8, 1, 2, m), rows(9, 1, 2, m)
        run(q, k, v, starts)
    assert prompt.attention(rows(7, 0, 4, 5), rows(8, 0, 2, 5), rows(9, 0, 2, 5)).shape == (0, 4, 5, D)
    # new outputs: zeros where there is no sequence
    pk = prompt.Packing(torch.tensor([1, 3], dtype=torch.int32).cuda())
    q, k, v = rows(7, 1, 4, 6), rows(8, 1, 2, 6), rows(9, 1, 2, 6)
    lse = torch.zeros(1, 4, 6, device="cuda")
    out = prompt.attention(q, k, v, pk, lse=lse)
    w = prompt.weights(q, k, lse, pk)
    assert not out[:, :, [0, 3, 4, 5]].any() and out[:, :, 1:3].any(3).all()
    assert not w[:, :, [0, 3, 4, 5]].any() and (w[:, :, 1:3] > 0).all()


@pytest.mark.parametrize("rising", [True, False])
def test_logits_that_rise_and_fall(rising):
    # the reference of the exponents has to follow: each key's logit tops the last ones' by far, in a step and over steps
    m, hq, hkv = 1200, 4, 2
    q, k, v = rows(10, 1, hq, m, std=0.05), rows(11, 1, hkv, m, std=0.3), rows(12, 1, hkv, m)
    size = torch.linspace(0.0, 60.0, m, device="cuda")
    if not rising:
        size = size.flip(0)
    q[..., 0] = 8.0
    k[..., 0] = size.bfloat16()
    run(q, k, v, [0, 1100, 1200])
    k[..., 0] = (size * torch.where(torch.arange(m, device="cuda") % 97 == 5, 2.0, 0.1)).bfloat16()   # a few tower
    run(q, k, v, [0, 1100, 1200])


@pytest.mark.parametrize("hq,hkv", [(4, 4), (8, 2)])
def test_what_a_query_does_not_see_may_hold_anything(hq, hkv):
    lens = [40, 300, 130, 1, 600, 90]
    starts = starts_of(lens, 5)
    m = starts[-1] + 9
    q, k, v = rows(13, 1, hq, m, std=1.5), rows(14, 1, hkv, m), rows(15, 1, hkv, m)
    spans = spans_of(starts, 1, m)
    clean = [x.clone() for x in (q, k, v)]
    was = run(q, k, v, starts)
    # tokens of no sequence, and a whole sequence between others
    for x in (q, k, v):
        for a, e, bad in ((0, 5, math.nan), (starts[-1], m, math.inf), (starts[2], starts[3], -math.inf), (starts[2] + 7, starts[2] + 8, math.nan)):
            x[:, :, a:e] = bad
    pk = prompt.Packing(torch.tensor(starts, dtype=torch.int32).cuda())
    lse = torch.full((1, hq, m), 7.0, device="cuda")
    got = prompt.attention(q, k, v, pk, lse=lse)
    w = prompt.weights(q, k, lse, pk)
    pk.sync()
    for i, (_, a, l) in enumerate(spans):
        if i == 2:
            continue
        for x, y in zip((got, lse, w), was):
            assert torch.equal(x[:, :, a:a + l], y[:, :, a:a + l]), i
    # rows of V that later queries of the same tile see, and earlier ones do not
    q, k, v = clean
    for row, bad in ((starts[1] + 150, math.inf), (starts[1] + 151, math.nan), (starts[4] + 599, -math.inf), (starts[4] + 1, math.nan),
                     (starts[3], math.inf)):
        v[:, 0, row, 7] = bad
    got = prompt.attention(q, k, v, pk, lse=lse)
    pk.sync()
    check_prompt(q, k, v, spans, got, lse)


def test_infinite_rows_in_long_prompts_and_parts_of_units():
    m, hq, hkv = 3000, 4, 2
    q, k, v = rows(16, 1, hq, m, std=0.3), rows(17, 1, hkv, m, std=0.3), rows(18, 1, hkv, m)
    for row in (0, 100, 127, 128, 1000, 1500, 2047, 2048, 2500, 2998, 2999):
        v[:, row % 2, row, row % 128] = math.inf if row % 3 else -math.inf
    lse = torch.zeros(1, hq, m, device="cuda")
    got = prompt.attention(q, k, v, lse=lse)
    torch.cuda.synchronize()
    check_prompt(q, k, v, [(0, 0, m)], got, lse)


def test_keys_and_queries_of_infinities_and_nan():
    # a key that is NaN reaches the queries that see it; so does one whose logit is +infinity; one of -infinity has no weight
    m = 200
    q, k, v = rows(19, 1, 2, m).abs(), rows(20, 1, 2, m), rows(21, 1, 2, m)
    k[0, 0, 50] = math.nan
    k[0, 1, 60, 3] = -math.inf
    lse = torch.zeros(1, 2, m, device="cuda")
    got = prompt.attention(q, k, v, lse=lse)
    assert torch.isnan(got[0, 0, 50:]).all() and torch.isfinite(got[0, 0, :50]).all()
    assert torch.isnan(lse[0, 0, 50:]).all() and torch.isfinite(lse[0, 0, :50]).all()
    check_prompt(q[:, 1:], k[:, 1:], v[:, 1:], [(0, 0, m)], got[:, 1:], lse[:, 1:])
    q[0, 1, 100] = math.nan
    got = prompt.attention(q, k, v, lse=lse)
    assert torch.isnan(got[0, 1, 100]).all() and torch.isfinite(got[0, 1, [99, 101]]).all()
    w = prompt.weights(q, k, lse)
    assert torch.isnan(w[0, 1, :101]).sum() == 101 and torch.isfinite(w[0, 1, 101:]).all()
    # a first key of -infinity: the query that sees it alone has no weights that add up
    k[0, 1, 0, 3] = -math.inf
    got = prompt.attention(q, k, v, lse=lse)
    assert lse[0, 1, 0] == -math.inf and torch.isfinite(lse[0, 1, 1:100]).all()
    w = prompt.weights(q, k, lse)
    assert torch.isnan(w[0, 1, 0])                  # of query 100 alone: query 0 has no weights


def test_weights_of_queries_that_saw_nothing():
    m = 300
    q, k = rows(22, 1, 4, m), rows(23, 1, 2, m)
    lse = torch.randn(1, 4, m, device="cuda", generator=torch.Generator("cuda").manual_seed(24)) + 5
    lse[0, :, 17] = lse[0, 2, 200:] = -math.inf
    lse[0, 1, 40] = math.inf
    check_weights(prompt.weights(q, k, lse), *weights64(q, k, lse, [(0, 0, m)]))


@pytest.mark.parametrize("lens", [[300, 1, 77], [1700, 900]])
def test_the_same_bits_every_time(lens):
    starts = starts_of(lens)
    m = starts[-1]
    q, k, v = rows(25, 1, 8, m, std=1.5), rows(26, 1, 2, m), rows(27, 1, 2, m)
    pk = prompt.Packing(torch.tensor(starts, dtype=torch.int32).cuda())
    got = []
    for _ in range(4):
        lse = torch.zeros(1, 8, m, device="cuda")
        out = prompt.attention(q, k, v, pk, lse=lse)
        got.append((out, lse, prompt.weights(q, k, lse, pk)))
    pk.sync()
    for x in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(x, got[0]))


@pytest.mark.parametrize("starts", [[0, 50, 40, 100], [-1, 50, 100], [0, 50, 2001], [5, 3]])
@pytest.mark.parametrize("m", [900, 2000])
def test_starts_that_fall_or_leave_the_tensors_write_nothing(starts, m):
    if m == 900 and 2001 in starts:
        starts = [0, 50, 901]
    q, k, v = rows(28, 1, 4, m), rows(29, 1, 2, m), rows(30, 1, 2, m)
    pk = prompt.Packing(torch.tensor(starts, dtype=torch.int32).cuda())
    out, lse, w = torch.full_like(q, 5.0), torch.full((1, 4, m), 7.0, device="cuda"), torch.full((1, 2, m), 3.0, device="cuda")
    for call in (lambda: prompt.attention(q, k, v, pk, out=out, lse=lse), lambda: prompt.weights(q, k, lse, pk, out=w)):
        call()
        with pytest.raises(binding.EvictError, match="index") as e:
            pk.sync()
        assert e.value.code == binding.EVICT_EDEVICE
        pk.sync()
    assert (out == 5).all() and (lse == 7).all() and (w == 3).all()
    pk.starts.copy_(torch.linspace(0, m, len(starts)).int())     # put right in place
    prompt.attention(q, k, v, pk, out=out, lse=lse)
    pk.sync()
    check_prompt(q, k, v, spans_of(pk.starts.tolist(), 1, m), out, lse)


def test_captured_calls_follow_the_starts():
    m = 1400
    q, k, v = rows(31, 1, 8, m), rows(32, 1, 2, m), rows(33, 1, 2, m)
    pk = prompt.Packing(torch.tensor([0, 10, 1400], dtype=torch.int32).cuda())
    out, lse, w = torch.zeros_like(q), torch.zeros(1, 8, m, device="cuda"), torch.zeros(1, 2, m, device="cuda")

    def both():
        prompt.attention(q, k, v, pk, out=out, lse=lse)
        prompt.weights(q, k, lse, pk, last=40, out=w)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both()
    torch.cuda.current_stream().wait_stream(s)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    for g in (g1, g2):
        with torch.cuda.graph(g):
            both()
    for g, starts in ((g1, [0, 10, 1400]), (g2, [3, 700, 701]), (g1, [0, 0, 1399]), (g2, [100, 200, 1300])):
        pk.starts.copy_(torch.tensor(starts, dtype=torch.int32))
        q.copy_(rows(40 + starts[1], 1, 8, m))
        out.fill_(5.0)
        lse.fill_(7.0)
        w.fill_(3.0)
        g.replay()
        pk.sync()
        spans = spans_of(starts, 1, m)
        check_prompt(q, k, v, spans, out, lse, out_was=5.0, lse_was=7.0)
        check_weights(w, *weights64(q, k, lse, spans, 40), 3.0)


def test_two_streams_at_once():
    streams = [torch.cuda.Stream() for _ in range(2)]
    args = []
    for i in range(2):
        m = 1500 + 200 * i
        args.append((rows(50 + i, 1, 8, m), rows(60 + i, 1, 2, m), rows(70 + i, 1, 2, m), torch.zeros(1, 8, m, device="cuda")))
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(5):
        for i, s in enumerate(streams):
            q, k, v, lse = args[i]
            with torch.cuda.stream(s):
                out = prompt.attention(q, k, v, lse=lse)
                got[i] = (out, prompt.weights(q, k, lse))
    torch.cuda.synchronize()
    for (q, k, v, lse), (out, w) in zip(args, got):
        spans = [(0, 0, q.shape[2])]
        check_prompt(q, k, v, spans, out, lse)
        check_weights(w, *weights64(q, k, lse, spans))


# steps of 64, 32 or 16 tokens by several heads, whose number does not divide the group's; the window longer than the
# sequence, as long, and shorter; one key tile and two
@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (7, 1), (24, 1), (9, 1), (16, 2)])
@pytest.mark.parametrize("last", [1, 16, 17, 32, 33, 64, 65])
def test_windows_of_few_tokens(hq, hkv, last):
    q, k = rows(80, 1, hq, 1700, std=1.5), rows(81, 1, hkv, 1700)
    lse = torch.randn(1, hq, 1700, device="cuda", generator=torch.Generator("cuda").manual_seed(82)) + 4.0
    for starts in ([0, 1400, 1416, 1417, 1480, 1700], [3, 130, 300]):
        pk = prompt.Packing(torch.tensor(starts, dtype=torch.int32).cuda())
        m = starts[-1] + 4 if starts[0] else 1700
        args = q[:, :, :m], k[:, :, :m], lse[:, :, :m].contiguous()
        w = torch.full((1, hkv, m), 3.0, device="cuda")
        prompt.weights(*args, pk, last=last, out=w)
        pk.sync()
        check_weights(w, *weights64(*args, spans_of(starts, 1, m), last), 3.0)


# more sequences than the schedule's tables in shared memory hold, most of them empty
@pytest.mark.parametrize("m", [1000, 2500])
@pytest.mark.parametrize("n", [4095, 4096, 4097, 20000])
def test_very_many_sequences(m, n):
    lens = [0] * n
    g = torch.Generator().manual_seed(n)
    for i in torch.randint(0, n, (m // 9,), generator=g).tolist():
        lens[i] = 1 + i % 7
    lens[n // 2] = 300
    starts = starts_of(lens)
    assert starts[-1] <= m
    q, k, v = rows(83, 1, 8, m, std=1.5), rows(84, 1, 2, m), rows(85, 1, 2, m)
    run(q, k, v, starts)


def test_calls_between_others_of_torchs_allocator():
    # workspaces go back to the allocator when the call returns: what takes their place comes behind the work
    q, k, v = rows(86, 1, 8, 3000), rows(87, 1, 2, 3000), rows(88, 1, 2, 3000)
    outs = []
    for i in range(6):
        lse = torch.empty(1, 8, 3000, device="cuda")
        out = prompt.attention(q, k, v, lse=lse)
        junk = [torch.full((1 << s,), float("nan"), device="cuda") for s in range(10, 26, 3)]
        w = prompt.weights(q, k, lse)
        del junk
        outs.append((out, lse, w))
    for got in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got, outs[0]))
    spans = [(0, 0, 3000)]
    check_prompt(q, k, v, spans, outs[0][0], outs[0][1])
    check_weights(outs[0][2], *weights64(q, k, outs[0][1], spans))


# units that go uncut beyond 1024 rows: three or more for every SM, dealt out the longest first
@pytest.mark.parametrize("lens", [[3700], [700, 1, 0, 1300, 64, 513, 1022, 400], [129] * 40, [0, 0, 4100, 3, 0]])
def test_uncut_units_of_long_planes(lens):
    starts = starts_of(lens, 2)
    m = starts[-1] + 5
    q, k, v = rows(90, 1, 32, m, std=1.5), rows(91, 1, 8, m), rows(92, 1, 8, m)
    v[0, :, starts[-1] - 3, 17], v[0, 2, 700, 5] = math.inf, -math.inf
    run(q, k, v, starts)


def test_uncut_units_of_windows_take_the_workspace_of_any_window():
    B, m, h = 6, 4100, 8
    q, k = rows(93, B, h, m, std=1.5), rows(94, B, h, m)
    lse = torch.randn(B, h, m, device="cuda", generator=torch.Generator("cuda").manual_seed(95)) + 6.0
    starts = torch.tensor([0, 1500, 4100], dtype=torch.int32).cuda()
    for last in (0, 64, 300, 0, 1):
        w = prompt.weights(q, k, lse, last=last)
        check_weights(w, *weights64(q, k, lse, spans_of(None, B, m), last))
        one = prompt.weights(q[:1], k[:1], lse[:1], prompt.Packing(starts), last=last)
        check_weights(one, *weights64(q[:1], k[:1], lse[:1], spans_of([0, 1500, 4100], 1, m), last))
    sizes = set()
    for last in (0, 1, 64, 300, 5000):
        fields = (B, m, *paged._rows(q, "q", 0, q.dtype, B, m), *paged._rows(k, "k", 0, k.dtype, B, m), *prompt._NO_ROWS * 2,
                  lse.data_ptr(), 0, 0, 0, last, 0.0, 0, 0, 0, 0)
        sizes.add(binding.evict_prompt_weights_workspace(binding.EvictPrompt.from_buffer_copy(prompt._PROMPT.pack(*fields))))
    assert len(sizes) == 1


def test_units_that_ctas_take_as_they_come():
    # which CTA takes which unit changes from run to run: no result does, nor those of a graph or of two calls at once
    lens = [700, 1, 0, 1300, 64, 513, 1022, 400, 900, 77]
    starts = starts_of(lens)
    m = starts[-1]
    pk = prompt.Packing(torch.tensor(starts, dtype=torch.int32).cuda())
    args = [(rows(96 + i, 1, 32, m, std=1.5), rows(98 + i, 1, 8, m), rows(100 + i, 1, 8, m)) for i in range(2)]

    def call(i, out=None, lse=None, w=None):
        q, k, v = args[i]
        lse = torch.empty(1, 32, m, device="cuda") if lse is None else lse
        out = prompt.attention(q, k, v, pk, out=out, lse=lse)
        return out, lse, prompt.weights(q, k, lse, pk, out=w)

    ref = [call(i) for i in range(2)]
    for i, (q, k, v) in enumerate(args):
        spans = spans_of(starts, 1, m)
        check_prompt(q, k, v, spans, *ref[i][:2])
        check_weights(ref[i][2], *weights64(q, k, ref[i][1], spans))
    same = lambda a, b: all(torch.equal(x, y) for x, y in zip(a, b))  # noqa: E731
    for _ in range(4):
        assert same(call(0), ref[0])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append((i, call(i)))
    torch.cuda.synchronize()
    assert all(same(x, ref[i]) for i, x in got)
    del got
    held = [torch.zeros_like(x) for x in ref[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(0, *held)
    for _ in range(3):
        for x in held:
            x.zero_()
        graph.replay()
        assert same(held, ref[0])
    pk.sync()


# weights' units that go uncut, in the order of the blocks' numbers (up to 256 sequences) and in the sequences'
@pytest.mark.parametrize("lens", [[700, 1, 0, 1300, 64, 513, 1022, 400, 900, 77], [30, 0, 257] * 100, [1500, 1400, 0, 0, 1300, 800]])
def test_weights_units_that_ctas_take_as_they_come(lens):
    starts = starts_of(lens, 1)
    m = starts[-1] + 3
    pk = prompt.Packing(torch.tensor(starts, dtype=torch.int32).cuda())
    q, k = rows(110, 1, 16, m, std=1.5), rows(111, 1, 16, m)
    lse = torch.randn(1, 16, m, device="cuda", generator=torch.Generator("cuda").manual_seed(112)) + 5.0
    w = torch.full((1, 16, m), 3.0, device="cuda")
    prompt.weights(q, k, lse, pk, out=w)
    pk.sync()
    check_weights(w, *weights64(q, k, lse, spans_of(starts, 1, m)), 3.0)
    for _ in range(4):
        again = torch.full_like(w, 3.0)
        prompt.weights(q, k, lse, pk, out=again)
        assert torch.equal(again, w)


def test_offsets_past_32_bits():
    # 2.5e9 elements of q and out; the last sequences against calls of their own
    lens = [1000] * 610 + [333, 1, 777]
    starts = starts_of(lens)
    m = starts[-1]
    assert m * 32 * D > 2 ** 31
    g = torch.Generator("cuda").manual_seed(120)
    q = torch.randn(1, m, 32, D, device="cuda", generator=g, dtype=torch.bfloat16).transpose(1, 2)
    k, v = (torch.randn(1, m, 8, D, device="cuda", generator=g, dtype=torch.bfloat16).transpose(1, 2) for _ in range(2))
    pk = prompt.Packing(torch.tensor(starts, dtype=torch.int32).cuda())
    lse = torch.empty(1, 32, m, device="cuda")
    out = prompt.attention(q, k, v, pk, lse=lse)
    w = prompt.weights(q, k, lse, pk)
    pk.sync()
    for i in (0, 500, 609, 610, 611, 612):
        a, b = starts[i], starts[i + 1]
        x = [t[:, :, a:b].contiguous() for t in (q, k, v, out, lse)]
        check_prompt(*x[:3], [(0, 0, b - a)], *x[3:])
        check_weights(w[:, :, a:b], *weights64(x[0], x[1], x[4], [(0, 0, b - a)]))
