"""Caches that evict by accumulated attention weight: starts of scores, weights of steps, and a serving run of
all of it, against plain 64-bit forms."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from kv_cache_token_bf16_gb300 import binding, paged, prompt  # noqa: E402
from tests.gpu_util import to_bits  # noqa: E402
from tests.paged_util import D, U32  # noqa: E402
from tests.prompt_util import SCALE, check_weights, kept  # noqa: E402
from tests.test_gpu_prompt import rows  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built(lib):
    pass


def block(seed, B, H, m):
    return rows(seed, B, H, m, "head"), rows(seed + 1, B, H, m, "head")


class Plain:
    """The same cache in torch."""

    def __init__(self, B, H, budget, n_sink, recent):
        self.cut = dict(budget=budget, n_sink=n_sink, recent=recent)
        self.k = self.v = torch.zeros(B, H, 0, D, dtype=torch.bfloat16, device="cuda")
        self.pos, self.score = torch.zeros(B, H, 0, dtype=torch.int32, device="cuda"), torch.zeros(B, H, 0, device="cuda")
        self.offset = 0

    def update(self, k, v, pos=None, score=None):
        B, H, m, _ = k.shape
        if pos is None:
            pos = (self.offset + torch.arange(m, device="cuda")).int().expand(B, m)
        self.offset += m
        score = torch.zeros(B, H, m, device="cuda") if score is None else score
        cat = [torch.cat([a, b], dim=2) for a, b in ((self.k, k), (self.v, v), (self.pos, pos[:, None].expand(B, H, m)),
                                                     (self.score, score))]
        idx = kept(cat[3], **self.cut).cuda()
        wide = idx[..., None].expand(-1, -1, -1, D)
        self.k, self.v = cat[0].gather(2, wide), cat[1].gather(2, wide)
        self.pos, self.score = cat[2].gather(2, idx), cat[3].gather(2, idx)

    def check(self, view, what=""):
        for got, ref, name in zip(view, (self.k, self.v, self.pos, self.score), ("k", "v", "pos", "score")):
            assert to_bits(got).tobytes() == to_bits(ref).tobytes(), f"{what}: {name} differs"


@pytest.mark.parametrize("B,H,budget,n_sink,recent,blocks", [
    (1, 1, 8, 0, 0, [3, 4, 1, 1, 1, 5, 1]), (2, 3, 64, 4, 8, [1, 62, 1, 1, 1, 40, 2]), (2, 2, 100, 2, 33, [300, 1, 1, 7, 64, 65]),
    (1, 8, 512, 4, 128, [2048, 1, 1, 1, 500]), (4, 2, 1000, 4, 64, [999, 1, 1, 3001]), (1, 2, 16, 3, 12, [16, 1, 1, 1])])
@pytest.mark.parametrize("ties", [False, True])
def test_eviction_by_given_scores(B, H, budget, n_sink, recent, blocks, ties):
    g = torch.Generator("cuda").manual_seed(budget)
    cache = binding.EvictCache("attention", B, H, budget=budget, n_sink=n_sink, recent=recent, max_block=max(blocks))
    ref = Plain(B, H, budget, n_sink, recent)
    for i, m in enumerate(blocks):
        k, v = block(100 * i, B, H, m)
        score = torch.randn(B, H, m, device="cuda", generator=g)
        score = torch.randint(0, 3, (B, H, m), device="cuda", generator=g).float() if ties else score
        if i == 2:
            score = None                            # starts from 0
        pos = (5 * i + torch.arange(m, device="cuda").int() * 2).expand(B, m).contiguous() if i % 3 == 1 else None
        view = cache.update_and_fetch(k, v, pos=pos, score=score)
        ref.update(k, v, pos, score)
        cache.sync()
        ref.check(view, i)
        assert cache.stats()["offset"] == ref.offset
    cache.close()


def test_scores_of_nan_and_infinities():
    B, H, n = 1, 2, 40
    score = torch.randn(B, H, n, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    score[0, 0, [3, 9, 20]] = torch.tensor([math.nan, math.inf, -math.inf], device="cuda")
    score[0, 1, 5:30] = -math.inf
    cache, ref = binding.EvictCache("attention", B, H, budget=24, n_sink=2, recent=3, max_block=n), Plain(B, H, 24, 2, 3)
    k, v = block(7, B, H, n)
    view = cache.update_and_fetch(k, v, score=score)
    ref.update(k, v, score=score)
    cache.sync()
    for got, want in zip(view[:3], (ref.k, ref.v, ref.pos)):
        assert torch.equal(got, want)


def test_update_from_the_host_starts_from_zero():
    k, v = block(9, 1, 2, 30)
    cache, ref = binding.EvictCache("attention", 1, 2, budget=20, n_sink=2, recent=4, max_block=30), Plain(1, 2, 20, 2, 4)
    kh, vh = k.cpu().pin_memory(), v.cpu().pin_memory()
    view = binding.evict_update_and_fetch_host(cache.handle, kh.data_ptr(), vh.data_ptr(), None, 30)
    cache.sync()
    ref.update(k, v)
    ref.check(binding.view_tensors(view, 1, 2, "bf16"))


def test_refusals():
    k, v = block(11, 1, 2, 8)
    q, lse = rows(12, 1, 4, 1), torch.zeros(1, 4, 1, device="cuda")
    with pytest.raises(binding.EvictError, match="bf16"):
        binding.EvictCache("attention", 1, 2, budget=16, dtype="fp32")
    with pytest.raises(binding.EvictError, match="per-token"):
        binding.EvictCache("attention", 1, 2, budget=16, per_token=True)
    other = binding.EvictCache("h2o", 1, 2, budget=16, max_block=8)
    with pytest.raises(binding.EvictError, match="makes its rows' scores"):
        other.update_and_fetch(k, v, score=torch.zeros(1, 2, 8, device="cuda"))
    other.update_and_fetch(k, v)
    with pytest.raises(binding.EvictError, match="accumulated attention"):
        other.weigh(q, lse)
    with pytest.raises(ValueError, match="accumulates"):
        other.attend(q, weigh=True)
    cache = binding.EvictCache("attention", 1, 2, budget=16, max_block=8)
    for bad in (torch.zeros(1, 2, 7, device="cuda"), torch.zeros(1, 2, 8), torch.zeros(1, 2, 8, device="cuda").double(),
                torch.zeros(1, 8, 2, device="cuda").transpose(1, 2)):
        with pytest.raises(ValueError, match="score"):
            cache.update_and_fetch(k, v, score=bad)
    cache.update_and_fetch(k, v)
    with pytest.raises(binding.EvictError, match="multiple"):
        cache.weigh(rows(13, 1, 3, 1), torch.zeros(1, 3, 1, device="cuda"))
    with pytest.raises(ValueError, match="lse"):
        cache.weigh(q, torch.zeros(1, 4, 2, device="cuda"))
    with pytest.raises(ValueError, match="scale"):
        cache.weigh(q, lse, scale=0)
    with pytest.raises(binding.EvictError, match="grouped"):
        binding.evict_update_and_fetch_group([cache.handle], [k.data_ptr()], [v.data_ptr()], None, 8)


def weigh64(score, k, q, lse, n_new, scale):
    """(scores, bound); see weights64. Queries of a key go through eight at a time: two additions each, three of the
    lanes, seven of the warps that share them."""
    B, H, n, _ = k.shape
    N, hq, m, _ = q.shape
    g, fan = hq // H, N // B
    w, bound = score.double().clone(), torch.zeros_like(score, dtype=torch.float64)
    for s in range(N):
        b, c = s // fan, m if n_new is None else n_new[s]
        for h in range(hq):
            z = scale * (q[s, h, :c].double() @ k[b, h // g].double().T)
            x = lse[s, h, :c].double()[:, None]
            p = torch.where(x == -math.inf, 0.0, torch.exp(z - x))
            e = 132 * U32 * abs(scale) * q[s, h, :c].double().norm(dim=1)[:, None] * k[b, h // g].double().norm(dim=1)
            w[b, h // g] += p.sum(0)
            bound[b, h // g] += (p * (e + 4 * U32 * (x.abs() + z.abs()) + 2.0 ** -20)).sum(0)
    return w, bound + (12 + 2 * -(-fan * m * g // 8)) * U32 * w.abs() + 1e-37


@pytest.mark.parametrize("B,fan,m,n,hq,hkv,ragged,layout", [
    (1, 1, 1, 1, 1, 1, False, "token"), (2, 1, 1, 100, 8, 2, False, "token"), (32, 1, 1, 512, 32, 8, False, "token"),
    (1, 16, 5, 5000, 32, 8, True, "token"), (3, 2, 3, 33, 28, 4, True, "wide"), (1, 64, 4, 40, 8, 8, False, "head"),
    (2, 1, 9, 31, 24, 1, True, "token"), (1, 3, 1, 257, 40, 8, False, "wide"), (1, 1, 700, 129, 2, 1, False, "head")])
@pytest.mark.parametrize("scale", [None, -0.05])
def test_weights_of_a_step(B, fan, m, n, hq, hkv, ragged, layout, scale):
    k, v = block(20, B, hkv, n)
    g = torch.Generator("cuda").manual_seed(21)
    score = torch.rand(B, hkv, n, device="cuda", generator=g)
    pos = torch.arange(n, device="cuda").int().expand(B, hkv, n).contiguous()
    cache = binding.EvictCache("attention", B, hkv, budget=n + 7, n_sink=0, max_block=1)
    cache.set_state(k, v, pos, score)
    q = rows(22, B * fan, hq, m, layout)
    lse = torch.randn(B * fan, hq, m, device="cuda", generator=g) + math.log(n)
    lse[0, 0, 0] = -math.inf
    n_new = torch.randint(0, m + 1, (B * fan,), device="cuda", generator=g).int() if ragged else None
    if ragged:
        lse[n_new.cpu().argmin(), :, n_new.min():] = math.nan       # padding is not looked at
    cache.weigh(q, lse, n_new=n_new, scale=scale)
    cache.sync()
    at = SCALE if scale is None else scale
    check_weights(cache.view()[3], *weigh64(score, k, q, lse, None if n_new is None else n_new.tolist(), at))
    once = cache.view()[3].clone()
    cache.set_state(k, v, pos, score)
    cache.weigh(q, lse, n_new=n_new, scale=scale)
    assert torch.equal(cache.view()[3], once)                       # the same bits
    cache.close()


def test_counts_out_of_range_are_cut_and_reported():
    k, v = block(23, 1, 2, 50)
    cache = binding.EvictCache("attention", 1, 2, budget=60, max_block=50)
    cache.update_and_fetch(k, v)
    q, lse = rows(24, 2, 4, 3), torch.full((2, 4, 3), 4.0, device="cuda")
    cache.weigh(q, lse, n_new=torch.tensor([-5, 99], dtype=torch.int32).cuda())
    with pytest.raises(binding.EvictError, match="index"):
        cache.sync()
    check_weights(cache.view()[3], *weigh64(torch.zeros(1, 2, 50, device="cuda"), k, q, lse, [0, 3], SCALE))
    empty = binding.EvictCache("attention", 1, 2, budget=60, max_block=50)
    empty.weigh(q, lse)                                             # no rows: nothing to do
    empty.sync()


def test_a_serving_run():
    """Packed prompts, their weights, a cache for each, and decode steps that add theirs."""
    hq, hkv, budget, lens = 8, 2, 96, [400, 60, 1, 250]
    starts = [0]
    for l in lens:
        starts.append(starts[-1] + l)
    m = starts[-1]
    q, k, v = rows(30, 1, hq, m, std=1.5), rows(31, 1, hkv, m), rows(32, 1, hkv, m)
    pk = prompt.Packing(torch.tensor(starts, dtype=torch.int32).cuda())
    lse = torch.empty(1, hq, m, device="cuda")
    prompt.attention(q, k, v, pk, lse=lse)
    score = prompt.weights(q, k, lse, pk, last=32)
    pk.sync()
    for i, (a, e) in enumerate(zip(starts, starts[1:])):
        cache = binding.EvictCache("attention", 1, hkv, budget=budget, n_sink=2, recent=16, max_block=400)
        ref = Plain(1, hkv, budget, 2, 16)
        part = [x[:, :, a:e].contiguous() for x in (k, v, score)]
        cache.update_and_fetch(part[0], part[1], score=part[2])
        ref.update(*part[:2], score=part[2])
        ref.check(cache.view(), i)
        for t in range(6):
            k1, v1 = block(1000 + 10 * i + t, 1, hkv, 1)
            cache.update_and_fetch(k1, v1)
            ref.update(k1, v1)
            ref.check(cache.view(), (i, t))
            q1 = rows(2000 + 10 * i + t, 1, hq, 1, std=1.5)
            one = torch.empty(1, hq, 1, device="cuda")
            out = cache.attend(q1, lse=one, weigh=True)
            assert torch.equal(out, paged.shared_attention(q1, prefix=(ref.k, ref.v)))
            check_weights(cache.view()[3], *weigh64(ref.score, ref.k, q1, one, None, SCALE))
            # every query's weights add up to 1
            assert abs(float((cache.view()[3].double() - ref.score.double()).sum()) - hq) < 1e-3
            ref.score = cache.view()[3].clone()
        cache.sync()
        cache.close()


def test_weights_add_up_behind_a_prefix_and_pages():
    # rows of the cache and own rows under one softmax: what the cache's rows got is what the own rows left
    hq, hkv, n, B = 8, 2, 200, 4
    k, v = block(40, 1, hkv, n)
    cache = binding.EvictCache("attention", 1, hkv, budget=n, n_sink=0, max_block=n)
    cache.update_and_fetch(k, v)
    own = paged.PagedCache(n_pages=40, page_size=16, n_kv_heads=hkv, batch=B, max_rows=64)
    own.grow(9)
    ko, vo = block(42, B, hkv, 9)
    own.append(ko, vo)
    q = rows(44, B, hq, 9)[:, :, 8:]
    lse = torch.empty(B, hq, 1, device="cuda")
    own.attend(q, prefix=cache.view()[:2], lse=lse)
    cache.weigh(q, lse)
    cache.sync()
    z = SCALE * torch.einsum("bhgd,bhnd->bhgn", q.double().reshape(B, hkv, -1, D), ko.double())
    left = torch.exp(z - lse.double().reshape(B, hkv, -1, 1)).sum()
    assert abs(float(cache.view()[3].double().sum() + left) - B * hq) < 1e-3


@pytest.mark.parametrize("default", [True, False], ids=["default", "own"])
def test_weights_on_another_stream(default):
    B, H, n = 2, 2, 64
    mine, other = torch.cuda.Stream(), torch.cuda.Stream()
    made = torch.cuda.current_stream() if default else mine
    k, v = block(50, B, H, 2 * n)
    q, lse = rows(52, B, 8, 2), torch.full((B, 8, 2), 4.0, device="cuda")
    with torch.cuda.stream(made):
        cache = binding.EvictCache("attention", B, H, budget=2 * n, max_block=n)
    first, second = [[x[:, :, i * n:(i + 1) * n].contiguous() for x in (k, v)] for i in range(2)]
    torch.cuda.synchronize()
    with torch.cuda.stream(made):
        torch.cuda._sleep(40_000_000)
        cache.update_and_fetch(*first)
    with torch.cuda.stream(other):
        cache.weigh(q, lse)                         # behind the update
        torch.cuda._sleep(40_000_000)
        cache.weigh(q, lse)                         # before the next one
    with torch.cuda.stream(made):
        cache.update_and_fetch(*second)
    torch.cuda.synchronize()
    cache.sync()
    zero = torch.zeros(B, H, n, device="cuda")
    w, bound = weigh64(zero, first[0], q, lse, None, SCALE)
    check_weights(cache.view()[3][:, :, :n], 2 * w, 2 * bound + 4 * U32 * w)
    assert (cache.view()[3][:, :, n:] == 0).all()
    cache.close()


def test_a_captured_decode_step():
    B, H, hq, budget = 3, 2, 8, 40
    cache, eager = (binding.EvictCache("attention", B, H, budget=budget, n_sink=2, recent=8, max_block=budget) for _ in range(2))
    k0, v0 = block(60, B, H, budget)
    k, v = block(62, B, H, 1)
    q = rows(64, B, hq, 1)
    out, lse = torch.zeros_like(q), torch.zeros(B, hq, 1, device="cuda")

    def step(c):
        c.update_and_fetch(k, v)
        c.attend(q, out=out, lse=lse, weigh=True)

    for c in (cache, eager):
        c.update_and_fetch(k0, v0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for c in (cache, eager):
        binding.evict_set_stream(c.handle, s.cuda_stream)
    with torch.cuda.stream(s):
        for c in (cache, eager):
            step(c)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step(cache)
        for t in range(5):
            for x, seed in ((k, 70), (v, 80), (q, 90)):
                x.copy_(rows(seed + t, *x.shape[:2], 1, "head"))
            g.replay()
            got = out.clone(), lse.clone()
            step(eager)
            assert torch.equal(out, got[0]) and torch.equal(lse, got[1])
            for i, (a, b) in enumerate(zip(cache.view(), eager.view())):
                if i != 2:                          # the captured step's positions are those of its capture
                    assert torch.equal(a, b), (t, i)
    torch.cuda.synchronize()
    cache.sync()
    eager.sync()


def test_tensors_over_the_rows_outlive_the_cache():
    def views():
        cache = binding.EvictCache("attention", 1, 2, budget=40, n_sink=0, max_block=50)
        cache.weigh(rows(71, 1, 4, 1), torch.zeros(1, 4, 1, device="cuda"))         # of no rows
        fetched = cache.update_and_fetch(*block(72, 1, 2, 30))
        cache.weigh(rows(74, 1, 4, 1), torch.full((1, 4, 1), 3.0, device="cuda"))
        cache.sync()
        assert cache.view()[3].shape == (1, 2, 30) and cache.view()[3].data_ptr() == fetched[3].data_ptr()
        return fetched, cache.view()

    fetched, view = views()                         # the cache itself is gone
    other = [torch.full((1 << 20,), 7.0, device="cuda") for _ in range(8)]
    k, v = block(72, 1, 2, 30)
    for x in (fetched, view):
        assert torch.equal(x[0], k) and torch.equal(x[1], v) and torch.equal(x[3], view[3])
        assert torch.equal(x[2], torch.arange(30, device="cuda").int().expand(1, 2, 30)) and (x[3] > 0).all()
    del other


def test_views_of_any_mode():
    cache = binding.EvictCache("attention", 1, 1, budget=8, n_sink=0, max_block=8)
    with torch.inference_mode():
        cache.update_and_fetch(*block(75, 1, 1, 8))
        cache.view()
    cache.view()[3].add_(1.0)                       # the user's own start
    cache.sync()
    assert (cache.view()[3] == 1).all()
    cache.close()


@pytest.mark.parametrize("fan,m,n,hq,hkv", [(40, 3, 70, 8, 2), (3, 100, 33, 16, 2), (513, 1, 300, 4, 4), (1, 257, 40, 1, 1)])
def test_weights_of_more_queries_than_are_looked_through_at_once(fan, m, n, hq, hkv):
    test_weights_of_a_step(1, fan, m, n, hq, hkv, True, "token", None)
    k, v = block(76, 2, hkv, n)
    cache = binding.EvictCache("attention", 2, hkv, budget=n, n_sink=0, max_block=n)
    cache.update_and_fetch(k, v)
    q, lse = rows(78, 2 * fan, hq, m), torch.full((2 * fan, hq, m), 5.0, device="cuda")
    n_new = torch.zeros(2 * fan, dtype=torch.int32)
    n_new[-1] = m                                   # all sequences of the first row, and most of the second, have none
    cache.weigh(q, lse, n_new=n_new.cuda())
    cache.sync()
    assert (cache.view()[3][0] == 0).all()
    check_weights(cache.view()[3], *weigh64(torch.zeros(2, hkv, n, device="cuda"), k, q, lse, n_new.tolist(), SCALE))
    cache.close()


# sizes that take the large products (every SM has a tile of 128 keys, 32768 tile-by-query pairs): a tile of one key, chunks
# of 256 queries that are full, a chunk of which nothing counts before one that does, units that begin inside a share
@pytest.mark.parametrize("B,fan,m,n,hq,hkv,ragged,layout", [
    (1, 16, 5, 2433, 32, 8, True, "token"), (3, 4, 32, 6528, 6, 2, False, "wide"), (24, 1, 9, 900, 40, 8, True, "head"),
    (1, 300, 1, 19457, 8, 1, True, "token")])
def test_weights_of_many_queries_on_many_rows(B, fan, m, n, hq, hkv, ragged, layout):
    assert -(-n // 128) * B * hkv >= 152 and -(-n // 128) * B * fan * m * hq >= 32768
    test_weights_of_a_step(B, fan, m, n, hq, hkv, ragged, layout, None)


def test_many_padded_queries_and_keys_of_infinities():
    n, fan, m = 20000, 64, 3
    k, v = block(80, 1, 2, n)
    k[0, 0, 5], k[0, 1, n - 1, 3] = math.inf, math.nan
    cache = binding.EvictCache("attention", 1, 2, budget=n, n_sink=0, max_block=n)
    cache.update_and_fetch(k, v)
    q, lse = rows(82, fan, 16, m), torch.full((fan, 16, m), 5.0, device="cuda")
    lse[50, 3], lse[60, 3], lse[60, 12], lse[61, 0, 1] = -math.inf, math.inf, math.nan, 9.0
    n_new = torch.zeros(fan, dtype=torch.int32)
    n_new[48:] = torch.tensor([3, 0, 3, 1] * 4)     # nothing in the first 1152 query rows of a head
    n_new[60] = 0                                   # which has the NaN
    cache.weigh(q, lse, n_new=n_new.cuda())
    cache.sync()
    zero = torch.zeros(1, 2, n, device="cuda")
    got, (w, bound) = cache.view()[3], weigh64(zero, k, q, lse, n_new.tolist(), SCALE)
    other = torch.ones(1, 2, n, dtype=torch.bool)
    other[0, 0, 5] = other[0, 1, n - 1] = False
    check_weights(got[other.cuda()], w[other.cuda()], bound[other.cuda()])
    assert torch.isnan(got[~other.cuda()]).all()
    cache.close()
    none = binding.EvictCache("attention", 1, 2, budget=n, n_sink=0, max_block=n)
    none.update_and_fetch(k, v)
    none.weigh(q, lse, n_new=torch.zeros(fan, dtype=torch.int32).cuda())
    none.sync()
    assert (none.view()[3] == 0).all()
    none.close()


def test_many_queries_with_counts_out_of_range():
    n = 10000
    k, v = block(84, 1, 2, n)
    cache = binding.EvictCache("attention", 1, 2, budget=n, max_block=n)
    cache.update_and_fetch(k, v)
    q, lse = rows(86, 64, 8, 3), torch.full((64, 8, 3), 4.0, device="cuda")
    n_new = torch.full((64,), 2, dtype=torch.int32)
    n_new[7], n_new[40] = -5, 99
    cache.weigh(q, lse, n_new=n_new.cuda())
    with pytest.raises(binding.EvictError, match="index"):
        cache.sync()
    check_weights(cache.view()[3], *weigh64(torch.zeros(1, 2, n, device="cuda"), k, q, lse, n_new.clamp(0, 3).tolist(), SCALE))
    cache.close()


def test_a_captured_step_of_many_queries():
    n, fan = 4000, 24
    k, v = block(88, 1, 8, n)
    stream = torch.cuda.Stream()
    q, lse = rows(90, fan, 32, 4), torch.full((fan, 32, 4), 6.0, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        cache = binding.EvictCache("attention", 1, 8, budget=n, n_sink=0, max_block=n)
        cache.update_and_fetch(k, v)
        cache.weigh(q, lse)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            cache.weigh(q, lse)
        q.mul_(0.5)
        graph.replay()
        graph.replay()
        stream.synchronize()
    cache.sync()
    got = cache.view()[3]
    zero = torch.zeros(1, 8, n, device="cuda")
    w1, b1 = weigh64(zero, k, q.double() * 2, lse, None, SCALE)
    w2, b2 = weigh64(zero, k, q, lse, None, SCALE)
    check_weights(got, w1 + 2 * w2, b1 + 2 * b2 + 6 * U32 * (w1 + 2 * w2))
    cache.close()


@pytest.mark.parametrize("m", [1, 8])
def test_offsets_past_32_bits(m):
    # 2.3e9 elements of kept keys, by few queries (the register products) and by more; the last caches' rows
    B, H, hq, n = 64, 8, 32, 35001
    assert B * H * n * D > 2 ** 31
    g = torch.Generator("cuda").manual_seed(130)
    k = torch.randn(B, H, n, D, device="cuda", generator=g, dtype=torch.bfloat16)
    cache = binding.EvictCache("attention", B, H, budget=n, n_sink=0, max_block=1)
    cache.set_state(k, k, torch.arange(n, device="cuda").int().expand(B, H, n).contiguous(), torch.zeros(B, H, n, device="cuda"))
    q = rows(131, B, hq, m)
    lse = torch.randn(B, hq, m, device="cuda", generator=g) + 10.0
    cache.weigh(q, lse)
    cache.sync()
    for b in (0, 60, 63):
        zero = torch.zeros(1, H, n, device="cuda")
        check_weights(cache.view()[3][b:b + 1], *weigh64(zero, k[b:b + 1], q[b:b + 1], lse[b:b + 1], None, SCALE))
    cache.close()


def test_weighing_beside_prompts_on_other_streams():
    # three kernels at once that each take all of an SM's tensor memory
    n = 6000
    k, v = block(140, 1, 8, n)
    cache = binding.EvictCache("attention", 1, 8, budget=n, n_sink=0, max_block=n)
    cache.update_and_fetch(k, v)
    q, lse = rows(142, 16, 32, 3), torch.full((16, 32, 3), 6.0, device="cuda")
    qp, kp, vp = rows(143, 1, 32, 2500), rows(144, 1, 8, 2500), rows(145, 1, 8, 2500)
    lp = torch.empty(1, 32, 2500, device="cuda")
    ref_out, ref_lse = prompt.attention(qp, kp, vp, lse=lp), lp.clone()
    ref_w = prompt.weights(qp, kp, ref_lse)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(6):
        cache.weigh(q, lse)
        with torch.cuda.stream(a):
            l = torch.empty(1, 32, 2500, device="cuda")
            got.append((prompt.attention(qp, kp, vp, lse=l), l))
        with torch.cuda.stream(b):
            got.append(prompt.weights(qp, kp, ref_lse))
    torch.cuda.synchronize()
    cache.sync()
    for x in got:
        if isinstance(x, tuple):
            assert torch.equal(x[0], ref_out) and torch.equal(x[1], ref_lse)
        else:
            assert torch.equal(x, ref_w)
    w, bound = weigh64(torch.zeros(1, 8, n, device="cuda"), k, q, lse, None, SCALE)
    check_weights(cache.view()[3], 6 * w, 6 * bound + 8 * U32 * 6 * w)
    cache.close()
