"""Prompts' attention and weights of keys where sizes and values are rare, against plain 64-bit forms."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from kv_cache_token_bf16_gb300 import binding, prompt  # noqa: E402
from tests.paged_util import D, U32, attend_bounds  # noqa: E402
from tests.prompt_util import SCALE, check_prompt, check_weights, weights64  # noqa: E402
from tests.test_gpu_prompt import rows, run, starts_of  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built(lib):
    pass


def big(seed, heads, m):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(1, m, heads, D, device="cuda", generator=g, dtype=torch.bfloat16).transpose(1, 2)


def test_a_plane_of_eight_million_tokens():
    # 16385 sequences; by the plane's length its blocks would be 2^31 steps. Some sequences against calls' own bounds.
    lens = [512] * 16384 + [77]
    starts = torch.tensor([0] + lens).cumsum(0)
    m = int(starts[-1])
    pk = prompt.Packing(starts.int().cuda())
    q, k, v = big(1, 1, m), big(2, 1, m), big(3, 1, m)
    lse = torch.empty(1, 1, m, device="cuda")
    out = prompt.attention(q, k, v, pk, out=torch.empty_like(q), lse=lse)
    w = prompt.weights(q, k, lse, pk)
    pk.sync()
    for i in (0, 1, 8191, 16383, 16384):
        a, b = int(starts[i]), int(starts[i + 1])
        x = [t[:, :, a:b].contiguous() for t in (q, k, v, out, lse)]
        check_prompt(*x[:3], [(0, 0, b - a)], *x[3:])
        check_weights(w[:, :, a:b], *weights64(x[0], x[1], x[4], [(0, 0, b - a)]))
    assert torch.isfinite(lse).all() and torch.isfinite(w).all()


def test_a_sequence_of_a_million_tokens():
    """Some queries and keys against 64 bits. The sum of a softmax is a chain of 2^15 additions, each rounded either way by
    up to 2^-24 of the sum so far: six of their deviations are 6 2^-24 / 3 2^7.5 < 2^-15. A key's weight is one of 2^13."""
    m = 1 << 20
    q, k, v = big(30, 1, m), big(31, 1, m), big(32, 1, m)
    lse = torch.empty(1, 1, m, device="cuda")
    out = prompt.attention(q, k, v, out=torch.empty_like(q), lse=lse)
    w = prompt.weights(q, k, lse)
    torch.cuda.synchronize()
    at = torch.tensor([0, 1, 5000, m // 2 + 77, m - 129, m - 2, m - 1], device="cuda")
    kd, vd = k[0, 0].double(), v[0, 0].double()
    z = SCALE * (q[0, 0, at].double() @ kd.T)
    z = torch.where(torch.arange(m, device="cuda") <= at[:, None], z, -math.inf)
    ref, p = torch.logsumexp(z, 1), torch.softmax(z, 1)
    bo, bl = attend_bounds(q[0, 0, at], float(kd.norm(dim=1).max()), (p @ vd).cpu(), ref.cpu(), (p @ vd.abs()).cpu(), weights=2.0 ** -8)
    assert bool(((lse[0, 0, at].double() - ref).abs().cpu() <= bl + 2.0 ** -15).all())
    assert bool(((out[0, 0, at].double() - p @ vd).abs().cpu() <= bo).all())
    for j in (0, 300, m - 1000, m - 1):
        z = SCALE * (q[0, 0, j:].double() @ kd[j])
        p = torch.exp(z - lse[0, 0, j:].double())
        off = 132 * U32 * SCALE * q[0, 0, j:].double().norm(dim=1) * kd[j].norm() + 4 * U32 * (lse[0, 0, j:].double().abs() + z.abs())
        bound = (p * (off + 2.0 ** -20)).sum() + 2.0 ** -15 * p.sum()
        assert abs(float(w[0, 0, j] - p.sum())) <= float(bound), j


def test_a_window_over_four_million_tokens():
    # the keys' weights of the last 64 queries: two steps a block, 2^31 if every query counted
    m, h, last = 1 << 22, 4, 64
    q, k = big(4, h, m), big(5, h, m)
    lse = torch.randn(1, h, m, device="cuda", generator=torch.Generator("cuda").manual_seed(6)) + 16.0
    w = prompt.weights(q, k, lse, last=last)
    torch.cuda.synchronize()
    at = torch.arange(m, device="cuda")
    for i in range(h):
        for a in (0, 1 << 21, m - 1000):
            e = min(m, a + 100_000)
            z = SCALE * (q[0, i, m - last:].double() @ k[0, i, a:e].double().T)
            x = lse[0, i, m - last:].double()[:, None]
            p = torch.where(at[a:e] <= at[m - last:, None], torch.exp(z - x), 0.0)
            # the bound of weights64
            off = 132 * U32 * SCALE * q[0, i, m - last:].double().norm(dim=1)[:, None] * k[0, i, a:e].double().norm(dim=1)
            bound = (p * (off + 4 * U32 * (x.abs() + z.abs()) + 2.0 ** -20)).sum(0) + 180 * U32 * p.sum(0) + 1e-37
            assert bool(((w[0, i, a:e].double() - p.sum(0)).abs() <= bound).all())


@pytest.mark.parametrize("hq,hkv,lens,last", [(4, 2, [300], 0), (8, 2, [1700], 0), (4, 4, [128, 640, 3], 0), (8, 1, [900, 300], 20)])
def test_queries_without_a_log_sum_exp_may_hold_anything(hq, hkv, lens, last):
    # no weights of a query whose log-sum-exp is -infinity, whatever its row is: padding, for one
    m = sum(lens)
    g = torch.Generator("cuda").manual_seed(7)
    q, k = big(8, hq, m), big(9, hkv, m)
    lse = torch.randn(1, hq, m, device="cuda", generator=g) + 5.0
    starts = torch.tensor([0] + lens).cumsum(0).tolist()
    drop = torch.rand(1, hq, m, device="cuda", generator=g) < 0.1
    drop[:, :, 128:256] = False                     # whole steps of queries that all count
    drop[:, 1, m - 1] = drop[:, :, 17] = True
    lse[drop] = -math.inf
    bad = q.clone()
    for i, x in enumerate((math.nan, math.inf, -math.inf)):
        bad[drop & (torch.arange(m, device="cuda") % 3 == i)] = x
    pk = prompt.Packing(torch.tensor(starts, dtype=torch.int32).cuda())
    w = prompt.weights(bad, k, lse, pk, last=last)
    pk.sync()
    spans = [(0, a, e - a) for a, e in zip(starts, starts[1:])]
    check_weights(w, *weights64(q, k, lse, spans, last))
    assert torch.equal(w, prompt.weights(q, k, lse, pk, last=last))


def test_weights_round_twice_at_most_where_the_maximum_moves():
    """The logits of a tile's first 32 columns are weighed before a far larger one is seen in the next, and their bf16
    weights move along. The last query of each sequence has the logits a, b, c at keys 0, 1, 32 and far lower ones
    elsewhere; row 1 alone has a 1 in its column of V. Its weight is rounded as it is made and as it moves, 2^-8 each, and
    the result once more; exponents and sums add 2^-15 (their logits are exact, of up to 29 in base 2)."""
    n, l = 1024, 64
    g = torch.Generator().manual_seed(550)
    a, b, c = [(lo + (hi - lo) * torch.rand(n, generator=g)).bfloat16() for lo, hi in ((4, 5), (2, 4), (14, 20))]
    q = torch.zeros(n, l, D, dtype=torch.bfloat16)
    q[:, -1, 0], q[:, -1, 1], q[:, -1, 2], q[:, -1, 3] = a, b, c, 1
    k, v = torch.zeros_like(q), torch.zeros_like(q)
    k[:, 0, 0] = k[:, 1, 1] = k[:, 32, 2] = 1
    k[:, [j for j in range(l) if j not in (0, 1, 32)], 3] = -200
    v[:, 1, 5] = 1
    q, k, v = (x.view(1, 1, n * l, D).cuda() for x in (q, k, v))
    pk = prompt.Packing((torch.arange(n + 1) * l).int().cuda())
    got = prompt.attention(q, k, v, pk, scale=1.0)
    pk.sync()
    got = got.view(n, l, D)[:, -1, 5].double().cpu()
    ref = torch.exp(b.double()) / sum(torch.exp(x.double()) for x in (a, b, c))
    assert ((got / ref - 1).abs() <= (1 + 2.0 ** -8) ** 3 * (1 + 2.0 ** -15) - 1).all()


# the largest plane whose units go uncut however few they are, and the first that is cut: some 50 units for 152 SMs
@pytest.mark.parametrize("m", [1536, 1537])
@pytest.mark.parametrize("cut", [False, True])
def test_planes_around_the_longest_that_goes_uncut(m, cut):
    q, k, v = rows(10, 1, 8, m, std=1.5), rows(11, 1, 2, m), rows(12, 1, 2, m)
    run(q, k, v, starts_of([m - 700, 1, 699]) if cut else None)


def test_a_key_of_nan_has_nan_weights_and_no_other_key():
    m = 700
    q, k = big(13, 8, m), big(14, 2, m)
    lse = torch.randn(1, 8, m, device="cuda", generator=torch.Generator("cuda").manual_seed(15)) + 5.0
    w, bound = weights64(q, k, lse, [(0, 0, m)])
    k[0, 0, 300, 5], k[0, 1, 699] = math.nan, math.inf
    got = prompt.weights(q, k, lse)
    bad = torch.zeros(1, 2, m, dtype=torch.bool, device="cuda")
    bad[0, 0, 300] = bad[0, 1, 699] = True          # (infinities of both signs among a row's products)
    assert torch.isnan(got[bad]).all()
    check_weights(got[~bad], w[~bad], bound[~bad])


LOG2E = math.log2(math.e)


def base2(scale):
    """What the kernels multiply a product by: the header's scale, a little larger, in base 2 and rounded to fp32."""
    return torch.tensor(scale * LOG2E * (1 + 2.0 ** -23), dtype=torch.float32).double().item()


def test_weights_of_large_log_sum_exps_do_not_lean():
    """Products of one element are exact, so a weight is 2^(z base2 - lse log2 e) but for roundings: of lse log2 e, half a
    step of 2^-11 at up to 8192, either way, whose mean over 16384 terms is within six of its deviations, 6 ln 2
    2^-11 / sqrt(12) / 128 < 5e-6; of the logit's difference to it (2^-22) and of ex2 (2^-22); of at most 300 additions
    (2^-24 each). log2 e alone in fp32 is 1.3e-8 of itself short: 4000 of it would be 5.3e-5."""
    m, hq = 2048, 8
    g = torch.Generator().manual_seed(16)
    q, k = torch.zeros(1, hq, m, D, dtype=torch.bfloat16), torch.zeros(1, 1, m, D, dtype=torch.bfloat16)
    q[..., 0] = torch.randint(230, 254, (1, hq, m), generator=g) * 16.0
    k[..., 0] = 1.0
    lse = q[..., 0].float() + torch.rand(1, hq, m, generator=g) - 0.5
    got = prompt.weights(q.cuda(), k.cuda(), lse.cuda(), scale=1.0)[0, 0].double().cpu()
    p = torch.exp2(q[..., 0].double() * base2(1.0) - lse.double() * LOG2E)[0].sum(0)
    ref = p.flip(0).cumsum(0).flip(0)
    off = (got[0] / ref[0] - 1).abs()
    assert off <= 5e-6 + 2 * 2.0 ** -22 + 300 * U32, float(off)


@pytest.mark.parametrize("m,n", [(1, 300), (209, 2500)], ids=["few", "many"])
def test_steps_of_large_log_sum_exps_are_exact(m, n):
    """As above, and every query of a head is the same, so all roundings lean to one side: that of lse log2 e would be
    2e-5 and more here, and is made up for. What stays: the difference's, half a step of 2^-18 at up to 64, times ln 2;
    ex2 and the factor, 2^-22 and 2^-24; at most 66 additions."""
    h = 8
    g = torch.Generator().manual_seed(17)
    l = []
    while len(l) < h:                               # log-sum-exps whose product with log2 e is rounded by much
        x = torch.rand((), generator=g) * 100 + 960
        y = x.double().item() * LOG2E
        if abs(torch.tensor(y).float().double().item() - y) * math.log(2) > 2e-5:
            l.append(x.item())
    lse = torch.tensor(l)[None, :, None].expand(1, h, m).contiguous()
    q = torch.zeros(1, h, m, D, dtype=torch.bfloat16)
    q[..., 0] = 1000.0
    k = torch.zeros(1, h, n, D, dtype=torch.bfloat16)
    k[..., 0] = 1 + torch.randint(-1, 2, (1, h, n), generator=g) / 128
    k[..., 0] *= (torch.tensor(l)[None, :, None] / 1000).bfloat16()
    cache = binding.EvictCache("attention", 1, h, budget=n, n_sink=0, max_block=n)
    cache.update_and_fetch(k.cuda(), k.cuda())
    cache.weigh(q.cuda(), lse.cuda(), scale=1.0)
    cache.sync()
    got = cache.view()[3].double().cpu()
    x = 1000.0 * k[..., 0].double() * base2(1.0) - lse[:, :, :1].double() * LOG2E
    assert x.abs().max() < 40
    ref = m * torch.exp2(x)
    off = ((got - ref).abs() / ref).max()
    assert off <= 2.0 ** -19 * math.log(2) + 2.0 ** -22 + U32 + 66 * U32, float(off)
    cache.close()


def test_weights_of_random_rows_do_not_lean():
    """Logits spread by 4: the weights are those of logits of some 13. The tensor cores cut 0.9e-7 of such a logit off in
    the mean and the scale adds 1.2e-7, so what stays is 0.4e-6 of a weight, 1.2e-6 without. Its deviation from weight to
    weight: half a step of 2^-19 of lse log2 e and as much of the products' sums, some 1e-6."""
    m = 2048
    q, k = rows(18, 1, 4, m, std=4.0), rows(19, 1, 4, m)
    lse = torch.empty(1, 4, m, dtype=torch.float64, device="cuda")
    for h in range(4):
        z = SCALE * (q[0, h].double() @ k[0, h].double().T)
        lse[0, h] = torch.logsumexp(z.masked_fill(torch.ones(m, m, dtype=torch.bool, device="cuda").triu_(1), -math.inf), 1)
    lse = lse.float()
    ref, _ = weights64(q, k, lse, [(0, 0, m)])
    off = prompt.weights(q, k, lse).double() - ref
    lean, norm = float(off.sum() / ref.sum()), float(off.norm() / ref.norm())
    assert abs(lean) <= 0.8e-6 and norm <= 2.5e-6, (lean, norm)


@pytest.mark.parametrize("fan,m,n", [(1, 3, 300), (24, 4, 3000)], ids=["few", "many"])
def test_steps_of_queries_without_a_log_sum_exp_may_hold_anything(fan, m, n):
    hq, hkv = 32, 8
    k = rows(20, 1, hkv, n, "head")
    q, lse = rows(21, fan, hq, m), torch.full((fan, hq, m), 6.0, device="cuda")
    drop = torch.rand(fan, hq, m, device="cuda", generator=torch.Generator("cuda").manual_seed(22)) < 0.2
    drop[0, :2] = True
    lse[drop] = -math.inf
    bad = q.clone()
    bad[drop] = math.nan
    bad[0, 0] = math.inf
    got = []
    for x in (q, bad):
        cache = binding.EvictCache("attention", 1, hkv, budget=n, n_sink=0, max_block=n)
        cache.update_and_fetch(k, k)
        cache.weigh(x, lse)
        cache.sync()
        got.append(cache.view()[3].clone())
        cache.close()
    assert torch.equal(*got) and torch.isfinite(got[0]).all() and (got[0] > 0).all()


def test_views_are_the_callers_own_objects():
    k = rows(23, 1, 2, 40, "head")
    cache = binding.EvictCache("attention", 1, 2, budget=40, n_sink=0, max_block=40)
    first = cache.update_and_fetch(k, k)
    first[0].requires_grad_()
    first[3].unsqueeze_(0)
    q = rows(24, 1, 4, 1)
    cache.attend(q, weigh=True)                     # (a K that requires a gradient would be refused)
    second = cache.view()
    cache.sync()
    assert second[3].shape == (1, 2, 40) and not second[0].requires_grad and second[0].data_ptr() == first[0].data_ptr()
    assert torch.equal(first[3][0], second[3]) and (second[3] > 0).all()
    cache.close()
    del first, second
