"""Prompts' attention and weights of keys where sizes and values are rare, against plain 64-bit forms."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from kv_cache_token_bf16_gb300 import prompt  # noqa: E402
from tests.paged_util import D, U32  # noqa: E402
from tests.prompt_util import SCALE, check_prompt, check_weights, weights64  # noqa: E402


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


def test_weights_round_once_where_the_maximum_moves():
    """The logits of a tile's first 32 columns are weighed before a far larger one is seen in the next, and their bf16
    weights move along. The last query of each sequence has the logits a, b, c at keys 0, 1, 32 (few bits, so exact)
    and far lower ones elsewhere; row 1 alone has a 1 in its column of V. The exponents' reference is a whole number, so
    that weight has the bits of e^b as bf16. e^b itself is off by 2^-16 at most (the logit times log2 e: 2^-22 of up to
    29; ex2 2^-22), and so is the sum; the result's own rounding is half a step, 2^-8 of it."""
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
    total = sum(torch.exp(x.double()) for x in (a, b, c))
    fits = torch.zeros(n, dtype=torch.bool)
    for side in (-1, 1):                            # either rounding where e^b is that close to the middle of two
        ref = (torch.exp(b.double()) * (1 + side * 2.0 ** -16)).float().bfloat16().double() / total
        fits |= (got - ref).abs() <= (2.0 ** -8 + 2.0 ** -15) * got.abs()
    assert fits.all(), int((~fits).sum())
