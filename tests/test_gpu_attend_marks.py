"""Infinities in values that only some queries of a unit see, with both groups of the wide kernel at them."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests.paged_util import D, attend64, attend_bounds  # noqa: E402
from tests.test_gpu_attend import _built, attend, make  # noqa: E402,F401


def plant(s, b, tokens, first_col):
    """+inf in one column of V of these rows of sequence b (`s["own"]` holds 0 there): {column: first such row}."""
    page, seen = s["vp"].shape[2], {}
    for i, j in enumerate(tokens):
        col = (first_col + 7 * i) % D
        s["vp"][int(s["table"][b, j // page]), :, j % page, col] = math.inf
        s["own"][b][1][:, j, col] = 0
        seen[col] = min(j, seen.get(col, j))
    return seen


def check_planted(s, out, planted):
    new = s["new"].tolist()
    ro, _, wt = attend64(s["q"], s["prefix"], s["own"], new)
    kmax = max(float(k.double().norm(dim=-1).max()) for k, _ in s["own"] if k.numel())
    bound = attend_bounds(s["q"], kmax, ro, torch.zeros(1), wt, weights=2.0 ** -8)[0]
    got = out.double().cpu()
    for b, n in enumerate(new):
        last = s["own"][b][0].shape[1] - n + torch.arange(n)          # the last row that each query sees
        inf = torch.zeros(n, D, dtype=torch.bool)
        for col, j in planted.get(b, {}).items():
            inf[:, col] = last >= j
        g, e = got[b, :, :n], (got[b, :, :n] - ro[b, :, :n]).abs()
        assert bool((g[:, inf] == math.inf).all()), b
        assert bool((e <= bound[b, :, :n])[:, ~inf].all()), b


@pytest.mark.parametrize("hq,h,m,n_prefix", [(8, 8, 300, 0), (60, 2, 5, 2100)], ids=["joint", "shared"])
def test_marks_outlive_the_units_behind(hq, h, m, n_prefix):
    # a CTA goes from a unit with marked rows, most of them behind the first group's queries, to many
    # units in which the second group has no work
    B = 400
    lens = [1 + b % 3 for b in range(B)]
    new = list(lens)
    full = {0: (m, m), 150: (m, 3 * m + 20), 399: (m, m + 1)}
    for b, (n, l) in full.items():
        new[b], lens[b] = n, l
    s = make(600, B, hq, h, m, n_prefix, 1, 16, lens, new)
    clean, _ = attend(s)
    planted = {}
    for b, (n, l) in full.items():
        rows = [l - n + t for t in range(n) if t in (1, 60) or (n > 130 and 130 <= t < 256 and t % 5 == 0) or t == n - 1]
        planted[b] = plant(s, b, rows, b)
    out, lse = attend(s)
    check_planted(s, out, planted)
    for b in range(B):
        if b not in full:
            assert torch.equal(out[b], clean[b])
    for _ in range(10):
        again, l2 = attend(s)
        assert torch.equal(again, out) and torch.equal(l2, lse)


def test_marked_rows_of_a_sequence_alone_and_in_a_batch():
    # the same sequence with and without others behind it: the same infinities
    lens, new = [300] + [2] * 300, [300] + [2] * 300
    s = make(610, 301, 4, 4, 300, 0, 1, 16, lens, new)
    cols = plant(s, 0, list(range(129, 299, 3)), 0)
    out, _ = attend(s)
    one = dict(s, q=s["q"][:1], new=s["new"][:1], own=s["own"][:1])
    from kv_cache_token_bf16_gb300 import paged
    one["cache"] = paged.PagedCache(k_pages=s["kp"], v_pages=s["vp"], table=s["table"][:1],
                                    lens=torch.tensor([300], dtype=torch.int32).cuda())
    alone, _ = attend(one)
    check_planted(one, alone, {0: cols})
    check_planted(s, out, {0: cols})
    assert torch.equal(alone[0] == math.inf, out[0] == math.inf)
