"""Every row of V arrives once, with its own weight: checks that a lost, doubled or exchanged row fails."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests.paged_util import D  # noqa: E402
from tests.test_gpu_attend import CASES, _built, attend, check, make  # noqa: E402,F401

IDS = ["-".join(str(x) for x in c[:7]) for c in CASES]


def tile_rows(case):
    """(own query rows of a KV head, its prefix's)."""
    B, hq, h, m, n_prefix, groups = case[:6]
    return m * hq // h, m * hq // h * (B // groups)


def few_rows_only(case):
    """The rule of the split between the two kernels: tiles of 16 query rows where a sequence fills at most
    two, and its prefix's rows as well, over few rows."""
    own, pre = tile_rows(case)
    n_prefix, groups = case[4], case[5]
    tiles = -(-pre // 16)
    return own <= 32 and (n_prefix == 0 or (tiles <= 2 and tiles * n_prefix * groups <= 2048))


FEW = [(c, i) for c, i in zip(CASES, IDS) if few_rows_only(c)]
MORE = [(1, 16, 1, 1, 2000, 1, 16, None, None), (2, 8, 1, 1, 1000, 1, 16, [700, 2001], None),
        (9, 32, 8, 2, 0, 1, 16, [2 + 113 * b for b in range(9)], [b % 3 for b in range(9)]),
        (3, 8, 2, 3, 100, 3, 256, [3, 1000, 513], None)]


@pytest.mark.parametrize("case", [c for c, _ in FEW] + MORE, ids=[i for _, i in FEW] + [f"more{i}" for i in range(len(MORE))])
def test_few_rows_keep_fifteen_bits_of_every_weight(case):
    """Two bf16 parts of a weight: the second's half step, 2^-8 of what is below 2^-7 of the weight."""
    assert few_rows_only(case)
    s = make(700, *case)
    out, lse = attend(s, out=torch.zeros_like(s["q"]))
    check(s, out, lse, weights=2.0 ** -15)


def mark_rows(s, h, n_prefix):
    """V of stream row j (prefix first) and head g: zeros but for column (j + 17 g) % 128, which holds one
    of eight values by j // 128, none below half another. A column's result is the weights of its few rows alone."""
    def rows_of(first, n):
        j = first + torch.arange(n)
        v = torch.zeros(h, n, D)
        for g in range(h):
            v[g, torch.arange(n), (j + 17 * g) % D] = (8 + (j // D) % 8).float() / 8
        return v.to(torch.bfloat16).cuda()
    if s["prefix"]:
        s["prefix"][1].copy_(rows_of(0, n_prefix).expand_as(s["prefix"][1]))
    for b, (_, v) in enumerate(s.get("own") or []):
        n = v.shape[1]
        v.copy_(rows_of(n_prefix, n))
        page = s["vp"].shape[2]
        for at in range(0, n, page):
            s["vp"][int(s["table"][b, at // page]), :, :min(page, n - at)] = v[:, at:at + page]


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_every_row_of_v_can_be_told_from_the_others(case):
    # the bound is 2^-7 of the weights of a column's own rows: at most some twenty of them, not hundreds
    s = make(710, *case)
    s["q"].mul_(0.25)                               # flat weights: no row may hide behind another
    mark_rows(s, case[2], case[4])
    out, lse = attend(s, out=torch.zeros_like(s["q"]))
    check(s, out, lse, weights=2.0 ** -15 if few_rows_only(case) else 2.0 ** -8)
