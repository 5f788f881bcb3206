"""The bounds that the GPU tests of attention go by catch what they are there for (no GPU needed)."""
import pytest

torch = pytest.importorskip("torch")

from tests.paged_util import D, attend64, attend_bounds  # noqa: E402


def problem(n, one_hot):
    g = torch.Generator().manual_seed(1)
    q, k = 0.4 * torch.randn(1, 1, 4, D, generator=g), torch.randn(1, 1, n, D, generator=g)
    v = torch.randn(1, 1, n, D, generator=g)
    if one_hot:
        j = torch.arange(n)
        v = torch.zeros(1, 1, n, D)
        v[0, 0, j, j % D] = (8 + (j // D) % 8).float() / 8
    return [x.to(torch.bfloat16) for x in (q, k, v)]


def within(q, k, v, out, weights):
    ref, lse, wt = attend64(q, (k, v), None)
    bound = attend_bounds(q, float(k.double().norm(dim=-1).max()), ref, lse, wt, weights=weights)[0]
    return bool(((out.to(torch.bfloat16).double() - ref).abs() <= bound).all())


@pytest.mark.parametrize("n", [40, 1000, 2000])
def test_lost_doubled_and_exchanged_rows_are_seen(n):
    q, k, v = problem(n, True)
    good = attend64(q, (k, v), None)[0]
    assert within(q, k, v, good, 2.0 ** -8)
    g = torch.Generator().manual_seed(2)
    for j in [0, n - 1] + torch.randint(0, n, (20,), generator=g).tolist():
        lost, twice, swapped = v.clone(), v.clone(), v.clone()
        lost[0, 0, j] = 0
        twice[0, 0, j] *= 2
        i = (j + 1) % n
        swapped[0, 0, [i, j]] = v[0, 0, [j, i]]
        for bad in (lost, twice, swapped):
            assert not within(q, k, v, attend64(q, (k, bad), None)[0], 2.0 ** -8), j


def test_weights_of_eight_bits_are_told_from_fifteen():
    # a weight cut to bf16, without its second part, is off by up to 2^-7
    q, k, v = problem(300, True)
    z = (q.double() @ k.double().transpose(-1, -2)) * D ** -0.5
    w = torch.exp(z - z.amax(-1, keepdim=True))
    cut = (w.float().view(torch.int32) & -65536).view(torch.float32).double()
    rest = (w - cut).to(torch.bfloat16).double()
    total = w.sum(-1, keepdim=True)
    assert within(q, k, v, (cut + rest) @ v.double() / total, 2.0 ** -15)
    assert not within(q, k, v, cut @ v.double() / total, 2.0 ** -15)
