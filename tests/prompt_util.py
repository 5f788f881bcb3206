"""Plain 64-bit forms of prompts' attention, the weights of keys and eviction by them, with the bounds that the
kernels' results keep. Rows and pairs in 64 bits on the tensors' device."""
import math

import torch

from tests.paged_util import D, U32, attend_bounds

SCALE = 1 / math.sqrt(D)


def spans_of(starts, batch, m):
    """(plane, first row, length) of every sequence."""
    if starts is None:
        return [(b, 0, m) for b in range(batch)]
    return [(0, a, e - a) for a, e in zip(starts, starts[1:])]


def _logits(q, k, b, a, l, h, g, scale):
    z = scale * (q[b, h, a:a + l].double() @ k[b, h // g, a:a + l].double().T)
    see = torch.ones(l, l, dtype=torch.bool, device=q.device).tril_()
    return torch.where(see, z, -math.inf), see


def prompt64(q, k, v, spans, scale=SCALE):
    """(out, lse, weight): weight is the sum of p |v|, for the bound. NaN where no sequence has a token."""
    out = torch.full(q.shape, math.nan, dtype=torch.float64, device=q.device)
    wt, lse = out.clone(), torch.full(q.shape[:3], math.nan, dtype=torch.float64, device=q.device)
    g = q.shape[1] // k.shape[1]
    for b, a, l in spans:
        for h in range(q.shape[1] if l else 0):
            z, see = _logits(q, k, b, a, l, h, g, scale)
            top = z.amax(1, keepdim=True)
            w = torch.exp(z - torch.where(top == -math.inf, 0.0, top))
            s = w.sum(1, keepdim=True)
            vh = v[b, h // g, a:a + l].double()
            p, fine = w / s, torch.isfinite(vh)
            out[b, h, a:a + l], wt[b, h, a:a + l] = p @ torch.where(fine, vh, 0.0), p @ torch.where(fine, vh, 0.0).abs()
            for j in (~fine.all(1)).nonzero()[:, 0].tolist():       # such a row reaches those that see it alone
                add = torch.where(fine[j], 0.0, vh[j]) * p[j:, j:j + 1]
                out[b, h, a + j:a + l] += add
                wt[b, h, a + j:a + l] += add.abs()
            lse[b, h, a:a + l] = (top + torch.log(s))[:, 0]
    return out, lse, wt


def weights64(q, k, lse, spans, last=0, scale=SCALE):
    """(weights, bound). A weight's exponent is off by the logit's error, 132 U32 |scale| |q| |k| (see attend_bounds),
    and by the roundings of lse * log2 e, of the product and of their difference, 4 U32 (|lse| + |z|); ex2 is within
    2^-21, and a sum of n positive terms passes through at most 20 additions in a step of 128 queries, one for every
    step and one for every part of a unit (152 at most), each within U32 of the whole."""
    w = torch.full(k.shape[:3], math.nan, dtype=torch.float64, device=q.device)
    bound = w.clone()
    g = q.shape[1] // k.shape[1]
    for b, a, l in spans:
        if not l:
            continue
        w[b, :, a:a + l] = bound[b, :, a:a + l] = 0.0
        first = max(0, l - last) if last else 0
        for h in range(q.shape[1]):
            z, see = _logits(q, k, b, a, l, h, g, scale)
            x = lse[b, h, a:a + l].double()[:, None]
            p = torch.where(x == -math.inf, 0.0, torch.exp(z - x))[first:]
            e = 132 * U32 * abs(scale) * q[b, h, a:a + l].double().norm(dim=1)[:, None] * k[b, h // g, a:a + l].double().norm(dim=1)
            e = (e + 4 * U32 * (x.abs() + torch.where(see, z.abs(), 0.0)))[first:] + 2.0 ** -20
            w[b, h // g, a:a + l] += p.sum(0)
            bound[b, h // g, a:a + l] += torch.where(p > 0, p * e, 0.0).sum(0)
    steps = g * max(-(-l // 128) for _, _, l in spans) if spans else 0
    return w, bound + (20 + steps + 152) * U32 * w.abs() + 1e-37


def check_prompt(q, k, v, spans, out, lse, scale=SCALE, out_was=None, lse_was=None):
    """out and lse within their bounds; elsewhere what they were."""
    ro, rl, wt = prompt64(q, k, v, spans, scale)
    kmax = k.double().norm(dim=-1)
    kmax = float(kmax[torch.isfinite(kmax)].max()) if kmax.numel() else 0.0
    bo, bl = (x.to(q.device) for x in attend_bounds(q, kmax, ro.cpu(), rl.cpu(), wt.cpu(), scale, weights=2.0 ** -8))
    has = torch.zeros(q.shape[0], q.shape[2], dtype=torch.bool, device=q.device)
    for b, a, l in spans:
        has[b, a:a + l] = True
    for got, ref, bound, was, name in ((out, ro, bo, out_was, "out"), (lse, rl, bl, lse_was, "lse")):
        if got is None:
            continue
        on = has[:, None].expand(got.shape[:3])
        x, r, lim = got.double()[on], ref[on], bound[on]
        same = (x == r) | (torch.isnan(x) & torch.isnan(r))
        bad = ~same & ~((x - r).abs() <= lim)
        assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} off, by {float(((x - r).abs() / lim)[bad].max()):.3g} bounds"
        if was is not None:
            assert (got[~on] == was).all(), f"{name}: rows of no sequence were written"


def check_weights(got, ref, bound, was=None):
    on = ~torch.isnan(bound)
    x, r, lim = got.double()[on], ref[on], bound[on]
    bad = ~((x - r).abs() <= lim)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} weights off, by {float(((x - r).abs() / lim)[bad].max()):.3g} bounds"
    if was is not None:
        assert (got[~on] == was).all(), "weights of no sequence were written"


def kept(score, n_sink, recent, budget):
    """Indices that stay, in order: the protected rows, then the heaviest, the first of equals (NaN last)."""
    n = score.shape[-1]
    if n <= budget:
        return torch.arange(n).expand(score.shape[:-1] + (n,))
    at = torch.arange(n)
    rank = torch.nan_to_num(score.double().cpu(), nan=-math.inf, posinf=math.inf, neginf=-math.inf)
    safe = (at < n_sink) | (at >= n - recent)
    order = torch.where(safe, 0, 1).expand(rank.shape)
    idx = rank.sort(dim=-1, descending=True, stable=True).indices
    idx = idx.gather(-1, order.gather(-1, idx).sort(dim=-1, stable=True).indices)
    return idx[..., :budget].sort(dim=-1).values
