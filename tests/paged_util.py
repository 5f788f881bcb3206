"""Plain 64-bit forms of rotation and attention, and the bounds that the kernels' results keep."""
import math

import torch

D = 128
U32 = 2.0 ** -24                    # half a step of fp32, relative
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U32}


def inv_freq(rotary_dim, base=10000.0):
    i = torch.arange(0, rotary_dim, 2, dtype=torch.float64)
    return (base ** (-i / rotary_dim)).float()


def rotate64(x, pos, freq, axis, pairs="half", transpose=False, scale=1.0):
    """x [B, H, m, 128], pos [axes, B, m] integers: the rotation in 64 bits, on the CPU. Angles are
    reduced in whole turns by exact rational arithmetic where positions are far."""
    x = x.double().cpu()
    pos = pos.cpu()
    r = 2 * len(freq)
    ang = torch.zeros(pos.shape[1], pos.shape[2], len(freq), dtype=torch.float64)
    for i, w in enumerate(freq.tolist()):
        ang[..., i] = pos[axis[i]].double() * w
    if transpose:
        ang = -ang
    c, s = (scale * ang.cos())[:, None], (scale * ang.sin())[:, None]
    y = x.clone()
    if pairs == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y[..., :r // 2], y[..., r // 2:r] = a * c - b * s, a * s + b * c
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = a * c - b * s, a * s + b * c
    return y


def rotate_bound(x, ref, rotary_dim, pairs, dtype, scale=1.0):
    """|error| of a rotated element. fp32: the angle in half turns is truncated to 2^-31 and rounded to
    fp32 (2^-25): pi * (2^-31 + 2^-25) < 1.6 U32 of an angle; sincospif is within one step (2 U32 of
    1); scaling it, two products and a sum round once each (4 U32). Under 8 U32 of |x| + |y|, and
    the output's rounding. bf16: the angle of up to pi rounds twice (2 pi U32 < 6.3 U32) and __sinf and
    __cosf are within 2^-21.19 < 7.1 U32 on [-pi, pi], with the other 4 under 18 U32."""
    units = 8 if dtype is torch.float32 else 18
    a = x.double().cpu().abs()
    t = torch.zeros_like(a)
    r = rotary_dim
    if pairs == "half":
        t[..., :r // 2] = t[..., r // 2:r] = a[..., :r // 2] + a[..., r // 2:r]
    else:
        t[..., 0:r:2] = t[..., 1:r:2] = a[..., 0:r:2] + a[..., 1:r:2]
    return units * U32 * abs(scale) * t + HALF[dtype] * ref.abs() + 1e-38


def attend64(q, prefix, own, n_new=None, scale=None):
    """(out, lse, weight) in 64 bits on the CPU, row by row. prefix: (K, V) [P, H, n, 128] or None; own: a list
    of (K, V) [H, rows, 128] of each sequence, or None; weight: sum of p |v|, for the bound. Padding
    rows are NaN."""
    q = q.double().cpu()
    B, hq, m, _ = q.shape
    scale = 1 / math.sqrt(D) if scale is None else scale
    out = torch.full_like(q, math.nan)
    wt = torch.full_like(q, math.nan)
    lse = torch.full((B, hq, m), math.nan, dtype=torch.float64)
    for b in range(B):
        n = m if n_new is None else n_new[b]
        ks, vs = [], []
        if prefix is not None and prefix[0].shape[2]:
            p = b // (B // prefix[0].shape[0])
            ks.append(prefix[0][p].double().cpu())
            vs.append(prefix[1][p].double().cpu())
        n_pre = ks[0].shape[1] if ks else 0
        rows = 0
        if own is not None:
            ks.append(own[b][0].double().cpu())
            vs.append(own[b][1].double().cpu())
            rows = ks[-1].shape[1]
        k, v = torch.cat(ks, 1), torch.cat(vs, 1)
        g = hq // k.shape[0]
        if n == 0:
            continue
        see = torch.full((n,), n_pre)
        if own is not None:
            see = n_pre + (rows - n + torch.arange(n) + 1).clamp(min=0)
        hide = torch.arange(k.shape[1])[None] >= see[:, None]
        for h in range(hq):
            z = (scale * (q[b, h, :n] @ k[h // g].T)).masked_fill(hide, -math.inf)
            top = z.amax(1, keepdim=True) if z.shape[1] else torch.full((n, 1), -math.inf, dtype=torch.float64)
            w = torch.exp(z - torch.where(top == -math.inf, 0.0, top))
            l = w.sum(1, keepdim=True)
            p = w / torch.where(see[:, None] > 0, l, 1.0)
            vh = torch.where(hide.all(0)[:, None], 0.0, v[h // g])      # rows that no query sees
            out[b, h, :n], wt[b, h, :n] = p @ vh, p @ vh.abs()
            lse[b, h, :n] = (top + torch.log(l))[:, 0]
    return out, lse, wt


def attend_bounds(q, kmax, out, lse, wt, scale=None, weights=2.0 ** -16):
    """|error| of out and of lse. A logit is 128 exact products summed in fp32 and scaled: off by at most
    e = 132 U32 * |scale| * |q| |k| (Cauchy-Schwarz for sum |q_d k_d|), so a weight is off by 2 e
    relative to the sum, ex2 and the sums by 2^-18 (2^17 terms in fp32 chains of 2^6), the weights'
    own rounding by `weights`; then the output's rounding. lse: e, 2^-18 and its own roundings."""
    scale = 1 / math.sqrt(D) if scale is None else scale
    e = 132 * U32 * abs(scale) * q.double().cpu().norm(dim=-1) * kmax
    bo = (2 * e + 2.0 ** -17 + 2 * weights)[..., None] * wt + 2.0 ** -8 * out.abs() + 1e-30
    return bo, e + 2.0 ** -18 + 4 * U32 * lse.abs()


def gather(pages, table, lens):
    """[n_pages, H, page, 128] -> per sequence [H, lens[b], 128]."""
    P = pages.shape[2]
    res = []
    for b, n in enumerate(lens):
        idx = table[b, :max(1, -(-n // P))].long()
        res.append(pages[idx].transpose(0, 1).flatten(1, 2)[:, :n])
    return res
