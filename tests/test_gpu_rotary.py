"""Rotary positions and the append to pages, against the definitions in 64 bits."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from kv_cache_token_bf16_gb300 import binding, paged  # noqa: E402
from tests.paged_util import D, inv_freq, rotate64, rotate_bound  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def rows(seed, b, h, m, dtype="bf16", layout="head"):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(b, m, h, D, generator=g).to(TYPES[dtype]).cuda()
    return x.transpose(1, 2) if layout == "token" else x.transpose(1, 2).contiguous()


def positions(seed, axes, b, m, lo=0, hi=1 << 17):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(lo, hi, (axes, b, m), generator=g, dtype=torch.int64).to(torch.int32).cuda()


def check(got, x, pos, freq, axis, pairs, transpose=False, scale=1.0):
    ref = rotate64(x, pos, freq, axis, pairs, transpose, scale)
    err = (got.double().cpu() - ref).abs()
    bound = rotate_bound(x, ref, 2 * len(freq), pairs, got.dtype, scale)
    assert bool((err <= bound).all()), float((err / bound).max())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("pairs", ["half", "adjacent"])
@pytest.mark.parametrize("rdim,axes,b,m,layout", [(128, 1, 1, 1, "head"), (128, 3, 2, 37, "token"), (96, 2, 3, 5, "head"),
                                                  (20, 4, 2, 3, "token"), (2, 1, 5, 2, "head"), (64, 1, 1, 1031, "token")])
def test_rotation_matches_the_definition(dtype, pairs, rdim, axes, b, m, layout):
    q, k = rows(1, b, 6, m, dtype, layout), rows(2, b, 2, m, dtype, layout)
    freq, axis = inv_freq(rdim), [i % axes for i in range(rdim // 2)]
    r = paged.Rotary(rdim, inv_freq=freq, axis=axis, n_axes=axes, pairs=pairs)
    pos = positions(3, axes, b, m)
    yq, yk = paged.rotate(r, (q, k), pos=pos)
    check(yq, q, pos, freq, axis, pairs)
    check(yk, k, pos, freq, axis, pairs)
    # behind the rotated elements the row is copied, bit for bit
    assert torch.equal(yq[..., rdim:], q[..., rdim:])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_far_and_negative_positions(dtype):
    # 2^31 * 1 radian in 64 bits is exact to 2^-22 of a radian only where the frequency has few bits:
    # powers of two make the reference's product exact
    freq = torch.tensor([2.0 ** -i for i in range(32)])
    pos = torch.tensor([[[2 ** 31 - 1, -2 ** 31, -1, 0, 1, 123456789, -987654321, 1 << 30]]], dtype=torch.int32).cuda()
    x = rows(5, 1, 3, 8, dtype)
    r = paged.Rotary(64, inv_freq=freq)
    check(paged.rotate(r, x, pos=pos), x, pos, freq, [0] * 32, "half")
    check(paged.rotate(r, x, pos=pos, transpose=True), x, pos, freq, [0] * 32, "half", transpose=True)


def test_without_positions_tokens_count_from_the_base():
    x, freq = rows(6, 3, 4, 17), inv_freq(128)
    r = paged.Rotary()
    pos = (1000 + torch.arange(17)).expand(1, 3, 17)
    check(paged.rotate(r, x, pos_base=1000), x, pos, freq, [0] * 64, "half")
    assert torch.equal(paged.rotate(r, x, pos_base=1000), paged.rotate(r, x, pos=pos[0].to(torch.int32).contiguous().cuda()))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("pairs", ["half", "adjacent"])
def test_in_place_scaled_and_unaligned(dtype, pairs):
    freq, pos = inv_freq(96), positions(8, 1, 2, 33)
    r = paged.Rotary(96, inv_freq=freq, pairs=pairs, scale=0.75)
    x = rows(7, 2, 5, 33, dtype)
    y = x.clone()
    assert paged.rotate(r, y, pos=pos, out=y) is y
    check(y, x, pos, freq, [0] * 48, pairs, scale=0.75)
    # the same rows one element off: taken element by element, in place as well
    flat = torch.zeros(x.numel() + 1, dtype=x.dtype, device="cuda")
    z = flat[1:].view(x.shape)
    z.copy_(x)
    check(paged.rotate(r, z, pos=pos), x, pos, freq, [0] * 48, pairs, scale=0.75)
    paged.rotate(r, z, pos=pos, out=z)
    check(z, x, pos, freq, [0] * 48, pairs, scale=0.75)
    assert float(flat[0]) == 0.0


def test_copied_elements_keep_their_bits():
    bits = torch.arange(-(1 << 15), 1 << 15, dtype=torch.int32).to(torch.int16).view(1, 1, 512, D).cuda()
    x = bits.view(torch.bfloat16)
    y = paged.rotate(paged.Rotary(32), x, pos_base=5)
    assert torch.equal(y.view(torch.int16)[..., 32:], bits[..., 32:])
    z = paged.rotate(paged.Rotary(20), x, pos_base=5)
    assert torch.equal(z.view(torch.int16)[..., 20:], bits[..., 20:])


@pytest.mark.parametrize("pairs", ["half", "adjacent"])
def test_the_transposed_rotation_is_the_gradient(pairs):
    freq, pos = inv_freq(64), positions(9, 2, 2, 11)
    axis = [i % 2 for i in range(32)]
    r = paged.Rotary(64, inv_freq=freq, axis=axis, pairs=pairs, scale=1.25)
    x, gy = rows(10, 2, 3, 11, "fp32"), rows(11, 2, 3, 11, "fp32")
    gx = paged.rotate(r, gy, pos=pos, transpose=True)
    check(gx, gy, pos, freq, axis, pairs, transpose=True, scale=1.25)
    # against differences: d/dx of <gy, rotate(x)> along single elements, in 64 bits (the map is linear)
    for e in (0, 1, 31, 32, 63, 64, 127):
        d = torch.zeros_like(x, dtype=torch.float64).cpu()
        d[1, 2, 7, e] = 1.0
        up = rotate64(x.double().cpu() + d, pos, freq, axis, pairs, scale=1.25)
        dn = rotate64(x.double().cpu() - d, pos, freq, axis, pairs, scale=1.25)
        diff = float(((up - dn) / 2 * gy.double().cpu()).sum())
        assert abs(diff - float(gx[1, 2, 7, e])) <= 16 * 2.0 ** -24 * 1.25 * float(gy[1, 2, 7].abs().max()) + 1e-12
    back = paged.rotate(paged.Rotary(64, inv_freq=freq, axis=axis, pairs=pairs), paged.rotate(
        paged.Rotary(64, inv_freq=freq, axis=axis, pairs=pairs), x, pos=pos), pos=pos, transpose=True)
    # each of the two rotations is off by at most 8 U32 (|x| + |y|) <= 16 U32 max |x|, and the second doubles
    assert float((back - x).abs().max()) <= 3 * 16 * 2.0 ** -24 * float(x.abs().max())


def test_rotation_on_another_stream_and_in_a_graph():
    r, x = paged.Rotary(), rows(12, 2, 4, 9)
    pos = positions(13, 1, 2, 9)
    want = paged.rotate(r, x, pos=pos)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(x)
    with torch.cuda.stream(s):
        paged.rotate(r, x, pos=pos, out=out)
    s.synchronize()
    assert torch.equal(out, want)
    p, g = pos.clone(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        paged.rotate(r, x, pos=p, out=out)
    for shift in (0, 1000):
        p.copy_(pos + shift)
        out.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, paged.rotate(r, x, pos=p))


def test_bad_rotate_tensors_are_refused():
    r, x = paged.Rotary(), rows(14, 2, 4, 3)
    for bad in (dict(pos=positions(1, 2, 2, 3)), dict(pos=positions(1, 1, 2, 3).long()), dict(out=x.float()),
                dict(out=x[:, :2]), dict(pos=positions(1, 1, 2, 3).cpu())):
        with pytest.raises(ValueError):
            paged.rotate(r, x, **bad)
    for bad in (x[0], x[..., :64], x.half(), x.transpose(2, 3), (x, x, x), (x, x.float()), (x, x[:1])):
        with pytest.raises(ValueError):
            paged.rotate(r, bad)


# --- append ---------------------------------------------------------------------------------
def pool(seed, n_pages, h, page, dtype="bf16", apart=False):
    """K and V pages; `apart`: both inside one tensor [n_pages, 2, ...], so pages are strided."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n_pages, 2, h, page, D, generator=g).to(TYPES[dtype]).cuda()
    return (x[:, 0], x[:, 1]) if apart else (x[:, 0].contiguous(), x[:, 1].contiguous())


def table_of(seed, batch, width, n_pages):
    g = torch.Generator().manual_seed(seed)
    return torch.randperm(n_pages, generator=g)[:batch * width].view(batch, width).to(torch.int32).cuda()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("page,m,lens,new,rdim,axes,given,apart", [
    (16, 1, [1, 16, 17, 40], None, 128, 1, False, False),
    (16, 5, [5, 0, 33, 31], [5, 0, 3, 1], 128, 3, True, True),
    (64, 70, [70, 200, 65], [70, 1, 64], 96, 1, True, False),
    (256, 3, [255, 257], None, 20, 2, False, True),
    (32, 9, [9, 50], [4, 9], 0, 1, False, False),
])
def test_append_matches_the_definition(dtype, page, m, lens, new, rdim, axes, given, apart):
    B, H, HQ = len(lens), 3, 6
    width = -(-max(lens) // page)
    kp, vp = pool(20, B * width + 2, H, page, dtype, apart)
    table = table_of(21, B, width, B * width + 2)
    k0, v0 = kp.clone(), vp.clone()
    cache = paged.PagedCache(k_pages=kp, v_pages=vp, table=table, lens=torch.tensor(lens, dtype=torch.int32).cuda())
    k, v, q = rows(22, B, H, m, dtype, "token"), rows(23, B, H, m, dtype), rows(24, B, HQ, m, dtype, "token")
    freq, axis = inv_freq(max(rdim, 2)), [i % axes for i in range(max(rdim, 2) // 2)]
    rot = paged.Rotary(rdim, inv_freq=freq, axis=axis, n_axes=axes) if rdim else None
    counts = new if new is not None else [m] * B
    at = torch.tensor([[lens[b] - counts[b] + t for t in range(m)] for b in range(B)])
    pos = positions(25, axes, B, m) if given else None
    used = pos if given else (at + 700).expand(axes, B, m)
    q_out = torch.full_like(q, 7.0)
    cache.append(k, v, rotary=rot, pos=pos, pos_base=700, q=q, q_out=q_out,
                 n_new=torch.tensor(new, dtype=torch.int32).cuda() if new is not None else None)
    cache.sync()
    rk = rotate64(k, used, freq, axis) if rdim else k.double().cpu()
    rq = rotate64(q, used, freq, axis) if rdim else q.double().cpu()
    bk, bq = rotate_bound(k, rk, rdim, "half", k.dtype), rotate_bound(q, rq, rdim, "half", q.dtype)
    written = set()
    for b in range(B):
        for t in range(m):
            if t >= counts[b]:
                assert bool((q_out[b, :, t] == 7.0).all())
                continue
            pg, row = int(table[b, int(at[b, t]) // page]), int(at[b, t]) % page
            written.add((pg, row))
            assert bool(((kp[pg, :, row].double().cpu() - rk[b, :, t]).abs() <= bk[b, :, t]).all())
            assert torch.equal(vp[pg, :, row], v[b, :, t])
            assert bool(((q_out[b, :, t].double().cpu() - rq[b, :, t]).abs() <= bq[b, :, t]).all())
            kp[pg, :, row], vp[pg, :, row] = k0[pg, :, row], v0[pg, :, row]
    assert len(written) == sum(counts)
    assert torch.equal(kp, k0) and torch.equal(vp, v0)       # nothing else was written


def test_append_skips_and_reports_what_lies_outside():
    B, H, page, m = 4, 2, 16, 2
    kp, vp = pool(30, 6, H, page)
    k0 = kp.clone()
    table = torch.tensor([[0, 1], [99, 2], [-1, 3], [4, 5]], dtype=torch.int32).cuda()
    lens = torch.tensor([2, 2, 2, 33], dtype=torch.int32).cuda()    # sequence 3 outgrows its two pages by a row
    cache = paged.PagedCache(k_pages=kp, v_pages=vp, table=table, lens=lens)
    k, v = rows(31, B, H, m), rows(32, B, H, m)
    q, q_out = rows(33, B, 4, m), torch.zeros(B, 4, m, D, dtype=torch.bfloat16, device="cuda")
    cache.append(k, v, q=q, q_out=q_out)
    with pytest.raises(binding.EvictError, match="index") as e:
        cache.sync()
    assert e.value.code == binding.EVICT_EDEVICE
    cache.sync()                                                    # reported once
    k0[0, :, :2] = k[0].clone()
    k0[5, :, 15] = k[3, :, 0]
    assert torch.equal(kp, k0)
    assert torch.equal(q_out, q)
    # new counts outside [0, m] are taken as the nearest of these; a row before the sequence's first is skipped
    kp.copy_(torch.zeros_like(kp))
    lens.copy_(torch.tensor([2, 1, 0, 1]))
    table.copy_(torch.tensor([[0, 0], [1, 1], [2, 2], [3, 3]]))
    cache.append(k, v, n_new=torch.tensor([5, -3, 0, 2], dtype=torch.int32).cuda())
    with pytest.raises(binding.EvictError, match="index"):
        cache.sync()
    want = torch.zeros_like(kp)
    want[0, :, :2] = k[0]
    want[3, :, 0] = k[3, :, 1]
    assert torch.equal(kp, want)


def test_append_beyond_32_bit_offsets():
    H, page = 8, 256
    n_pages = (1 << 31) // (H * page * D) + 3                       # the last pages lie past 2^31 elements
    kp = torch.zeros(n_pages, H, page, D, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    table = torch.tensor([[n_pages - 1], [n_pages - 2]], dtype=torch.int32).cuda()
    cache = paged.PagedCache(k_pages=kp, v_pages=vp, table=table, lens=torch.tensor([256, 1], dtype=torch.int32).cuda())
    k, v = rows(34, 2, H, 1), rows(35, 2, H, 1)
    cache.append(k, v)
    cache.sync()
    assert torch.equal(kp[n_pages - 1, :, 255], k[0, :, 0]) and torch.equal(vp[n_pages - 2, :, 0], v[1, :, 0])
    kp[n_pages - 1, :, 255] = 0
    kp[n_pages - 2, :, 0] = 0
    assert not bool(kp.any())


def test_pages_are_handed_out_and_taken_back():
    c = paged.PagedCache(n_pages=5, page_size=16, n_kv_heads=2, batch=3, max_rows=40)
    c.grow([17, 1, 0])
    assert c.rows() == [17, 1, 0] and c.lens.tolist() == [17, 1, 0]
    used = c.table[0, :2].tolist() + c.table[1, :1].tolist()
    assert len(set(used)) == 3
    with pytest.raises(ValueError, match="free"):
        c.grow([0, 32, 16])
    with pytest.raises(ValueError, match="pages"):
        c.grow([32, 0, 0])
    assert c.rows() == [17, 1, 0]
    c.release(0)
    c.grow([0, 31, 16])
    assert c.rows() == [0, 32, 16]
    live = c.table[1, :2].tolist() + c.table[2, :1].tolist()
    assert len(set(live)) == 3 and c.table[1, 0].item() == used[2]
    with pytest.raises(ValueError):
        c.grow([1, 1])
    given = paged.PagedCache(k_pages=c.k_pages, v_pages=c.v_pages, table=c.table, lens=c.lens)
    with pytest.raises(ValueError, match="caller"):
        given.grow(1)


def test_bad_append_tensors_are_refused():
    c = paged.PagedCache(n_pages=5, page_size=16, n_kv_heads=2, batch=3, max_rows=40)
    k = rows(36, 3, 2, 1)
    for a, kw in (((k.float(), k), {}), ((k, k[:, :, :0]), {}), ((k[:2], k[:2]), {}), ((k, k), dict(q_out=k)),
                  ((k, k), dict(q=rows(1, 3, 4, 2))), ((k, k), dict(n_new=torch.zeros(2, dtype=torch.int32).cuda()))):
        with pytest.raises(ValueError):
            c.append(*a, **kw)


@pytest.mark.parametrize("shared", [0, 1, 2])
def test_outputs_like_an_expanded_input(shared):
    # an input that repeats itself along an axis gets an output that does not
    shape = [3, 4, 5, D]
    small = list(shape)
    small[shared] = 1
    g = torch.Generator().manual_seed(77)
    x = torch.randn(*small, generator=g).cuda().expand(*shape)
    rot = paged.Rotary()
    out = paged.rotate(rot, x, pos_base=9)
    assert torch.equal(out, paged.rotate(rot, x.contiguous(), pos_base=9))
    q = x.to(torch.bfloat16)[:, :, :, :].contiguous()[:, :1].expand(*shape)
    k = torch.randn(1, 2, 40, D, generator=g).to(torch.bfloat16).cuda()
    got = paged.shared_attention(q, prefix=(k, k))
    assert torch.equal(got, paged.shared_attention(q.contiguous(), prefix=(k, k)))
