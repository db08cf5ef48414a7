"""GPU: quantising writes into the serving cache and reads back, against the
plain quantiser (codes exactly) and fp64 values."""
import numpy as np
import pytest
import torch

import transform_codec_b200 as kvc
from serving_ref import FORMATS, HostCache, code_values, quantise, signless

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}


def _rows(rng, n, heads, dim, dt):
    x = rng.standard_normal((n, heads, dim)) * np.exp(rng.standard_normal((n, heads, 1)))
    return torch.from_numpy(x.astype(np.float32)).to(dt)


def _filled(fmt, heads, dim, page, pages, seed):
    g = torch.Generator().manual_seed(seed)
    c = kvc.QuantCache(fmt, heads, dim, page, pages)
    for t in (c.codes, c.micro):
        if t is not None:
            t.copy_(torch.randint(0, 120, t.shape, dtype=torch.uint8, generator=g))
    c.scales.copy_(torch.rand(c.scales.shape, generator=g))
    return c


def _expect(c, before, k, v, slots):
    """The cache's arrays (CPU) after the write, by the plain quantiser."""
    codes, scales, micro = (None if t is None else t.clone() for t in before)
    qc, qs, qm = quantise(c.format, torch.stack((k, v), 1))
    for i, s in enumerate(slots.tolist()):
        if s < 0:
            continue
        p, at = s // c.page_tokens, s % c.page_tokens
        codes[p, :, :, at], scales[p, :, :, at] = qc[i], qs[i]
        if micro is not None:
            micro[p, :, :, at] = qm[i]
    return codes, scales, micro


def _arrays(c):
    return c.codes.cpu(), c.scales.cpu(), None if c.micro is None else c.micro.cpu()


def _same(c, want):
    codes, scales, micro = _arrays(c)
    assert torch.equal(signless(c.format, codes), signless(c.format, want[0]))
    assert torch.equal(scales.nan_to_num(-7.0), want[1].nan_to_num(-7.0))
    if micro is not None:
        assert torch.equal(micro, want[2])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("n,heads,dim,page", [(1, 1, 32, 16), (1, 8, 128, 64), (3, 5, 96, 16), (33, 12, 64, 32),
                                              (70, 2, 256, 1024), (65, 3, 160, 16), (700, 8, 128, 64)])
def test_write_matches_the_plain_quantiser(fmt, dt, n, heads, dim, page):
    rng = np.random.default_rng(n * 31 + dim)
    k, v = (_rows(rng, n, heads, dim, DT[dt]) for _ in range(2))
    pages = -(-n // page) + 1
    c = _filled(FORMATS[fmt], heads, dim, page, pages, n)
    slots = torch.from_numpy(rng.permutation(pages * page)[:n].astype(np.int64))
    slots[2::5] = -1
    want = _expect(c, _arrays(c), k, v, slots)
    kvc.cache_write(c, k.cuda(), v.cuda(), slots.cuda())
    _same(c, want)
    assert kvc.read_result(c.res) == (kvc.OK, 0)


@pytest.mark.parametrize("fmt", FORMATS)
def test_write_many_tokens(fmt):
    """Enough rows for several a thread, and a tile that the last tokens do not fill."""
    rng = np.random.default_rng(5)
    n, heads, dim, page = 4099, 8, 64, 16
    k, v = (_rows(rng, n, heads, dim, torch.bfloat16) for _ in range(2))
    c = _filled(FORMATS[fmt], heads, dim, page, 300, 1)
    slots = torch.from_numpy(rng.permutation(300 * page)[:n].astype(np.int64))
    want = _expect(c, _arrays(c), k, v, slots)
    kvc.cache_write(c, k.cuda(), v.cuda(), slots.cuda())
    _same(c, want)


@pytest.mark.parametrize("fmt", FORMATS)
def test_write_strided_inputs(fmt):
    """Views of a fused projection, and [head][token] slices."""
    rng = np.random.default_rng(9)
    n, heads, dim = 37, 4, 64
    fused = _rows(rng, n, 5 * heads, dim, torch.float16)
    k, v = fused[:, heads:2 * heads], fused[:, 3 * heads:4 * heads]
    slots = torch.arange(n, dtype=torch.int64) + 5
    g = fused.cuda()
    c = _filled(FORMATS[fmt], heads, dim, 16, 4, 2)
    want = _expect(c, _arrays(c), k, v, slots)
    kvc.cache_write(c, g[:, heads:2 * heads], g[:, 3 * heads:4 * heads], slots.cuda())
    _same(c, want)
    slices = torch.stack((k, v)).transpose(1, 2).contiguous().cuda()  # [2][heads][n][dim]
    c2 = _filled(FORMATS[fmt], heads, dim, 16, 4, 2)
    kvc.cache_write(c2, slices[0].transpose(0, 1), slices[1].transpose(0, 1), slots.cuda())
    _same(c2, want)


@pytest.mark.parametrize("fmt", FORMATS)
def test_write_special_rows(fmt):
    """Zeros, NaN, infinities, values below the floor, the largest finite value, negative zeros, single spikes."""
    f = torch.zeros(12, 2, 64)
    f[1, :, 3] = float("nan")
    f[2, 0, 60] = float("inf")
    f[2, 1, 0] = -float("inf")
    f[3] = 2.0 ** -97
    f[4] = 2.0 ** -96
    f[5] = torch.finfo(torch.float32).max
    f[6] = -0.0
    f[7, :, 17] = 3.0
    f[8] = -1e30
    f[9] = torch.linspace(-1, 1, 64)
    f[10] = 2.0 ** -149
    f[11, :, 0], f[11, :, 1:] = 1.0, 2.0 ** -20
    slots = torch.arange(12, dtype=torch.int64)
    c = _filled(FORMATS[fmt], 2, 64, 16, 1, 3)
    want = _expect(c, _arrays(c), f, f.flip(0), slots)
    kvc.cache_write(c, f.cuda(), f.flip(0).cuda(), slots.cuda())
    _same(c, want)
    assert torch.isnan(c.scales[0, 0, :, 1]).all() and torch.isnan(c.scales[0, 0, :, 2]).all()
    assert (c.scales[0, 0, :, 3] == 0).all() and (c.scales[0, 0, :, 10] == 0).all()
    out = torch.zeros(2, 2, 12, 64, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    kvc.cache_read(c, i32(0)[None], i32(0), i32(0, 12), out)
    got = out[0].cpu()
    assert torch.isnan(got[:, 1]).all() and torch.isnan(got[:, 2]).all()
    assert torch.isfinite(got[:, 3:]).all() and (got[:, 3] == 0).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_halfway_values(fmt):
    """Quotients that lie exactly between two codes go to the even one."""
    peak = {"e4m3": 448.0, "int8": 127.0, "e2m1": 2688.0}[fmt]
    x = torch.zeros(1, 1, 32)
    if fmt == "int8":
        x[0, 0] = torch.arange(32) - 15.5
    elif fmt == "e4m3":
        x[0, 0] = torch.cat([(torch.arange(16) + 8.5) * 2.0, (torch.arange(16) + 0.5) * 2.0 ** -9])
    else:
        x[0, 0] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 4) * 448.0
    x[0, 0, 31] = peak  # scale 1 up to the fp32 product
    k = x * torch.tensor([1.0])
    c = _filled(FORMATS[fmt], 1, 32, 16, 1, 4)
    slots = torch.zeros(1, dtype=torch.int64)
    want = _expect(c, _arrays(c), k, -k, slots)
    kvc.cache_write(c, k.cuda(), (-k).cuda(), slots.cuda())
    _same(c, want)


def test_slots_out_of_range_are_refused_on_the_device():
    c = _filled(kvc.CACHE_INT8, 2, 64, 16, 3, 5)
    k = torch.randn(4, 2, 64).to(torch.bfloat16)
    slots = torch.tensor([7, 48, 2 ** 40, 12], dtype=torch.int64)
    want = _expect(c, _arrays(c), k, k, torch.tensor([7, -1, -1, 12]))
    kvc.cache_write(c, k.cuda(), k.cuda(), slots.cuda())
    _same(c, want)
    assert kvc.read_result(c.res)[0] == kvc.ERR_INVALID
    kvc.cache_write(c, k.cuda(), k.cuda(), torch.full((4,), -1, dtype=torch.int64, device="cuda"))
    assert kvc.read_result(c.res)[0] == kvc.ERR_INVALID  # until the caller clears it
    c.res.zero_()
    kvc.cache_write(c, k.cuda(), k.cuda(), torch.tensor([0, 1, 2, 47], device="cuda"))
    assert kvc.read_result(c.res)[0] == kvc.OK


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("heads,dim,page,lens", [(1, 32, 16, [1]), (8, 128, 64, [511]), (3, 96, 16, [5, 0, 40, 17]),
                                                 (12, 64, 32, [700, 1, 333]), (2, 256, 16, [33, 64])])
def test_read_ranges(fmt, dt, heads, dim, page, lens):
    host = HostCache(FORMATS[fmt], heads, dim, page, lens, seed=dim)
    c = host.gpu()
    start = [n // 3 for n in lens]
    n = [a - b for a, b in zip(lens, start)]
    out_start = np.concatenate([[2], 2 + np.cumsum(n)])  # the first two rows and the last three are not asked for
    total = int(out_start[-1]) + 3
    out = torch.full((2, heads, total, dim), 7.0, dtype=DT[dt], device="cuda")
    i32 = lambda x: torch.tensor(list(x), dtype=torch.int32, device="cuda")  # noqa: E731
    kvc.cache_read(c, host.table.cuda(), i32(start), i32(out_start), out)
    want = torch.full((2, heads, total, dim), 7.0, dtype=torch.float64)
    for b in range(len(lens)):
        want[:, :, out_start[b]:out_start[b + 1]] = host.values(b)[:, :, start[b]:]
    got = out.double().cpu()
    assert torch.equal(got[:, :, :2], want[:, :, :2]) and torch.equal(got[:, :, -3:], want[:, :, -3:])
    # the fp32 product, then the rounding to the type: half a step each
    f = torch.finfo(DT[dt])
    bound = want.abs() * (2.0 ** -24 + f.eps / 2 * (1 + 2.0 ** -23)) + f.smallest_normal * f.eps / 2
    assert ((got - want).abs() <= bound).all()
    assert kvc.read_result(c.res) == (kvc.OK, 0)


def test_read_refuses_bad_indices_on_the_device():
    host = HostCache(kvc.CACHE_E4M3, 2, 64, 16, [40, 20], seed=1)
    c = host.gpu()
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    whole = torch.zeros(2, 2, 60, 64, device="cuda")
    kvc.cache_read(c, host.table.cuda(), i32(0, 0), i32(0, 40, 60), whole)
    assert kvc.read_result(c.res)[0] == kvc.OK
    bad = host.table.clone()
    bad[0, 1] = c.n_pages
    for table, start, rows in ((bad, (0, 0), slice(16, 32)), (host.table, (0, -5), slice(40, 45)),
                               (host.table, (1000, 0), slice(0, 40))):
        c.res.zero_()
        out = torch.full_like(whole, 9.0)
        kvc.cache_read(c, table.cuda(), i32(*start), i32(0, 40, 60), out)
        assert kvc.read_result(c.res)[0] == kvc.ERR_INVALID
        assert (out[:, :, rows] == 9.0).all()
    c.res.zero_()
    out = torch.full((2, 2, 50, 64), 9.0, device="cuda")  # ranges that pass the end of out: what fits is read
    kvc.cache_read(c, host.table.cuda(), i32(0, 0), i32(0, 40, 60), out)
    assert torch.equal(out, whole[:, :, :50])
    assert kvc.read_result(c.res)[0] == kvc.ERR_INVALID


def test_offsets_beyond_32_bits():
    """A cache of more than 2^32 code bytes: its last pages are written and read back."""
    heads, dim, page = 8, 256, 1024
    pages = (1 << 32) // (2 * heads * page * dim) + 3
    c = kvc.QuantCache(kvc.CACHE_INT8, heads, dim, page, pages)
    assert c.codes.numel() > 1 << 32
    rng = np.random.default_rng(2)
    n = 50
    k, v = (_rows(rng, n, heads, dim, torch.bfloat16) for _ in range(2))
    first = pages * page - n
    kvc.cache_write(c, k.cuda(), v.cuda(), torch.arange(first, first + n, device="cuda"))
    qc, qs, _ = quantise(c.format, torch.stack((k, v), 1))
    assert torch.equal(c.codes[-1, :, :, -n:].cpu(), qc.permute(1, 2, 0, 3))
    assert int(torch.count_nonzero(c.codes[:64])) == 0
    out = torch.zeros(2, heads, n, dim, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    kvc.cache_read(c, i32(pages - 1)[None], i32(page - n), i32(0, n), out)
    want = (code_values(c.format, qc, None) * qs.double()[..., None]).permute(1, 2, 0, 3)
    assert torch.equal(out.cpu(), want.float())


def test_empty_calls():
    c = _filled(kvc.CACHE_E2M1, 2, 64, 16, 2, 6)
    before = _arrays(c)
    z = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    kvc.cache_write(c, z, z, torch.zeros(0, dtype=torch.int64, device="cuda"))
    _same(c, before)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out = torch.full((2, 2, 4, 64), 3.0, device="cuda")
    kvc.cache_read(c, i32(0, 1)[None], i32(5), i32(2, 2), out)
    kvc.cache_read(c, torch.zeros(0, 2, dtype=torch.int32, device="cuda"), i32(), i32(0), out)
    assert (out == 3.0).all() and kvc.read_result(c.res)[0] == kvc.OK
