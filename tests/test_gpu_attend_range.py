"""GPU: attention over the serving cache at the ends of the values' range: rows
as small as a write stores, zero rows beside very large ones, sums of many."""
import pytest
import torch

import transform_codec_b200 as kvc
from serving_ref import FORMATS, HostCache, attention, check_out, quantise
from test_gpu_attend import _randn, i32

pytestmark = pytest.mark.gpu


def _set_values(host, b, rows):
    """Sequence b's value rows [heads][n][dim], quantised as a write does."""
    pos = torch.arange(host.lens[b])
    page, at = host.table[b].long()[pos // host.page], pos % host.page
    codes, scales, micro = quantise(host.fmt, rows.transpose(0, 1))
    host.codes[page, 1, :, at], host.scales[page, 1, :, at] = codes, scales
    if micro is not None:
        host.micro[page, 1, :, at] = micro


def _rows(seed, heads, n, dim, low, high):
    """Rows whose largest magnitude is 2^low .. 2^high, spread over the logarithm; both ends are there."""
    x = _randn(seed, heads, n, dim)
    x = x / x.abs().amax(-1, keepdim=True)
    e = torch.linspace(low, high, n)[torch.randperm(n, generator=torch.Generator().manual_seed(seed))]
    return (x.double() * torch.exp2(e.double())[:, None]).float()


def _check(host, q, starts, prefix=None):
    """Against fp64. The logarithm of a scale of 2^-107 or 2^120 is off by 2^-22 of
    itself, and beside it a score keeps 2^-18: together 2^-14.9 of a weight, which
    is 2^-6.9 of the 2^-8 that bf16 weights are already granted."""
    n, Hq, D = q.shape
    att = kvc.Attention(q.dtype, Hq, host.heads, D, max_rows=n, max_seqs=len(host.lens),
                        max_queries=max(b - a for a, b in zip(starts, starts[1:])), max_kv=max(host.lens),
                        prefix_tokens=0 if prefix is None else prefix[0].shape[1])
    out = torch.zeros(n, Hq, D, dtype=q.dtype, device="cuda")
    lse = torch.zeros(n, Hq, device="cuda")
    att.run(q.cuda(), out, cache=host.gpu(), page_table=host.table.cuda(), kv_len=i32(host.lens),
            q_start=i32(starts), lse=lse, prefix=None if prefix is None else tuple(p.cuda() for p in prefix))
    assert kvc.read_result(att.res) == (kvc.OK, 0)
    want, wl, (tol, ltol) = attention(q, starts, host, prefix, None, D ** -0.5)
    check_out(out, lse, want, wl, (tol * (1 + 2.0 ** -6.9), ltol))
    return out


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim,group,queries", [(64, 4, 1), (128, 8, 1), (128, 8, 3)])
def test_rows_as_small_as_a_write_stores(fmt, dim, group, queries):
    """Largest magnitudes from 2^-96, the least that is not stored as zero: scales down to 2^-107."""
    host = HostCache(FORMATS[fmt], 2, dim, 16, [130, 40], seed=2)
    for b in range(2):
        _set_values(host, b, _rows(b, 2, host.lens[b], dim, -95.99, -90))
    assert (host.scales[host.scales > 0].min() < 2.0 ** -102)
    q = _randn(3, 2 * queries, 2 * group, dim, dt=torch.bfloat16, spread=1.5)
    out = _check(host, q, [0, queries, 2 * queries])
    assert (out != 0).any()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("queries", [1, 3])
@pytest.mark.parametrize("top", [1e13, 1e30, 1e38])
def test_zero_and_tiny_rows_beside_large_ones(fmt, queries, top):
    """Every token takes its share of the sum, whatever its values' size."""
    host = HostCache(FORMATS[fmt], 1, 128, 16, [70, 33, 2], seed=4)
    for b in range(3):
        x = _randn(b + 5, 1, host.lens[b], 128)
        x = x / x.abs().amax(-1, keepdim=True) * top
        x[:, 1::3] = 0.0
        x[:, 2::6] *= 2.0 ** -95 / top
        _set_values(host, b, x)
    q = _randn(3, 3 * queries, 8, 128, dt=torch.bfloat16, spread=0.5)
    _check(host, q, [0, queries, 2 * queries, 3 * queries])


@pytest.mark.parametrize("fmt", FORMATS)
def test_small_and_large_rows_next_to_a_prefix(fmt):
    host = HostCache(FORMATS[fmt], 2, 128, 16, [60, 35], seed=4)
    q = _randn(3, 2, 16, 128, dt=torch.bfloat16, spread=0.5)
    for size in (2.0 ** -90, 2.0 ** 70):
        for b in range(2):
            rows = _rows(b, 2, host.lens[b], 128, -95.9, -91) if size < 1 else _randn(b, 2, host.lens[b], 128) * size
            rows[:, 3::4] = 0.0
            _set_values(host, b, rows)
        k, v = (_randn(s, 2, 300, 128, dt=torch.bfloat16) for s in (1, 2))
        _check(host, q, [0, 1, 2], (k, v * size))


def test_sum_of_many_zero_rows():
    """70,000 tokens whose values are zero, most of them 2^7.5 times the weight of the first ones, on one block."""
    n, dim = 70000, 64
    host = HostCache(kvc.CACHE_INT8, 1, dim, 1024, [n], seed=4)
    pos = torch.arange(n)
    page, at = host.table[0].long()[pos // 1024], pos % 1024
    host.codes[page, 1, 0, at], host.scales[page, 1, 0, at] = 0, 0.0
    host.codes[page, 0, 0, at], host.scales[page, 0, 0, at] = 127, 7.5 * 0.6931471805599453 / 127 / dim
    host.codes[page[:64], 0, 0, at[:64]], host.scales[page[:64], 0, 0, at[:64]] = 0, 0.0
    q = torch.ones(1, 1, dim, dtype=torch.bfloat16)
    att = kvc.Attention(q.dtype, 1, 1, dim, max_rows=1, max_seqs=1, max_kv=n)
    att._ws_bytes = kvc.lib().kvc_attend_workspace_min(att._ref)
    out, lse = torch.ones(1, 1, dim, dtype=q.dtype, device="cuda"), torch.zeros(1, 1, device="cuda")
    att.run(q.cuda(), out, cache=host.gpu(), page_table=host.table.cuda(), kv_len=i32(host.lens), lse=lse, scale=1.0)
    want, wl, tol = attention(q, [0, 1], host, scale=1.0)
    check_out(out, lse, want, wl, tol)
    assert (out == 0).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("gap", [100, 128, 140])
def test_large_values_far_below_the_largest_score(fmt, gap):
    """Zero rows with scores 2^gap of the others', in parts and warps of their own, beside rows of 1e30: what the
    others weigh is below fp32's range and their share of the answer is not."""
    dim = 128
    for n, prefix_rows in ((70, 0), (2000, 0), (70, 200)):
        host = HostCache(FORMATS[fmt], 1, dim, 16, [n], seed=4)
        _set_values(host, 0, torch.cat((torch.zeros(1, 16, dim), _randn(5, 1, n - 16, dim) * 1e30), 1))
        pos = torch.arange(n)
        page, at = host.table[0].long()[pos // 16], pos % 16
        keys = torch.full((n, 1, dim), 0.0)
        keys[:16] = 1.0
        kc, ks, km = quantise(host.fmt, keys)
        host.codes[page, 0, :, at], host.scales[page, 0, :, at] = kc, ks
        if km is not None:
            host.micro[page, 0, :, at] = km
        prefix = None
        if prefix_rows:
            prefix = (torch.zeros(1, prefix_rows, dim).bfloat16(), _randn(6, 1, prefix_rows, dim, dt=torch.bfloat16))
        q = torch.ones(1, 8, dim, dtype=torch.bfloat16)
        scale = gap * 0.6931471805599453 / dim
        att = kvc.Attention(q.dtype, 8, 1, dim, max_rows=1, max_seqs=1, max_kv=n, prefix_tokens=prefix_rows)
        out, lse = torch.zeros(1, 8, dim, dtype=q.dtype, device="cuda"), torch.zeros(1, 8, device="cuda")
        att.run(q.cuda(), out, cache=host.gpu(), page_table=host.table.cuda(), kv_len=i32([n]), lse=lse, scale=scale,
                prefix=None if prefix is None else tuple(p.cuda() for p in prefix))
        want, wl, (tol, ltol) = attention(q, [0, 1], host, prefix, None, scale)
        assert want.abs().max() > 1e-14
        check_out(out, lse, want, wl, (tol * (1 + 2.0 ** -6.9), ltol))
